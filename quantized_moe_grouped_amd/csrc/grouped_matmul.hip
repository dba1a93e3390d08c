// Products grouped by expert, without a combine, and the gradient of the
// weights: the instances of product_kernel (grouped_product.h) that store their
// sums, plain or through SwiGLU, and the entry points.
#include "grouped_product.h"

namespace gmmgm {

int product_run(const gmmgm_args* a, void* stream) {
  Plan pl;
  const int st = product_plan(a, &pl);
  if (st != GMMFR_OK) return st;
  if (pl.p.m == 0) return GMMFR_OK;
  hipStream_t s = (hipStream_t)stream;
  auto with = [&](auto enc_) -> hipError_t {
    constexpr int ENC = decltype(enc_)::value;
    constexpr bool MX = ENC == kFp4 || ENC == kFp8;
    if constexpr (!MX) {
      if (pl.col) return pl.glu ? launch<ENC, false, true, false, true>(pl, s) : launch<ENC, false, true, false, false>(pl, s);
    }
    return pl.glu ? launch<ENC, false, false, false, true>(pl, s) : launch<ENC, false, false, false, false>(pl, s);
  };
  const hipError_t done = pl.enc == kBf16   ? with(std::integral_constant<int, kBf16>{})
                          : pl.enc == kF16  ? with(std::integral_constant<int, kF16>{})
                          : pl.enc == kFp4  ? with(std::integral_constant<int, kFp4>{})
                                            : with(std::integral_constant<int, kFp8>{});
  return done == hipSuccess ? GMMFR_OK : GMMFR_ERR_HIP;
}

int wgrad_run(const gmmgw_args* a, void* stream) {
  Plan pl;
  const int st = wgrad_plan(a, &pl);
  if (st != GMMFR_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t done = pl.enc == kBf16 ? (pl.few ? launch<kBf16, true, true, true, false, kStore, true>(pl, s)
                                                    : launch<kBf16, true, true, true, false>(pl, s))
                                          : (pl.few ? launch<kF16, true, true, true, false, kStore, true>(pl, s)
                                                    : launch<kF16, true, true, true, false>(pl, s));
  return done == hipSuccess ? GMMFR_OK : GMMFR_ERR_HIP;
}

}  // namespace gmmgm

extern "C" {

using namespace gmmgm;

int gmm_grouped_matmul_plan(const gmmgm_args* args, gmmgm_plan_info* info) {
  Plan pl;
  const int st = describe(product_plan(args, &pl), pl, info);
  if (st == GMMFR_OK && pl.p.m == 0) info->grid = 0;
  return st;
}

int gmm_grouped_matmul_workspace(const gmmgm_args* args, size_t* workspace_bytes) {
  Plan pl;
  const int st = product_plan(args, &pl);
  if (st != GMMFR_OK) return st;
  if (!workspace_bytes) return GMMFR_ERR_NULLPTR;
  *workspace_bytes = 0;
  return GMMFR_OK;
}

int gmm_grouped_matmul(const gmmgm_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  return product_run(args, stream);
}

int gmm_grouped_matmul_wgrad_workspace(const gmmgw_args* args, size_t* workspace_bytes) {
  Plan pl;
  const int st = wgrad_plan(args, &pl);
  if (st != GMMFR_OK) return st;
  if (!workspace_bytes) return GMMFR_ERR_NULLPTR;
  *workspace_bytes = 0;
  return GMMFR_OK;
}

int gmm_grouped_matmul_wgrad_plan(const gmmgw_args* args, gmmgm_plan_info* info) {
  Plan pl;
  return describe(wgrad_plan(args, &pl), pl, info);
}

int gmm_grouped_matmul_wgrad(const gmmgw_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  return wgrad_run(args, stream);
}

}  // extern "C"
