// The weight gradient of rows that were kept in FP8 with one E8M0 scale per 32
// columns:  dw[g][p][j] = sum over the group's rows i of X[i][p] * Y[i][j], where
// X or Y is code * 2^(scale - 127), and the other, and the matrix core's operands,
// bf16 or fp16.
//
// Scales lie across the reduction, which the scaled matrix instructions cannot
// take (theirs lie along it), so codes become 16-bit values on their way: they
// are copied to LDS as they are, half the bytes, and the thread that copied
// sixteen of a row turns them into 16-bit values (one instruction for two, exact
// in bf16), two steps before the matrix core has them.  In fp16, values past
// 65504 become infinite and those below 2^-14 lose bits.  The sums are those of
// the 16-bit weight gradient on the widened rows, to the bit.
//
// 32768 rows over 32 experts, 7168 x 4096, fp32 results (one MI355X): 2.26 to
// 2.32 ms, 0.83 to 0.85 PFLOP/s, the 16-bit gradient of the same rows 2.24,
// widening them first 2.37 and a copy of them in memory.  Matrix cores 39% busy
// at 1.92 GHz.  Timed in copies of the kernel: without its 3.8 GB of stores 1.88
// ms, of that without the copies 1.46, without reading fragments 1.69, without
// widening 1.66.
#include "grouped_product.h"

namespace gmmgm {

int wgrad_fp8_plan(const gmmgx_args* a, Plan* pl, bool* x8) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->x) || !given(a->dy) || !given(a->group_list) || !given(a->dw)) return GMMFR_ERR_NULLPTR;
  *x8 = a->x.dtype == GMMFR_DT_FLOAT8_E4M3FN;
  const gmmfr_tensor &rows = *x8 ? a->x : a->dy, &scale = *x8 ? a->x_scale : a->dy_scale;
  const gmmfr_tensor &other = *x8 ? a->dy : a->x, &none = *x8 ? a->dy_scale : a->x_scale;
  if (rows.dtype != GMMFR_DT_FLOAT8_E4M3FN) return GMMFR_ERR_DTYPE;
  if (!given(scale)) return GMMFR_ERR_NULLPTR;
  if (given(none)) return GMMFR_ERR_UNSUPPORTED;
  if (scale.dtype != GMMFR_DT_FLOAT8_E8M0) return GMMFR_ERR_DTYPE;
  gmmgw_args wide = {};
  wide.x = a->x;
  wide.dy = a->dy;
  (*x8 ? wide.x : wide.dy).dtype = other.dtype;  // as if they were widened
  wide.group_list = a->group_list;
  wide.dw = a->dw;
  wide.group_list_type = a->group_list_type;
  wide.accumulate = a->accumulate;
  wide.tuning_config = a->tuning_config;
  wide.tuning_config_len = a->tuning_config_len;
  const int st = wgrad_plan(&wide, pl);
  if (st != GMMFR_OK) return st;
  const int64_t columns = *x8 ? pl->p.k : pl->p.n;
  if (columns % 64 != 0 || !shape_is(scale, 3, pl->p.m, columns / 64, 2)) return GMMFR_ERR_SHAPE;
  if (aligned({&scale}) != GMMFR_OK) return GMMFR_ERR_ALIGN;
  (*x8 ? pl->p.xs : pl->p.ws) = (const uint8_t*)scale.data;
  return GMMFR_OK;
}

// The 16-bit weight gradient's tiles, with short stages for the smaller too: its
// two operands' stages would not fit twice a CU beside the codes otherwise.
template <int ENC, int EIGHT>
hipError_t launch_fp8(Plan& pl, hipStream_t s) {
  void* args[] = {&pl.p};
  const void* kernel = pl.kind == kLarge
                           ? (const void*)product_kernel<ENC, true, true, true, false, 256, 256, 32, 2, 2, 4, false, 1, kStore, EIGHT>
                           : (const void*)product_kernel<ENC, true, true, true, false, 128, 128, 32, 2, 2, 4, false, 2, kStore, EIGHT>;
  return hipLaunchKernel(kernel, dim3(pl.grid), dim3(256), args, (size_t)(2 * pl.p.e + 1) * 4, s);
}

}  // namespace gmmgm

extern "C" {

using namespace gmmgm;

int gmm_grouped_matmul_wgrad_fp8_workspace(const gmmgx_args* args, size_t* workspace_bytes) {
  Plan pl;
  bool x8;
  const int st = wgrad_fp8_plan(args, &pl, &x8);
  if (st != GMMFR_OK) return st;
  if (!workspace_bytes) return GMMFR_ERR_NULLPTR;
  *workspace_bytes = 0;
  return GMMFR_OK;
}

int gmm_grouped_matmul_wgrad_fp8(const gmmgx_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  Plan pl;
  bool x8;
  const int st = wgrad_fp8_plan(args, &pl, &x8);
  if (st != GMMFR_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t done = pl.enc == kBf16 ? (x8 ? launch_fp8<kBf16, kX8>(pl, s) : launch_fp8<kBf16, kW8>(pl, s))
                                          : (x8 ? launch_fp8<kF16, kX8>(pl, s) : launch_fp8<kF16, kW8>(pl, s));
  return done == hipSuccess ? GMMFR_OK : GMMFR_ERR_HIP;
}

}  // extern "C"
