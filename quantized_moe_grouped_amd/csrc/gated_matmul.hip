// The gated feed-forward block of a layer's experts (or, with one group, of a
// dense layer), for training: both projections, the activation and the product
// of the two in one kernel, and the way back through all three from behind the
// block's last projection.
//
//   forward:  (u | v) = x W,  h = a(u) v;  (u | v) kept in 16 bits, in FP8, or not
//   backward: dh = dy Wd^T,  du = dh v a'(u),  dv = dh a(u),  h = a(u) v again
//
// Instances of product_kernel (grouped_product.h) whose epilogue works on the
// fp32 sums in registers (gate.h): neither the projections of the forward pass
// nor dh of the backward pass goes through memory in between.
//
// What bounds it (one MI355X, bf16, inputs not in the caches):
//   - forward, 32768 rows over 32 experts of 7168 x 2 2048, (e,k,n): 1.67 ms with
//     nothing kept, 1.74 in 16 bits, 1.72 in FP8 = 1.12 PFLOP/s: the products
//     (SwiGLU alone 1.70), matrix cores 67% busy at the clock that the card's
//     power leaves; 12% more rows are multiplied than there are.
//   - backward of the same from FP8: 1.04 ms.  The product alone takes 0.91, half
//     a round of 4.5 with half of the chip; 0.41 GB more are written and read a
//     call, which is 0.08 ms at the copy rate.
//     Timed in copies of the kernel: without the stores 0.99, without the loads
//     1.05, without the gate's arithmetic 1.07 (of 1.09).
//   - one token through 8 of 32 experts: the weights, 6.5 TB/s.
// The way back's large tile has four waves of 128 x 128, whose 256 accumulation
// registers leave the others free for what was kept, asked for three blocks
// ahead, and one loop over the 16 blocks (1337 -> 1062 us; unrolled, with the
// values spilled, 1252; eight waves of 64 x 128, one block ahead: 1103; the first
// blocks' asked for at the tile's begin: 1068).
#include "grouped_product.h"

namespace gmmgm {

// What is kept: nothing, x's own type, or FP8 with E8M0 scales; (m, 2 f).
int kept_plan(const gmmfr_tensor& kept, const gmmfr_tensor& scale, int type, int64_t m, int64_t f, Params* p) {
  if (!given(kept)) {
    if (given(scale)) return GMMFR_ERR_NULLPTR;
    p->keep = kKeepNone;
  } else if (kept.dtype == GMMFR_DT_FLOAT8_E4M3FN) {
    if (!given(scale)) return GMMFR_ERR_NULLPTR;
    if (scale.dtype != GMMFR_DT_FLOAT8_E8M0) return GMMFR_ERR_DTYPE;
    if (f % 32 != 0 || !shape_is(scale, 3, m, 2 * f / 64, 2)) return GMMFR_ERR_SHAPE;
    p->keep = kKeepFp8;
  } else {
    if (kept.dtype != type) return GMMFR_ERR_DTYPE;
    if (given(scale)) return GMMFR_ERR_UNSUPPORTED;
    p->keep = kKeepFull;
  }
  if (p->keep != kKeepNone && !shape_is(kept, 2, m, 2 * f)) return GMMFR_ERR_SHAPE;
  p->kept = kept.data;
  p->kept_scale = (uint8_t*)scale.data;
  return aligned({&kept, &scale});
}

bool in_16_bits(int dtype) { return dtype == GMMFR_DT_BFLOAT16 || dtype == GMMFR_DT_FLOAT16; }

int forward_plan(const gmmgf_args* a, Plan* pl) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->x) || !given(a->w) || !given(a->group_list) || !given(a->h)) return GMMFR_ERR_NULLPTR;
  if (!in_16_bits(a->x.dtype) || a->h.dtype != a->x.dtype) return GMMFR_ERR_DTYPE;
  if (a->activation != GMMGF_ACT_SWIGLU && a->activation != GMMGF_ACT_GEGLU) return GMMFR_ERR_ATTR;
  gmmgm_args product = {};
  product.x = a->x;
  product.w = a->w;
  product.group_list = a->group_list;
  product.y = a->h;
  product.group_list_type = a->group_list_type;
  product.transpose_w = a->transpose_w;
  product.activation = GMMGM_ACT_SWIGLU;  // a gate of its columns' first half
  product.tuning_config = a->tuning_config;
  product.tuning_config_len = a->tuning_config_len;
  // (a scale's 32 columns are one tile's: none thinner where they are kept in FP8)
  const bool fp8 = given(a->kept) && a->kept.dtype == GMMFR_DT_FLOAT8_E4M3FN;
  const int st = product_plan(&product, pl, kFewTiles | (fp8 ? 0 : kThinGate));
  if (st != GMMFR_OK) return st;
  pl->p.act = a->activation;
  pl->p.hidden = nullptr;
  return kept_plan(a->kept, a->kept_scale, a->x.dtype, pl->p.m, pl->p.n / 2, &pl->p);
}

int backward_plan(const gmmgb_args* a, Plan* pl) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->dy) || !given(a->w) || !given(a->group_list) || !given(a->kept) || !given(a->d)) return GMMFR_ERR_NULLPTR;
  if (!in_16_bits(a->dy.dtype) || a->d.dtype != a->dy.dtype) return GMMFR_ERR_DTYPE;
  if (given(a->h) && a->h.dtype != a->dy.dtype) return GMMFR_ERR_DTYPE;
  if (a->activation != GMMGF_ACT_SWIGLU && a->activation != GMMGF_ACT_GEGLU) return GMMFR_ERR_ATTR;
  if (a->d.ndim != 2 || a->d.dims[1] % 2 != 0) return GMMFR_ERR_SHAPE;
  gmmgm_args product = {};
  product.x = a->dy;
  product.w = a->w;
  product.group_list = a->group_list;
  product.y = a->d;
  product.y.dims[1] /= 2;  // the sums are dh
  product.group_list_type = a->group_list_type;
  product.transpose_w = a->transpose_w;
  product.activation = GMMGM_ACT_NONE;
  product.tuning_config = a->tuning_config;
  product.tuning_config_len = a->tuning_config_len;
  int st = product_plan(&product, pl, kFewTiles);
  if (st != GMMFR_OK) return st;
  Params& p = pl->p;
  if (p.n > 32768) return GMMFR_ERR_SHAPE;  // 2 f, as in the forward pass
  if (given(a->h) && !shape_is(a->h, 2, p.m, p.n)) return GMMFR_ERR_SHAPE;
  p.act = a->activation;
  p.hidden = a->h.data;
  st = aligned({&a->h});
  return st != GMMFR_OK ? st : kept_plan(a->kept, a->kept_scale, a->dy.dtype, p.m, p.n, &p);
}

template <bool GLU, int FORM>
int run(Plan& pl, void* stream) {
  if (pl.p.m == 0) return GMMFR_OK;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t done = pl.enc == kBf16 ? (pl.col ? launch<kBf16, false, true, false, GLU, FORM>(pl, s)
                                                    : launch<kBf16, false, false, false, GLU, FORM>(pl, s))
                                          : (pl.col ? launch<kF16, false, true, false, GLU, FORM>(pl, s)
                                                    : launch<kF16, false, false, false, GLU, FORM>(pl, s));
  return done == hipSuccess ? GMMFR_OK : GMMFR_ERR_HIP;
}

int no_workspace(int status, size_t* workspace_bytes) {
  if (status != GMMFR_OK) return status;
  if (!workspace_bytes) return GMMFR_ERR_NULLPTR;
  *workspace_bytes = 0;
  return GMMFR_OK;
}

}  // namespace gmmgm

extern "C" {

using namespace gmmgm;

int gmm_gated_matmul_workspace(const gmmgf_args* args, size_t* workspace_bytes) {
  Plan pl;
  return no_workspace(forward_plan(args, &pl), workspace_bytes);
}

int gmm_gated_matmul_plan(const gmmgf_args* args, gmmgm_plan_info* info) {
  Plan pl;
  const int st = describe(forward_plan(args, &pl), pl, info);
  if (st == GMMFR_OK && pl.p.m == 0) info->grid = 0;
  return st;
}

int gmm_gated_matmul(const gmmgf_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  Plan pl;
  const int st = forward_plan(args, &pl);
  return st != GMMFR_OK ? st : run<true, kGated>(pl, stream);
}

int gmm_gated_matmul_backward_workspace(const gmmgb_args* args, size_t* workspace_bytes) {
  Plan pl;
  return no_workspace(backward_plan(args, &pl), workspace_bytes);
}

int gmm_gated_matmul_backward_plan(const gmmgb_args* args, gmmgm_plan_info* info) {
  Plan pl;
  const int st = describe(backward_plan(args, &pl), pl, info);
  if (st == GMMFR_OK && pl.p.m == 0) info->grid = 0;
  return st;
}

int gmm_gated_matmul_backward(const gmmgb_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  Plan pl;
  const int st = backward_plan(args, &pl);
  if (st != GMMFR_OK) return st;
  return pl.p.keep == kKeepFp8 ? run<false, kBackFp8>(pl, stream) : run<false, kBackFull>(pl, stream);
}

}  // extern "C"
