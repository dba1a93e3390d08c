// The weight gradient of rows that were kept in FP8 with one E8M0 scale per 32
// columns:  dw[g][p][j] = sum over the group's rows i of X[i][p] * Y[i][j], where
// X or Y is code * 2^(scale - 127), and the other, and the matrix core's operands,
// bf16 or fp16.
//
// Scales lie across the reduction, which the scaled matrix instructions cannot
// take (theirs lie along it), so codes become 16-bit values on their way: they
// are copied to LDS as they are, half the bytes, and the thread that copied
// sixteen of a row turns them into 16-bit values (one instruction for two), a
// step before the matrix core has them: the nearest of the type.  bf16 holds all
// of them under scales of 2^-124 and more, and below that those from its least
// subnormal, 2^-133, on; in fp16 values past 65504 become infinite and those
// below 2^-14 lose bits.  The sums are those of the 16-bit weight gradient on the
// widened rows, to the bit, where the groups' rows are not split.
//
// 32768 rows over 32 experts, 7168 x 4096, fp32 results (one MI355X): 2.26 to
// 2.33 ms, 0.83 to 0.85 PFLOP/s, the 16-bit gradient of the same rows 2.24,
// widening them first 2.37 and a copy of them in memory.  Matrix cores 40% busy
// at 1.85 GHz.  Timed in copies of the kernel: without its 3.8 GB of stores 1.88
// ms, of that without the copies 1.46, without reading fragments 1.69, without
// widening 1.66.
#include "grouped_product.h"

namespace gmmgm {

// Where the tiles leave workgroups without one and groups are long, the rows of
// each are split into parts of 1024 and more: their sums go to a workspace, one
// after the other in memory, and sum_parts adds them in their order.  Long by the
// average, as the host knows no more: a list with one long group among short ones
// is not split, nor are 8000 rows over 4 experts of 512 x 512 (35 us, where 8192
// rows take 27).  256-row tiles if their parts fill three quarters of the chip
// (us, whole, and split with 128-row and 256-row tiles; fp32 results):
//   1 of 1024 x 1024, 16384 rows  248,  59,  55    1 of 512 x 512, 8192 rows  124, 30, 46
//   2 of 832 x 864, 25694         198,  69,  66    4 of 512 x 512, 16384       65, 31, 47
//   1 of 2048 x 2048, 16384       240, 179, 140    1 of 128 x 128, 4096        64, 25, 39
int parts_of(const Params& p, Kind kind) {
  const int64_t tiles = p.e * ceil_div(p.k, kTileM[kind]) * ceil_div(p.n, kTileN[kind]);
  int64_t parts = 256 * kPerCu[kind] / tiles;
  if (parts > p.m / p.e / 1024) parts = p.m / p.e / 1024;
  if (parts > 16) parts = 16;
  return parts < 2 ? 1 : (int)parts;
}

typedef float sum4 __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(256) void sum_parts(const sum4* parts, void* dw, int64_t fours, int splits, int out, int accumulate) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < fours; i += (int64_t)gridDim.x * 256) {
    sum4 v = parts[i];
    for (int s = 1; s < splits; ++s) {
      const sum4 o = parts[s * fours + i];
      v = sum4{v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w};
    }
    if (out == kOutF32) {
      if (accumulate) {
        const sum4 o = ((const sum4*)dw)[i];
        v = sum4{v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w};
      }
      ((sum4*)dw)[i] = v;
    } else if (out == kOutF16) {
      typedef _Float16 v4h __attribute__((ext_vector_type(4)));
      ((v4h*)dw)[i] = v4h{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
    } else {
      typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
      ((v4bf*)dw)[i] = v4bf{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
    }
  }
}

int wgrad_fp8_plan(const gmmgx_args* a, Plan* pl, bool* x8, size_t* workspace) {
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
  const int st = wgrad_plan(&wide, pl, true);
  if (st != GMMFR_OK) return st;
  const int64_t columns = *x8 ? pl->p.k : pl->p.n;
  if (columns % 64 != 0 || !shape_is(scale, 3, pl->p.m, columns / 64, 2)) return GMMFR_ERR_SHAPE;
  if (aligned({&scale}) != GMMFR_OK) return GMMFR_ERR_ALIGN;
  (*x8 ? pl->p.xs : pl->p.ws) = (const uint8_t*)scale.data;
  Params& p = pl->p;
  int64_t expected, height, cap;
  tuning(a->tuning_config, a->tuning_config_len, &expected, &height, &cap);
  if (height == 0) {
    const int parts = parts_of(p, kLarge);
    if (parts > 1 && parts * p.e * ceil_div(p.k, 256) * ceil_div(p.n, 256) >= 192) pl->kind = kLarge;
    p.tiles_m = (int32_t)ceil_div(p.k, kTileM[pl->kind]);
    p.tiles_n = (int32_t)ceil_div(p.n, kTileN[pl->kind]);
  }
  p.splits = parts_of(p, pl->kind);
  pl->grid = grid_of(*pl, (int64_t)p.e * p.splits * p.tiles_m * p.tiles_n, cap);
  *workspace = p.splits > 1 ? (size_t)p.splits * p.e * p.k * p.n * 4 : 0;
  return GMMFR_OK;
}

// The 16-bit weight gradient's tiles, with short stages for the smaller too: its
// two operands' stages would not fit twice a CU beside the codes otherwise.
template <int ENC, int EIGHT>
hipError_t launch_fp8(Plan& pl, hipStream_t s) {
  pl.p.grid = pl.grid;
  void* args[] = {&pl.p};
  const void* kernel = pl.kind == kLarge
                           ? (const void*)product_kernel<ENC, true, true, true, false, 256, 256, 32, 2, 2, 4, false, 1, kStore, EIGHT>
                           : (const void*)product_kernel<ENC, true, true, true, false, 128, 128, 32, 2, 2, 4, false, 2, kStore, EIGHT>;
  return hipLaunchKernel(kernel, dim3(pl.grid), dim3(256), args, (size_t)(2 * pl.p.e + 1) * 4, s);
}

int launch_parts(Plan& pl, bool x8, hipStream_t s) {
  const hipError_t done = pl.enc == kBf16 ? (x8 ? launch_fp8<kBf16, kX8>(pl, s) : launch_fp8<kBf16, kW8>(pl, s))
                                          : (x8 ? launch_fp8<kF16, kX8>(pl, s) : launch_fp8<kF16, kW8>(pl, s));
  return done == hipSuccess ? GMMFR_OK : GMMFR_ERR_HIP;
}

}  // namespace gmmgm

extern "C" {

using namespace gmmgm;

int gmm_grouped_matmul_wgrad_fp8_workspace(const gmmgx_args* args, size_t* workspace_bytes) {
  Plan pl;
  bool x8;
  size_t need;
  const int st = wgrad_fp8_plan(args, &pl, &x8, &need);
  if (st != GMMFR_OK) return st;
  if (!workspace_bytes) return GMMFR_ERR_NULLPTR;
  *workspace_bytes = need;
  return GMMFR_OK;
}

int gmm_grouped_matmul_wgrad_fp8_plan(const gmmgx_args* args, gmmgm_plan_info* info) {
  Plan pl;
  bool x8;
  size_t need;
  return describe(wgrad_fp8_plan(args, &pl, &x8, &need), pl, info);
}

int gmm_grouped_matmul_wgrad_fp8(const gmmgx_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  Plan pl;
  bool x8;
  size_t need;
  int st = wgrad_fp8_plan(args, &pl, &x8, &need);
  if (st != GMMFR_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  Params& p = pl.p;
  if (need == 0) return launch_parts(pl, x8, s);
  if (!workspace || workspace_bytes < need) return GMMFR_ERR_WORKSPACE;
  if (((uintptr_t)workspace & 15u) != 0) return GMMFR_ERR_ALIGN;
  void* dw = p.y;
  int out = p.out, accumulate = p.accumulate, splits = p.splits;
  p.y = workspace;
  p.out = kOutF32;
  p.accumulate = 0;
  st = launch_parts(pl, x8, s);
  if (st != GMMFR_OK) return st;
  int64_t fours = (int64_t)p.e * p.k * p.n / 4;
  void* kargs[] = {&workspace, &dw, &fours, &splits, &out, &accumulate};
  const int64_t groups = ceil_div(fours, 256);
  return hipLaunchKernel((const void*)sum_parts, dim3((uint32_t)(groups < 2048 ? groups : 2048)), dim3(256), kargs, 0, s) == hipSuccess
             ? GMMFR_OK
             : GMMFR_ERR_HIP;
}

}  // extern "C"
