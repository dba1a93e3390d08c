// Products grouped by expert, without a combine: rows of x sorted by expert
// and split by groupList, each group multiplied by its expert's weights, and
// the gradient of the weights.
//
//   product:  y[i][j]     = sum_q x[i][q] * w[g(i)][q][j]
//   SwiGLU:   y[i][j]     = u / (1 + exp(-u)) * v,  u = column j and v = column n/2 + j of the product
//   wgrad:    dw[g][p][j] = sum_{i in g} x[i][p] * dy[i][j]
//
// Operands are bf16 or fp16, or microscaled: FP8 E4M3 or FP4 E2M1 rows with
// FP4 E2M1 weights and one E8M0 scale per 32 values along the reduction.
// Sums run in fp32 on the matrix cores; the result is rounded once, on
// storing.  The gated block's forms (gate.h, gated_matmul.hip) work on the sums
// before that; the weight gradient takes one operand in FP8 with scales across
// the reduction, too (wgrad_fp8.hip).
//
// One kernel template, product_kernel: C(M,N) += A(M,R) * B(R,N) over the
// tiles of all experts.  In the product M is the group's rows, N the weight
// columns and R = k; in wgrad M = k, N = n and R the group's rows, which both
// operands then hold along their slow axis.
//
//   - The grid is persistent; tiles come in a raster that gives each XCD
//     blocks of neighbouring tiles (shared operand panels in its L2).
//   - Operands go HBM -> LDS with buffer_load_dwordx4 ... lds, 16 bytes per
//     lane, no VGPRs.  The buffer descriptor ends with the group's last row
//     (or the reduction's last row), so whatever lies past it arrives in LDS
//     as zeros: ragged groups and odd sizes need no other masking and no row
//     of another group is multiplied.
//   - The copies of one running stream of k-steps cross tile borders: the
//     next tile's first stages load under the present tile's epilogue.
//   - v_mfma_f32_32x32x16_{bf16,f16} or v_mfma_scale_f32_32x32x64_f8f6f4 with
//     the weights as the instruction's A operand and the rows as B: each lane
//     then holds four neighbouring columns of one row, and a swap of two
//     registers between the wave's halves makes them eight, stored in 16
//     bytes.
//   - Fragments of the next slice are read between the present one's products in
//     the 256-row tiles: all at once before them they hold the LDS, and the
//     waves' issue (bf16 and FP4 products 1-2% slower, the gated forms 1-2%,
//     weight gradients of 1024 rows an expert and more 4%, those of FP8 rows
//     2-4%).  Before them (EARLY) where that costs nothing and the reads
//     between them do: 128-row tiles, whose two workgroups a CU hide each
//     other's (between: 1-2% slower; not those of FP8 rows, alike), FP8 with FP4
//     (2-4%), and 16-bit weight gradients of shorter groups (16 experts of 1024 x
//     1024, 200 rows each that are not in the caches: 25 us, between 26 to 30 from
//     box to box).
//
// What bounds it (one MI355X; rows over experts):
//   - 16 bit, 256-row tiles, 32768 x 2048 x 7168 over 32, (e,k,n): 0.90 to 0.95
//     ms from box to box, 1.02 to 1.06 PFLOP/s.  Matrix cores busy 67% of the
//     cycles at the clock that the card's power leaves (1.85 GHz, within three
//     calls 1.31); between them the waits for LDS and barriers.
//   - weight gradient of the same: 1.10 ms, 49% busy: one workgroup a CU (its
//     sums fill the registers), whose 1.9 GB of fp32 results go out ahead of
//     copies that the next tile's first step waits for.
//   - FP4, 131072 x 7168 x 4096 over 32, SwiGLU: 2.01 to 2.08 ms, 3.7 to 3.8
//     PFLOP/s, 54% busy: a product is a quarter of the 16-bit one's time for the
//     same bytes copied and read.
//   - FP8 with FP4, 30001 x 2112 x 7152 over 64: 0.61 ms, 47% busy; a third of
//     the rows multiplied do not exist, and reads of 64-byte rows of weights
//     conflict in 28% of the LDS' active cycles.
//   - rows whose bytes are no multiple of 128 cost twice the requests to the
//     L2: fp16, 20011 rows over 64, 2040 columns, 128-row tiles: 1.02 ms with
//     k = 7160, 0.80 ms with 7168.
//   - narrow tiles: HBM; bf16 weights stream at 4.9 to 6.4 TB/s, 256 experts'
//     FP4 weights under 2048 skewed rows at 4.2 (0.48 ms).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "../../include/gmmfr.h"
#include "gate.h"

namespace gmmgm {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
#define LDS_PTR(T) __attribute__((address_space(3))) T*

constexpr int kMaxExperts = 1024;
constexpr int kXcds = 8;
constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset past every descriptor's end

// operand encodings
enum Enc { kBf16 = 0, kF16 = 1, kFp4 = 2, kFp8 = 3 };  // of the rows; weights: the same, or FP4 with kFp4 and kFp8
enum Out { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2 };
// what becomes of a tile's sums: stored (with GLU through SwiGLU); the gated
// block's forward pass (GLU) and its way back (the sums are dh) from what was
// kept in 16 bits or in FP8
enum Form { kStore = 0, kGated = 1, kBackFull = 2, kBackFp8 = 3 };
// weight gradient: the operand that is FP8 with a scale per 32 of its columns
enum Eight { kNone8 = 0, kX8 = 1, kW8 = 2 };

struct Params {
  const void* x;             // (m,k); 16-bit, FP8, or FP4 (m,k/2)
  const void* w;             // weights, or dy (m,n) for wgrad
  const uint8_t* xs;         // E8M0 (m, k/32)
  const uint8_t* ws;         // E8M0 (e, n, k/32)
  const int64_t* group_list; // (e)
  void* y;                   // (m, n or n/2), or dw (e,k,n)
  int64_t m, k, n;
  int32_t e, cumulative;     // groupList holds ends (type 0) instead of counts
  int32_t tiles_m, tiles_n;  // tiles along M (wgrad) and N
  int32_t out, accumulate;
  int32_t grid;              // workgroups (gridDim lies behind all this, a line of arguments more to fetch: 0.25 us)
  // gated forms: what is kept of both projections (an output, or the way back's
  // input) as (m, 2 n') with n' the columns of h, and h itself (way back)
  void* kept;
  uint8_t* kept_scale;       // E8M0 (m, 2 n'/32) where it is kept in FP8
  void* hidden;
  int32_t keep, act;
  int32_t splits;            // weight gradient of FP8 rows: parts of every group's rows
};

__device__ __forceinline__ int64_t uniform64(int64_t x) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)x));
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(const LDS_PTR(void))p; }

// 16 (or 4) bytes per lane from buffer `r` at byte offset `off` to LDS: lane i
// of the wave fills [lds + 16 i, lds + 16 i + 16).  Offsets at or past the
// descriptor's end give zeros.  Inline asm because the compiler would
// otherwise wait for every copy in flight before each LDS read; the kernel
// waits itself (wait_vmcnt) before the barrier that publishes a stage.  No
// output registers; M0 is used by nothing else here.
__device__ __forceinline__ void copy16(v4i r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(off), "s"(r)
               : "memory");
}
// The same past the caches, for weights that are read once.
__device__ __forceinline__ void copy16_once(v4i r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(off), "s"(r)
               : "memory");
}
__device__ __forceinline__ void copy4(v4i r, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(off), "s"(r)
               : "memory");
}

// A raw buffer over [base, base + bytes), bytes at most 2^31.
__device__ __forceinline__ v4i buffer(const void* base, uint32_t bytes) {
  const int64_t b = uniform64((int64_t)base);
  return v4i{(int)b, (int)((b >> 32) & 0xFFFF), __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Barrier that publishes this wave's LDS writes and finished reads, without
// waiting for copies in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS position of 16-byte chunk c of row r, C chunks a row.  Rows along the
// reduction's fast axis: 16 rows read at one chunk index (ds_read_b128) fall
// on 16 different chunks of the 256-byte bank window.
template <int C>
__device__ __forceinline__ int swz_row(int r) {
  if constexpr (C == 4) return ((r >> 1) ^ (r >> 3)) & 3;
  else if constexpr (C == 8) return (r ^ ((r >> 3) & 1)) & 7;
  else return r & 15;
}
// Rows across the reduction, read with ds_read_b64_tr_b16: one read of 32
// lanes touches 4 rows x 4 chunks (lanes 0-31) or 2 x 4 rows x 2 chunks; the
// rows' chunks are moved apart by whole groups of 4 chunks, and by 2 for the
// second set of rows.  Two rows of 8 chunks share one window: only bit 1 of r
// needs the move there.
template <int C>
__device__ __forceinline__ int swz_col(int r) {
  if constexpr (C >= 16) return ((r & 3) << 2) | (((r >> 3) & 1) << 1);
  else return (((r >> 1) & 1) << 2) | (((r >> 3) & 1) << 1);
}

// groupList -> s_ends[g] (end row of expert g) and s_pre[g] (tiles before
// expert g; s_pre[e] = all).  Device data are not trusted: entries are clamped
// to [0, m], type-0 ends become the running maximum and type-1 ends the
// running sum capped at m.  Every wave scans 64 entries a round in registers
// (all loads first); one wave writes.  Sums of two values below 2^31 fit 32
// bits, so the capped sum needs no more.
static __device__ void group_table(const Params& p, int bm, int32_t* s_ends, int32_t* s_pre) {
  const int lane = threadIdx.x & 63;
  constexpr int kRounds = kMaxExperts / 64;
  const int rounds = (p.e + 63) / 64;
  uint32_t v[kRounds];
#pragma unroll
  for (int b = 0; b < kRounds; ++b) {
    v[b] = 0;
    if (b < rounds) {
      const int g = b * 64 + lane;
      const int64_t c = g < p.e ? p.group_list[g] : 0;
      v[b] = (uint32_t)(c < 0 ? 0 : (c > p.m ? p.m : c));
    }
  }
  const uint32_t m = (uint32_t)p.m;
  uint32_t end_carry = 0, tile_carry = 0;
  const bool writer = threadIdx.x < 64;
#pragma unroll
  for (int b = 0; b < kRounds; ++b) {
    if (b < rounds) {
      const int g = b * 64 + lane;
      uint32_t x = v[b];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)x, d);
        if (lane >= d) x = p.cumulative ? max(x, o) : min(x + o, m);
      }
      x = p.cumulative ? max(x, end_carry) : min(x + end_carry, m);
      uint32_t before = (uint32_t)__shfl_up((int)x, 1);
      if (lane == 0) before = end_carry;
      end_carry = (uint32_t)__shfl((int)x, 63);
      uint32_t t = g < p.e ? ((x - before + bm - 1) / bm) * (uint32_t)p.tiles_n : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)t, d);
        if (lane >= d) t += o;
      }
      t += tile_carry;
      tile_carry = (uint32_t)__shfl((int)t, 63);
      if (writer && g < p.e) {
        s_ends[g] = (int32_t)x;
        s_pre[g + 1] = (int32_t)t;
      }
    }
  }
  if (threadIdx.x == 0) s_pre[0] = 0;
  __syncthreads();
}

// The experts whose groups are longer than twice the average first, the others
// from the end: a weight gradient's tiles last as long as their group, and long
// ones that began last would run alone (FP8 rows, 6007 of them skewed over 48 of
// 1088 x 1600, results of 16 bits: 121 -> 105 us; over such lists of other sizes
// between 15% less and 8% more).  Not for rows of 16 bits: over thirty skewed
// lists it took between 10% less and 13% more, and 2% more of even ones.  One
// round of 64 experts a time, few instructions: every workgroup does this before
// its first copy.
static __device__ void length_order(const Params& p, const int32_t* s_ends, int32_t* s_order) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const uint64_t below = (1ull << lane) - 1;
    int front = 0, back = p.e;
#pragma unroll 1
    for (int g = lane; g - lane < p.e; g += 64) {
      const int rows = g < p.e ? s_ends[g] - (g ? s_ends[g - 1] : 0) : 0;
      const bool is = (int64_t)rows * p.e > 2 * p.m;
      const uint64_t all = __ballot(g < p.e), longs = __ballot(is), rest = all & ~longs;
      if (g < p.e) s_order[is ? front + __popcll(longs & below) : back - 1 - __popcll(rest & below)] = g;
      front += __popcll(longs);
      back -= __popcll(rest);
    }
  }
  __syncthreads();
}

struct Tile {
  int g;       // expert
  int m0;      // first row along M: a row of x, or of dw
  int valid;   // rows of the tile that exist
  int n0;      // first column (SwiGLU: of y)
  int r0, r1;  // the reduction's range (wgrad: the group's rows)
  bool alone;  // the group has no other tile along M
  int part;    // of the group's rows (weight gradient of FP8 rows)
};

template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// f(i) of the i in [LO, HI) that is known only when it runs, by halving.
template <int LO, int HI, typename F>
__device__ __forceinline__ void one_of(int i, F&& f) {
  if constexpr (HI - LO == 1) {
    f(std::integral_constant<int, LO>{});
  } else {
    if (i < (LO + HI) / 2) one_of<LO, (LO + HI) / 2>(i, f);
    else one_of<(LO + HI) / 2, HI>(i, f);
  }
}

// ENC: operand encoding.  XCOL / WCOL: the operand's fast axis is M / N (16
// bit only) instead of the reduction.  WGRAD: see above.  GLU: SwiGLU
// epilogue; the tile's columns alternate 32 gate columns and the 32 up columns
// that belong to them.  KWAVES: all waves compute the whole tile, each on its
// own slice of every stage, and their sums meet in LDS (few rows: the weights
// are streamed once and the tile is narrow).  EARLY: a slice's fragments are
// read before the products of the one before it, not between them.
template <int ENC, bool XCOL, bool WCOL, bool WGRAD, bool GLU, int BM, int BN, int BK, int WM, int WN, int STAGES,
          bool KWAVES, int OCC, int FORM = kStore, int EIGHT = kNone8, bool EARLY = (BM < 256 && EIGHT == kNone8) || ENC == kFp8>
__global__ __launch_bounds__(WM* WN * 64, OCC) void product_kernel(Params p) {
  constexpr int NWAVES = WM * WN, NT = NWAVES * 64;
  constexpr bool MX = ENC == kFp4 || ENC == kFp8;
  static_assert(!MX || (!XCOL && !WCOL && !WGRAD), "microscaled operands run along the reduction");
  constexpr int XBITS = ENC == kFp4 ? 4 : (ENC == kFp8 ? 8 : 16), WBITS = MX ? 4 : 16;
  constexpr int KSLICE = MX ? 64 : 16;  // reduction length of one matrix instruction
  constexpr int NS = BK / KSLICE;       // slices of a stage
  constexpr int MY_M = KWAVES ? 1 : WM, MY_N = KWAVES ? 1 : WN;  // waves across the tile
  constexpr int WTM = BM / MY_M, WTN = BN / MY_N, FM = WTM / 32, FN = WTN / 32;
  static_assert(FM >= 1 && FN >= 1 && FM * 32 * MY_M == BM && FN * 32 * MY_N == BN && (!GLU || FN % 2 == 0 || (FORM == kGated && BN == 32)), "tile");
  // columns of a block that are gates, and the ups behind them: blocks of either, or half and half
  constexpr int GC = GLU && BN == 32 ? 16 : 32;
  static_assert(!(KWAVES && WGRAD), "the narrow tile has the same steps everywhere");
  static_assert(FORM == kStore || (!MX && !WGRAD && GLU == (FORM == kGated)), "gated forms");
  static_assert(KWAVES ? NS == NWAVES : NS == 2 || NS == 4, "one slice of a stage for each wave, or two or four");
  // chunks of a stage row: BK values along the reduction, or BM / BN across it
  constexpr int XC = XCOL ? BM / 8 : BK * XBITS / 128, WC = WCOL ? BN / 8 : BK * WBITS / 128;
  constexpr int X_BYTES = BM * BK * XBITS / 8, W_BYTES = BN * BK * WBITS / 8;
  constexpr int XI = X_BYTES / 16 / NT, WI = W_BYTES / 16 / NT;  // copies of a thread for one stage
  // An operand in FP8 (EIGHT): its codes are copied as they are, with their
  // rows' scales, and each thread turns what it copied itself into 16-bit
  // values for the stage that is multiplied next; two such stages are enough.
  constexpr bool X8 = EIGHT == kX8, W8 = EIGHT == kW8;
  static_assert(EIGHT == kNone8 || (WGRAD && STAGES % 2 == 0 && NS == 2), "FP8 rows are the weight gradient's");
  constexpr int EB = X8 ? BM : BN, EC = EB / 16;               // its columns; 16-code chunks of a row
  constexpr int E_BYTES = EB * BK, EI = E_BYTES / 16 / NT;      // codes of a stage, copies of a thread
  constexpr int ER = 64 / EC, EROWS = EI * ER;                  // rows of a wave's copy, of all of them
  constexpr int ED = EB / 128 + 1 <= 2 ? 2 : 4;                 // dwords that hold a row's scales, wherever they begin
  static_assert(EIGHT == kNone8 || (EI >= 1 && EI * 16 * NT == E_BYTES && EROWS * ED <= 64), "whole copies");
  static_assert(XI >= 1 && WI >= 1 && XI * 16 * NT == X_BYTES && WI * 16 * NT == W_BYTES, "whole copies");
  static_assert((XCOL || NT / XC % 16 == 0) && (WCOL || NT / WC % 16 == 0), "one swizzle for all copies of a lane");
  constexpr int STEP_COPIES = (X8 ? EI + 1 : XI) + (W8 ? EI + 1 : WI);
  static_assert((STAGES - 2) * STEP_COPIES < 64, "vmcnt range");
  // E8M0 scales come a group at a time: with KWAVES 16 bytes a row (512
  // values), by copies; else 32 bytes (1024 values) into the registers of the
  // thread that looks after the row, which hands each step's on through LDS.
  // (A row's bytes are a line of their own: the more of it a fetch takes, the
  // less of the L2's path the scales need.  16 bytes a time cost a step of the
  // 256-row FP4 tile 1000 of 5100 cycles.)
  constexpr int SPG = MX ? (KWAVES ? 512 : 1024) / BK : 1;  // k-steps of one group of scales
  constexpr int XW = (BM + 63) / 64, SROWS = MX ? XW * 64 + BN : 1;  // rows whose scales are staged
  static_assert(!MX || (KWAVES ? SROWS <= NT : SROWS == NT), "a thread for each row's scales");
  constexpr int SB = BK / 128;  // words of a row's scales in one step
  static_assert(!MX || KWAVES || SB == 1 || SB == 2, "words of a step");

  __shared__ __attribute__((aligned(16))) uint8_t sX[(X8 ? 2 : STAGES) * X_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sW[(W8 ? 2 : STAGES) * W_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t s_codes[EIGHT ? STAGES * E_BYTES : 1];
  __shared__ __attribute__((aligned(16))) uint32_t s_row_sc[EIGHT ? STAGES * NWAVES * 64 : 1];  // a wave's rows' scales
  // KWAVES: groups of scales as they lie in memory, from the dword that holds a
  // row's first one: up to STAGES - 1 in flight (a tile may end within a
  // group) and the one in use.  s_sc2: the dword after the 16 bytes, for rows
  // that begin in the middle of a dword.
  __shared__ __attribute__((aligned(16))) v4u s_sc[MX && KWAVES ? STAGES * SROWS : 1];
  __shared__ __attribute__((aligned(16))) uint32_t s_sc2[MX && KWAVES ? STAGES * SROWS : 1];
  // else: the scales of two steps, SB words a row
  __shared__ __attribute__((aligned(16))) uint32_t s_step[MX && !KWAVES ? 2 * SROWS * SB : 1];
  // KWAVES: the sums of one wave
  __shared__ __attribute__((aligned(16))) v4f s_sum[KWAVES ? FM * FN * 4 * 64 : 1];
  static_assert(NT > 256 || BM > 128 ||
                    sizeof(sX) + sizeof(sW) + sizeof(s_codes) + sizeof(s_row_sc) + sizeof(s_sc) + sizeof(s_sc2) + sizeof(s_step) +
                            sizeof(s_sum) +
                            (2 * kMaxExperts + 1) * 4 <= 80 * 1024,
                "two workgroups a CU");
  extern __shared__ __attribute__((aligned(16))) int32_t s_dyn[];
  int32_t* s_ends = s_dyn;
  int32_t* s_pre = s_dyn + p.e;

  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = KWAVES ? 0 : wave / WN, wn = KWAVES ? 0 : wave % WN;
  group_table(p, WGRAD ? 1 : BM, s_ends, s_pre);
  const int parts = EIGHT != kNone8 ? p.splits : 1;
  const int total = WGRAD ? p.e * parts * p.tiles_m * p.tiles_n : s_pre[p.e];
  if constexpr (EIGHT != kNone8) length_order(p, s_ends, s_pre);  // the tiles' numbers need no table here
  const int64_t F = GLU ? p.n / 2 : p.n;  // columns of y
  const int64_t x_row = WGRAD ? p.k * (X8 ? 1 : 2) : p.k * XBITS / 8;  // bytes
  const int64_t w_row = WCOL ? p.n * (W8 ? 1 : 2) : p.k * WBITS / 8;
  const int64_t s_row = (W8 ? p.n : p.k) / 32;
  const bool s_split = MX && (s_row & 3) != 0;  // k % 128 == 64: odd rows' scales begin mid-dword

  // ---- tiles: blocks of neighbouring raster tiles are dealt to the XCDs
  // (workgroup b runs on XCD b % 8), as many a block as its 32 CUs run at once
  // (with 64 of the 256-row tiles an XCD may have two rounds left where others
  // have none: FP8 ragged 638 -> 609 us, weight gradients 2-10%) and fewer
  // when there are few tiles, so that every XCD gets some
  const int G = p.grid;
  const int block = max(1, min(BM >= 256 ? 32 : 64, (total + kXcds - 1) / kXcds));
  auto tile_at = [&](int j) -> int {
    int64_t t;
    if (G % kXcds == 0) {
      const int i = j * (G / kXcds) + (int)blockIdx.x / kXcds;
      t = ((int64_t)(i / block) * kXcds + blockIdx.x % kXcds) * block + i % block;
    } else {
      t = (int64_t)j * G + blockIdx.x;
    }
    return t < total ? (int)t : -1;
  };
  auto coord = [&](int t) -> Tile {
    Tile c;
    int local, mtiles;
    if constexpr (WGRAD) {
      const int n = t / (p.tiles_m * p.tiles_n);
      int at = n;
      c.part = 0;
      if constexpr (EIGHT != kNone8) {
        if (parts > 1) {
          at = n / parts;
          c.part = n - at * parts;
        }
      }
      c.g = EIGHT != kNone8 ? __builtin_amdgcn_readfirstlane(s_pre[at]) : at;
      local = t - n * p.tiles_m * p.tiles_n;
      mtiles = p.tiles_m;
    } else {
      int lo = 0, hi = p.e - 1;  // the largest g with s_pre[g] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pre[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      c.g = __builtin_amdgcn_readfirstlane(lo);
      local = __builtin_amdgcn_readfirstlane(t - s_pre[c.g]);
      mtiles = 0;
    }
    const int begin = __builtin_amdgcn_readfirstlane(c.g ? s_ends[c.g - 1] : 0);
    const int end = __builtin_amdgcn_readfirstlane(s_ends[c.g]);
    if constexpr (!WGRAD) mtiles = (int)(((int64_t)end - begin + BM - 1) / BM);
    // inside an expert: groups of GM tiles along M, N swept inside a group
    constexpr int GM = BM >= 256 ? 4 : 8;
    const int grp = local / (GM * p.tiles_n), in = local - grp * GM * p.tiles_n;
    const int size = min(GM, mtiles - grp * GM);
    const int mt = grp * GM + in % size, nt = in / size;
    c.m0 = (WGRAD ? 0 : begin) + mt * BM;
    c.valid = min(BM, (WGRAD ? (int)p.k : end) - c.m0);
    c.n0 = nt * (GLU ? BN / 2 : BN);
    c.r0 = WGRAD ? begin : 0;
    c.r1 = WGRAD ? end : (int)p.k;
    if constexpr (EIGHT != kNone8) {
      if (parts > 1) {  // parts of whole steps
        const int64_t len = ((uint32_t)(end - begin) / parts + BK) / BK * BK;
        c.r0 = (int)min(begin + c.part * len, (int64_t)end);
        c.r1 = (int)min(c.r0 + len, (int64_t)end);
      }
    }
    c.alone = mtiles == 1;
    return c;
  };
  auto steps_of = [&](const Tile& c) -> int {
    const int s = (int)(((int64_t)c.r1 - c.r0 + BK - 1) / BK);
    return KWAVES ? s : max(s, STAGES);  // the pipeline below wants that many, of zeros if need be
  };

  // column of the weights for column q of the tile; -1 past the last
  auto column = [&](const Tile& c, int q) -> int {
    if constexpr (GLU) {
      const int f = c.n0 + q / (2 * GC) * GC + q % GC;
      return f < F ? f + ((q & GC) ? (int)F : 0) : -1;
    } else {
      return c.n0 + q < p.n ? c.n0 + q : -1;
    }
  };

  // ---- the copy stream's state: where the next step of its tile comes from.
  // Sizes from there to the operand's end fit 32 bits: rows along the
  // reduction are cut to the tile's, rows across it to one stage.
  const uint8_t* x_at = nullptr;
  const uint8_t* w_at = nullptr;
  const uint8_t* xs_at = nullptr;  // the tile's row and column scales, from a whole dword on
  const uint8_t* ws_at = nullptr;
  uint32_t x_size = 0, w_size = 0, xs_size = 0, ws_size = 0;
  int r_left = 0;                  // of the reduction, from the step on
  bool w_once = false;             // KWAVES: no other tile reads these weights
  uint32_t x_skip = 0, w_skip = 0; // rows across the reduction: bytes of a row before the tile
  uint32_t x_off[XI], w_off[WI], s_off[2] = {kOutside, kOutside}, s_odd[2] = {0, 0};
  // EIGHT: offsets of the codes; the lane's row, dword of its scales and where
  // they begin in the first of them, for the rows that the lane converts
  const uint8_t* es_at = nullptr;
  uint32_t es_skip = 0, e_off[EI > 0 ? EI : 1], es_off = kOutside, e_odd = 0, e_odd_next = 0;  // a bit per copy: 2 bytes in
  const int es_row = EIGHT ? (lane / ED / ER) * (NT / EC) + wave * ER + lane / ED % ER : 0;
  const int x_ch = XCOL ? 0 : ((lane % XC) ^ swz_row<XC>(tid / XC)) * 16;
  const int w_ch = WCOL ? 0 : ((lane % WC) ^ swz_row<WC>(tid / WC)) * 16;
  auto cut = [](int64_t bytes) -> uint32_t { return (uint32_t)(bytes > (int64_t)kOutside ? (int64_t)kOutside : bytes); };
  auto set_eight = [&](const Tile& c, int tid) {
    if constexpr (EIGHT != kNone8) {
      const int64_t row = X8 ? x_row : w_row;
      const int first = X8 ? c.m0 : c.n0, left = X8 ? c.valid : (int)min((int64_t)BN, p.n - c.n0);
      const uint8_t* at = (const uint8_t*)(X8 ? p.xs : p.ws) + (int64_t)c.r0 * s_row + first / 32;
      const uint32_t in = (uintptr_t)at & 3;
      es_at = at - in;
      es_skip = first / 32 - in;  // (wraps: sizes below are taken modulo 2^32)
      es_off = lane < EROWS * ED ? ((in + (uint32_t)es_row * (uint32_t)s_row) & ~3u) + lane % ED * 4 : kOutside;
      e_odd_next = 0;
#pragma unroll
      for (int q = 0; q < EI; ++q) {
        const int slot = q * NT + tid, r = slot / EC, col = slot % EC * 16;
        e_off[q] = col < left ? (uint32_t)(r * (int)row + col) : kOutside;
        e_odd_next |= ((in + (uint32_t)r * (uint32_t)s_row) & 2) << (2 * q);
      }
    }
  };
  auto set_sources = [&](const Tile& c) {
    // indices pass through an opaque point: the offsets are computed here,
    // once a tile, and not kept in parts across the k-loop
    int lane = threadIdx.x & 63, tid = threadIdx.x;
    asm volatile("" : "+v"(lane), "+v"(tid));
    r_left = c.r1 - c.r0;
    w_once = c.alone;
    set_eight(c, tid);
    if constexpr (XCOL) {  // wgrad: from (first row of the group, first column of the tile)
      x_skip = c.m0 * (X8 ? 1 : 2);
      x_at = (const uint8_t*)p.x + (int64_t)c.r0 * x_row + x_skip;
#pragma unroll
      for (int q = 0; q < (X8 ? 0 : XI); ++q) {
        const int slot = q * NT + tid, r = slot / XC;
        const int col = ((slot % XC) ^ swz_col<XC>(r)) * 8;
        x_off[q] = col < c.valid ? (uint32_t)(r * (int)x_row + col * 2) : kOutside;
      }
    } else {
      x_at = (const uint8_t*)p.x + c.m0 * x_row;
      x_size = c.valid * (uint32_t)x_row;
#pragma unroll
      for (int q = 0; q < XI; ++q) x_off[q] = (uint32_t)((q * (NT / XC) + tid / XC) * (int)x_row + x_ch);
    }
    if constexpr (WCOL) {  // from the tile's first column, of the expert's first row (or the group's)
      w_skip = c.n0 * (W8 ? 1 : 2);
      w_at = (const uint8_t*)p.w + (WGRAD ? (int64_t)c.r0 : c.g * p.k) * w_row + w_skip;
#pragma unroll
      for (int q = 0; q < (W8 ? 0 : WI); ++q) {
        const int slot = q * NT + tid, r = slot / WC;
        const int col = column(c, ((slot % WC) ^ swz_col<WC>(r)) * 8);
        w_off[q] = col >= 0 ? (uint32_t)(r * (int)w_row + (col - c.n0) * 2) : kOutside;
      }
    } else {
      w_at = (const uint8_t*)p.w + ((int64_t)c.g * p.n + c.n0) * w_row;
      w_size = cut((p.n - c.n0) * w_row);
#pragma unroll
      for (int q = 0; q < WI; ++q) {
        const int col = column(c, q * (NT / WC) + tid / WC);
        w_off[q] = col >= 0 ? (uint32_t)(col - c.n0) * (uint32_t)w_row + w_ch : kOutside;
      }
    }
  };
  auto set_scale_sources = [&](const Tile& c) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    if constexpr (MX) {
      const uint8_t* xb = p.xs + c.m0 * s_row;
      const uint8_t* wb = p.ws + ((int64_t)c.g * p.n + c.n0) * s_row;
      const uint32_t xf = (uintptr_t)xb & 3, wf = (uintptr_t)wb & 3;
      xs_at = xb - xf;
      ws_at = wb - wf;
      // up to the end of the dword that holds the last scale (a dword that the
      // descriptor cuts would read as zero)
      xs_size = cut((p.xs + p.m * s_row - xs_at + 3) & ~(int64_t)3);
      ws_size = cut((p.ws + (int64_t)p.e * p.n * s_row - ws_at + 3) & ~(int64_t)3);
      // of the staged rows: x first, then columns
#pragma unroll
      for (int u = 0; u < (KWAVES ? 1 : 2); ++u) {
        const int i = KWAVES ? tid : (tid & ~63) + u * 32 + ((tid & 63) >> 1);
        const int row = i < XW * 64 ? (i < c.valid ? i : -1) : (i < SROWS ? column(c, i - XW * 64) : -1);
        const uint32_t at = (uint32_t)(i < XW * 64 ? row : row - c.n0) * (uint32_t)s_row + (i < XW * 64 ? xf : wf);
        s_off[u] = row >= 0 ? at & ~3u : kOutside;
        s_odd[u] = (at & 3) * 8;  // bits
      }
    }
  };
  // Copies of the stream's next step (step kt of its tile) into stage `st`:
  // first its scales (into `slot`, when the step begins a group of them), then
  // one copy after the other.  A copy keeps the CU's address path busy for 16
  // to 21 cycles; all at once they block every wave in turn, so they are
  // issued between the products.
  // Without KWAVES two lanes take a row's 32 bytes, 16 each (a fetch of 64
  // separate lines would hold the address path four times as long): lane l of
  // copy u the half l & 1 of staged row 64 wave + 32 u + l / 2.
  v4u sc_half[2];
  uint32_t sc_next[2] = {0, 0}, sc_odd[2] = {0, 0};  // the dword after the second half; bits to shift by
  auto issue_scales = [&](int kt, int slot) {
    if constexpr (MX && KWAVES) {
      if (kt % SPG == 0 && wave * 64 < SROWS) {
        const v4i r = wave < XW ? buffer(xs_at, xs_size) : buffer(ws_at, ws_size);
        const uint32_t at = kt / SPG * 16;
        copy16(r, s_off[0] + at, __builtin_amdgcn_readfirstlane(lds_addr(s_sc)) + (slot * SROWS + wave * 64) * 16);
        if (s_split)
          copy4(r, s_off[0] + at + 16, __builtin_amdgcn_readfirstlane(lds_addr(s_sc2)) + (slot * SROWS + wave * 64) * 4);
      }
    } else if constexpr (MX) {
      if (kt % SPG == 0) {
        const v4i r = wave < XW ? buffer(xs_at, xs_size) : buffer(ws_at, ws_size);
        const __amdgpu_buffer_rsrc_t b = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(((uint64_t)(uint32_t)r.y << 32) | (uint32_t)r.x), 0, r.z, 0x00020000);
        const int at = kt / SPG * 32 + (lane & 1) * 16;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          sc_half[u] = __builtin_amdgcn_raw_buffer_load_b128(b, (int)s_off[u] + at, 0, 0);
          if (s_split) sc_next[u] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)s_off[u] + at + 16, 0, 0);
          sc_odd[u] = s_odd[u];
        }
      }
    }
  };
  // The coming step's scales, from the lanes that hold them; blocks past k
  // become zero bytes (2^-127, where the next row's may be a NaN).
  auto hand_on = [&](int kt, int slot) {
    if constexpr (MX && !KWAVES) {
      constexpr int PER = SPG / 2;  // steps of a half
      const int pos = kt % SPG, w = pos % PER * SB;
      const bool mine = (lane & 1) == pos / PER;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const v4u v = sc_half[u];
        uint32_t d[SB];
        if constexpr (SB == 2) {
          d[0] = w ? v.z : v.x;
          d[1] = w ? v.w : v.y;
        } else {
          d[0] = w & 2 ? (w & 1 ? v.w : v.z) : (w & 1 ? v.y : v.x);
        }
        if (s_split) {
          uint32_t next = w + SB == 4 ? sc_next[u] : (SB == 2 ? v.z : (w == 0 ? v.y : w == 1 ? v.z : v.w));
          if constexpr (SB == 2) {
            d[0] = __builtin_amdgcn_alignbit(d[1], d[0], sc_odd[u]);
            d[1] = __builtin_amdgcn_alignbit(next, d[1], sc_odd[u]);
          } else {
            d[0] = __builtin_amdgcn_alignbit(next, d[0], sc_odd[u]);
          }
        }
#pragma unroll
        for (int q = 0; q < SB; ++q) {
          const int bytes = ((int)p.k - kt * BK) / 32 - 4 * q;
          if (bytes < 4) d[q] &= bytes <= 0 ? 0u : (1u << (8 * bytes)) - 1;
        }
        uint32_t* to = &s_step[(slot * SROWS + wave * 64 + u * 32 + (lane >> 1)) * SB];
        if (mine) {
          if constexpr (SB == 2) *(uint64_t*)to = (uint64_t)d[1] << 32 | d[0];
          else *to = d[0];
        }
      }
    }
  };
  auto across = [&](uint32_t row, uint32_t skip) -> uint32_t {  // size of one stage's rows
    return r_left > 0 ? min(r_left, BK) * row - skip : 0u;
  };
  auto issue_whole = [&](int st, auto q_) {
    constexpr int Q = decltype(q_)::value;
    // in the last step of a reduction that is no multiple of BK, chunks past
    // the row's end would be the next row's
    if constexpr (Q < XI) {
      const v4i xr = buffer(x_at, XCOL ? across((uint32_t)x_row, x_skip) : x_size);
      copy16(xr, XCOL || x_ch * 8 / XBITS < r_left ? x_off[Q] : kOutside,
             __builtin_amdgcn_readfirstlane(lds_addr(sX)) + st * X_BYTES + (Q * NWAVES + wave) * 1024);
    } else {
      const v4i wr = buffer(w_at, WCOL ? across((uint32_t)w_row, w_skip) : w_size);
      const uint32_t off = WCOL || w_ch * 8 / WBITS < r_left ? w_off[Q - XI] : kOutside;
      const uint32_t to = __builtin_amdgcn_readfirstlane(lds_addr(sW)) + st * W_BYTES + ((Q - XI) * NWAVES + wave) * 1024;
      // (one token through bf16 experts 50.5 -> 47.7 us; microscaled ones
      // alike.  Where a group has several tiles the others find the weights in
      // the L2: 48 rows an expert 350 -> 274 us)
      if (KWAVES && !MX && w_once) copy16_once(wr, off, to);
      else copy16(wr, off, to);
    }
  };
  auto issue_copy = [&](int st, auto q_) {
    constexpr int Q0 = decltype(q_)::value;
    if constexpr (EIGHT && Q0 < EI) {
      // an operand in FP8 goes first, as it is needed first, and its scales
      const v4i r = buffer(X8 ? x_at : w_at, X8 ? across((uint32_t)x_row, x_skip) : across((uint32_t)w_row, w_skip));
      copy16(r, e_off[Q0], __builtin_amdgcn_readfirstlane(lds_addr(s_codes)) + st * E_BYTES + (Q0 * NWAVES + wave) * 1024);
    } else if constexpr (EIGHT && Q0 == EI) {
      // up to the end of the dword that holds the last row's last; rows past it
      // get zeros, whatever theirs would be: 2^-127 times codes of zero
      const v4i r = buffer(es_at, r_left > 0 ? (min(r_left, BK) * (uint32_t)s_row - es_skip + 3) & ~3u : 0u);
      copy4(r, es_row < r_left ? es_off : kOutside,
            __builtin_amdgcn_readfirstlane(lds_addr(s_row_sc)) + (st * NWAVES + wave) * 256);
    } else {
      issue_whole(st, std::integral_constant<int, X8 ? Q0 - EI - 1 + XI : W8 ? Q0 - EI - 1 : Q0>{});
    }
  };
  auto advance = [&]() {
    x_at += XCOL ? BK * x_row : BK * XBITS / 8;
    w_at += WCOL ? BK * w_row : BK * WBITS / 8;
    if constexpr (EIGHT) es_at += BK * s_row;
    // (never below nothing: past the last tile zeros are still copied)
    if constexpr (!XCOL) x_size = x_size > BK * XBITS / 8 ? x_size - BK * XBITS / 8 : 0;
    if constexpr (!WCOL) w_size = w_size > BK * WBITS / 8 ? w_size - BK * WBITS / 8 : 0;
    r_left = max(r_left - BK, 0);
  };
  auto no_sources = [&]() {
    x_size = w_size = 0;
    r_left = 0;
  };
  auto no_scale_sources = [&]() { xs_size = ws_size = 0; };

  // ---- fragments.  A fragment holds 32 rows (x) or columns (w) of one slice:
  // lane l row l % 32, and its h = l / 32 half of the slice.  The addresses of
  // a lane, but for the stage, the fragment and the slice, are fixed.
  using XFrag = std::conditional_t<ENC == kFp8, v8i, std::conditional_t<MX, v4i, v8s>>;
  using WFrag = std::conditional_t<MX, v4i, v8s>;
  auto wide = [](auto v) -> v8i {  // as the instruction's type takes it (FP4: the upper half is not read)
    if constexpr (sizeof(v) == 32) return v;
    else return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
  };
  // rows along the reduction: pair u of chunks (chunk 2 u + h) of a row
  constexpr int XU = XCOL ? FM : XC / 2, WU = WCOL ? FN : WC / 2;
  uint32_t x_adr[XU], w_adr[WU];
  auto row_adr = [&](int row, int u, auto c_) -> uint32_t {
    constexpr int C = decltype(c_)::value;
    return row * (C * 16) + (((2 * u + h) ^ swz_row<C>(row)) << 4);
  };
  // rows across it, by transposing reads: within 16 lanes, lane i receives
  // element i % 16 of the four rows addressed by lanes 4 b .. 4 b + 3
  // (b = 0..3, 4 elements each)
  auto col_adr = [&](int first, auto c_) -> uint32_t {
    constexpr int C = decltype(c_)::value;
    const int i = lane & 15, grp = lane >> 4;
    const int r = (grp >> 1) * 8 + (i >> 2), col = first + (grp & 1) * 16 + (i & 3) * 4;
    return r * (C * 16) + ((((col >> 3) ^ swz_col<C>(r)) << 4) | ((col & 7) << 1));
  };
#pragma unroll
  for (int u = 0; u < XU; ++u)
    x_adr[u] = lds_addr(sX) + (XCOL ? col_adr(wm * WTM + u * 32, std::integral_constant<int, XCOL ? XC : 16>{})
                                    : row_adr(wm * WTM + (lane & 31), u, std::integral_constant<int, XCOL ? 8 : XC>{}));
#pragma unroll
  for (int u = 0; u < WU; ++u)
    w_adr[u] = lds_addr(sW) + (WCOL ? col_adr(wn * WTN + u * 32, std::integral_constant<int, WCOL ? WC : 16>{})
                                    : row_adr(wn * WTN + (lane & 31), u, std::integral_constant<int, WCOL ? 8 : WC>{}));
  auto lds4 = [](uint32_t a) -> v4i { return *(const LDS_PTR(v4i))a; };
  auto frag_row = [&](uint32_t a0, uint32_t a1, auto* f) {
    const v4i lo = lds4(a0);
    if constexpr (sizeof(*f) == 32) {
      const v4i hi = lds4(a1);
      *f = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    } else {
      *f = __builtin_bit_cast(std::remove_reference_t<decltype(*f)>, lo);
    }
  };
  auto frag_col = [&](uint32_t a, int row_bytes) -> v8s {
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(v4s))a);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(v4s))(a + 4 * row_bytes));
    return v8s{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  };
  // s: the slice (a constant once unrolled; the wave's own with KWAVES)
  auto read_x = [&](int st, int s, int i, XFrag& f) {
    constexpr int XP = XBITS == 8 ? 2 : 1;  // chunk pairs of a slice
    const uint32_t xs = (X8 ? st & 1 : st) * X_BYTES;
    if constexpr (XCOL) {
      f = frag_col(x_adr[i] + xs + s * (16 * XC * 16), XC * 16);
    } else if constexpr (KWAVES) {
      const int row = i * 32 + (lane & 31);
      constexpr auto c = std::integral_constant<int, XCOL ? 8 : XC>{};
      const uint32_t at = lds_addr(sX) + xs;
      frag_row(at + row_adr(row, s * XP, c), at + row_adr(row, s * XP + XP - 1, c), &f);
    } else {
      const uint32_t at = xs + i * (32 * XC * 16);
      frag_row(x_adr[s * XP] + at, x_adr[s * XP + XP - 1] + at, &f);
    }
  };
  auto read_w = [&](int st, int s, int j, WFrag& f) {
    const uint32_t ws = (W8 ? st & 1 : st) * W_BYTES;
    if constexpr (WCOL) {
      f = frag_col(w_adr[j] + ws + s * (16 * WC * 16), WC * 16);
    } else if constexpr (KWAVES) {
      frag_row(lds_addr(sW) + ws + row_adr(j * 32 + (lane & 31), s, std::integral_constant<int, WCOL ? 8 : WC>{}), 0, &f);
    } else {
      frag_row(w_adr[s] + ws + j * (32 * WC * 16), 0, &f);
    }
  };
  auto read_frags = [&](int st, int s, XFrag (&xf)[FM], WFrag (&wf)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) read_x(st, s, i, xf[i]);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_w(st, s, j, wf[j]);
  };
  // Those of them that are read after product m of the slice before, in the
  // order in which the products want them: in the first half of the slice, one
  // or two after a product.  All at once they hold the LDS, and with it every
  // wave's issue, before the first product.
  auto read_after = [&](int st, int s, XFrag (&xf)[FM], WFrag (&wf)[FN], auto m_) {
    constexpr int M = decltype(m_)::value, ALL = FM + FN, HALF = FM * FN / 2;
    constexpr int A = ALL * M / HALF < ALL ? ALL * M / HALF : ALL, B = ALL * (M + 1) / HALF < ALL ? ALL * (M + 1) / HALF : ALL;
    if constexpr (B > A) {
      __builtin_amdgcn_sched_barrier(0);
      static_for<B - A>([&](auto q_) {
        constexpr int Q = A + decltype(q_)::value;  // w0 x0 w1 .. x1 ..
        if constexpr (Q == 0) read_w(st, s, 0, wf[0]);
        else if constexpr (Q == 1) read_x(st, s, 0, xf[0]);
        else if constexpr (Q <= FN) read_w(st, s, Q - 1, wf[Q - 1]);
        else read_x(st, s, Q - FN, xf[Q - FN]);
      });
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // EIGHT: the codes of stage `st` that this thread copied, and their scales,
  // once those copies have landed (the caller waits) ...
  v4u e_raw[EI > 0 ? EI : 1];
  uint32_t e_scale[EI > 0 ? EI : 1];
  auto fetch_codes = [&](int st) {
    if constexpr (EIGHT != kNone8) {
      const int chunk = lane % EC;
#pragma unroll
      for (int q = 0; q < EI; ++q) {
        e_raw[q] = *(const v4u*)(s_codes + st * E_BYTES + (q * NT + tid) * 16);
        const uint8_t* sc = (const uint8_t*)(s_row_sc + (st * NWAVES + wave) * 64 + (q * ER + lane / EC) * ED);
        e_scale[q] = sc[chunk / 2 + ((e_odd >> (2 * q)) & 2)];
      }
    }
  };
  // ... and half H of copy Q of them, eight values, into the stage's own place.
  auto widen = [&](int st, auto part_) {
    if constexpr (EIGHT != kNone8) {
      constexpr int Q = decltype(part_)::value / 2, H = decltype(part_)::value % 2, C = X8 ? XC : WC;
      const float scale = __uint_as_float(e_scale[Q] << 23);  // the conversions take the exponent, 0 as 2^-127 and 255 as NaN
      v4u o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t four = e_raw[Q][2 * H + i / 2];
        if constexpr (ENC == kBf16) {
          o[i] = i % 2 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, scale, true))
                       : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, scale, false));
        } else {
          o[i] = i % 2 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, scale, true))
                       : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, scale, false));
        }
      }
      const int slot = Q * NT + tid, r = slot / EC, chunk = 2 * (slot % EC) + H;
      *(v4u*)((X8 ? sX + (st & 1) * X_BYTES : sW + (st & 1) * W_BYTES) + r * (C * 16) + ((chunk ^ swz_col<C>(r)) << 4)) = o;
    }
  };
  constexpr int WIDEN = EIGHT ? 2 * EI : 0;  // pieces of a step

  // This step's scales, one register a fragment.  Slice q of a step takes its
  // blocks 2 q (lanes with h = 0) and 2 q + 1: of a step's bytes each lane
  // keeps every second one.  With four slices byte s is slice s's, with two it
  // is byte 2 s.
  uint32_t xsc[FM], wsc[FN];
  auto read_scales = [&](const Tile& c, int kt, int slot) {
    if constexpr (MX && KWAVES) {
      const bool in = kt * BK + wave * 64 < (int)p.k;  // this wave's slice exists
      auto one = [&](int row, uint32_t odd) -> uint32_t {
        const int at = 2 * ((kt % SPG) * NS + wave) + h + (int)odd;
        const uint8_t* b = at < 16 ? (const uint8_t*)&s_sc[slot * SROWS + row] + at
                                   : (const uint8_t*)&s_sc2[slot * SROWS + row] + (at - 16);
        const uint32_t v = *b;
        return in ? v : 0u;
      };
#pragma unroll
      for (int i = 0; i < FM; ++i) xsc[i] = one(i * 32 + (lane & 31), s_split ? ((c.m0 + lane) & 1) * 2 : 0);
#pragma unroll
      for (int j = 0; j < FN; ++j) wsc[j] = one(XW * 64 + j * 32 + (lane & 31), s_split ? (lane & 1) * 2 : 0);
    }
  };
  // Without KWAVES in two halves, with products between: the words of the
  // coming step, and what the lane keeps of them.
  using Words = std::conditional_t<SB == 2, uint64_t, uint32_t>;
  Words x_words[FM], w_words[FN];
  auto fetch_scales = [&](int slot) {
    if constexpr (MX && !KWAVES) {
      const Words* base = (const Words*)s_step + slot * SROWS;
#pragma unroll
      for (int i = 0; i < FM; ++i) x_words[i] = base[wm * WTM + i * 32 + (lane & 31)];
#pragma unroll
      for (int j = 0; j < FN; ++j) w_words[j] = base[XW * 64 + wn * WTN + j * 32 + (lane & 31)];
    }
  };
  auto keep_scales = [&]() {
    if constexpr (MX && !KWAVES) {
      auto one = [&](Words v) -> uint32_t {
        if constexpr (SB == 2)
          return __builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, h ? 0x07050301u : 0x06040200u);
        else
          return v >> (8 * h);
      };
#pragma unroll
      for (int i = 0; i < FM; ++i) xsc[i] = one(x_words[i]);
#pragma unroll
      for (int j = 0; j < FN; ++j) wsc[j] = one(w_words[j]);
    }
  };

  // 256 accumulators a lane (one wave a SIMD) live in the accumulation
  // registers, and are read from there one by one when they are stored
  constexpr bool IN_AGPRS = FM * FN == 16;
  v16f acc[FM][FN];
  auto sum_at = [&](int i, int j, int r) -> float {
    if constexpr (IN_AGPRS) {
      float o;
      asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(o) : "a"(acc[i][j][r]));
      return o;
    } else {
      return acc[i][j][r];
    }
  };
  // An fp32 sum but for FP8 with FP4: there the instruction drops what lies 2^-14
  // below a 32-value block's largest product (no other takes these types; before
  // their rounding such outputs are 1.5e-5 of their norm off, FP4 with FP4 5e-8).
  // between(m): what is issued after product m of the slice
  auto multiply = [&](XFrag (&xf)[FM], WFrag (&wf)[FN], auto s_, auto between) {
    constexpr int S = KWAVES ? 0 : decltype(s_)::value * (NS == 4 ? 1 : 2);  // byte of the scale registers
    static_for<FM * FN>([&](auto m_) {
      constexpr int i = decltype(m_)::value / FN, j = decltype(m_)::value % FN;
      if constexpr (ENC == kBf16)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, wf[j]),
                                                            __builtin_bit_cast(v8bf, xf[i]), acc[i][j], 0, 0, 0);
      else if constexpr (ENC == kF16)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, wf[j]),
                                                           __builtin_bit_cast(v8h, xf[i]), acc[i][j], 0, 0, 0);
      else
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(wf[j]), wide(xf[i]), acc[i][j], 4, ENC == kFp4 ? 4 : 0, S & 3,
                                                                    (int)wsc[j], S & 3, (int)xsc[i]);
      between(m_);
    });
    // The sums are needed here as far as the compiler can tell: it would move
    // the products of a whole step behind the next branch, past the barrier,
    // with the fragments of all its slices held until then.
    static_for<FM * FN>([&](auto m_) {
      v16f& a = acc[decltype(m_)::value / FN][decltype(m_)::value % FN];
      if constexpr (IN_AGPRS) asm volatile("" : "+a"(a));
      else asm volatile("" : "+v"(a));
    });
  };
  auto nothing = [](auto) {};

  // ---- epilogue: lane l holds row l % 32 of each 32 x 32 block and columns
  // 8 (r / 4) + 4 h + r % 4, r = 0..15
  auto store_block = [&](const Tile& c, int lane, int i, int col, const float (&v)[16]) {
    const int h = lane >> 5, row = wm * WTM + i * 32 + (lane & 31);
    if (row >= c.valid) return;
    const int64_t g = EIGHT != kNone8 ? (int64_t)c.part * p.e + c.g : (int64_t)c.g;
    const int64_t at = (WGRAD ? g * p.k * p.n : 0) + (int64_t)(c.m0 + row) * F;
    if (p.out == kOutF32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = c.n0 + col + 8 * q + 4 * h;
        if (n >= F) continue;
        v4f o = v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        v4f* d = (v4f*)((float*)p.y + at + n);
        if (WGRAD && p.accumulate) {
          const v4f old = *d;
          o = v4f{o.x + old.x, o.y + old.y, o.z + old.z, o.w + old.w};
        }
        *d = o;
      }
    } else {
      uint32_t d[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (p.out == kOutBf16) {
          typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
          d[q] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2 * q], (__bf16)v[2 * q + 1]});
        } else {
          typedef _Float16 v2h __attribute__((ext_vector_type(2)));
          d[q] = __builtin_bit_cast(uint32_t, v2h{(_Float16)v[2 * q], (_Float16)v[2 * q + 1]});
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        // columns 16 q .. 16 q + 15: after the swap the lower half holds the
        // first eight, the upper half the others.  Both halves hold the same
        // row, so both are here.
        const auto a = __builtin_amdgcn_permlane32_swap(d[4 * q], d[4 * q + 2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(d[4 * q + 1], d[4 * q + 3], false, false);
        const int n = c.n0 + col + 16 * q + 8 * h;
        if (n < F) *(v4u*)((uint16_t*)p.y + at + n) = v4u{a[0], b[0], a[1], b[1]};
      }
    }
  };
  auto gated_block = [&](const Tile& c, int lane, int i, int col, const float (&u)[16], const float (&v)[16]) {
    const int row = wm * WTM + i * 32 + (lane & 31);
    if (row >= c.valid || c.n0 + col >= F) return;
    const int64_t at = c.m0 + row;
    const int n = c.n0 + col, width = (int)F;
    if (p.keep == kKeepFp8) {
      uint8_t* codes = (uint8_t*)p.kept + at * 2 * F;
      uint8_t* scales = p.kept_scale + at * (F / 16);
      store_fp8(codes, scales, n, lane, u);
      store_fp8(codes + F, scales + F / 32, n, lane, v);
    } else if (p.keep == kKeepFull) {
      uint16_t* kept = (uint16_t*)p.kept + at * 2 * F;
      store_16<ENC == kF16>(kept, n, width, lane, u);
      store_16<ENC == kF16>(kept + F, n, width, lane, v);
    }
    float o[16];
    if (p.act == GMMGF_ACT_GEGLU) geglus(u, v, o);
    else swiglus(u, v, o);
    store_16<ENC == kF16>((uint16_t*)p.y + at * F, n, width, lane, o);
  };
  // One block of the way back; `k`: what was kept for it.
  constexpr bool BACK = FORM == kBackFull || FORM == kBackFp8, BACK8 = FORM == kBackFp8;
  auto load_kept = [&](const Tile& c, int lane, int i, int j, Kept<BACK8>& k) {
    const int row = wm * WTM + i * 32 + (lane & 31), n = c.n0 + wn * WTN + j * 32, width = (int)F;
    if (row >= c.valid || n >= F) return;
    const int64_t at = c.m0 + row;
    if constexpr (BACK8) {
      const uint8_t* codes = (const uint8_t*)p.kept + at * 2 * F;
      const uint8_t* scales = p.kept_scale + at * (F / 16) + n / 32;
      k.gate[0] = load_fp8(codes, n, lane);
      k.up[0] = load_fp8(codes + F, n, lane);
      k.gate_scale = scales[0];
      k.up_scale = scales[F / 32];
    } else {
      const uint16_t* kept = (const uint16_t*)p.kept + at * 2 * F;
      load_16(kept, n, width, lane, k.gate);
      load_16(kept + F, n, width, lane, k.up);
    }
  };
  auto back_block = [&](const Tile& c, int lane, int i, int j, Kept<BACK8> k, const float (&sums)[16]) {
    const int row = wm * WTM + i * 32 + (lane & 31), n = c.n0 + wn * WTN + j * 32, width = (int)F;
    if (row >= c.valid || n >= F) return;
    const int64_t at = c.m0 + row;
    uint16_t* d = (uint16_t*)p.y + at * 2 * F;
    if constexpr (BACK8) {
      spread_fp8(k.gate[0]);
      spread_fp8(k.up[0]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float dh[8], u[8], v[8], h[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) dh[r] = sums[8 * q + r];
      if constexpr (BACK8) {
        values_fp8(k.gate[0][2 * q], k.gate[0][2 * q + 1], k.gate_scale, u);
        values_fp8(k.up[0][2 * q], k.up[0][2 * q + 1], k.up_scale, v);
      } else {
        values_16<ENC == kF16>(k.gate[q], u);
        values_16<ENC == kF16>(k.up[q], v);
      }
      if (p.act == GMMGF_ACT_GEGLU) gate_back8<true>(dh, u, v, h);
      else gate_back8<false>(dh, u, v, h);
      store_piece<ENC == kF16>(d, n, width, lane, q, u);
      store_piece<ENC == kF16>(d + F, n, width, lane, q, v);
      if (p.hidden) store_piece<ENC == kF16>((uint16_t*)p.hidden + at * F, n, width, lane, q, h);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The same for a block that is half gates, half ups: a lane's first eight
  // values and its last eight, sixteen columns of h.
  auto gated_half = [&](const Tile& c, int lane, const v16f& sums) {
    const int row = lane & 31;
    if (row >= c.valid) return;
    const int64_t at = c.m0 + row;
    float u[8], v[8], o[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) u[r] = sums[r], v[r] = sums[8 + r];
    if (p.keep == kKeepFull) {
      uint16_t* kept = (uint16_t*)p.kept + at * 2 * F;
      store_piece<ENC == kF16>(kept, c.n0, (int)F, lane, 0, u);
      store_piece<ENC == kF16>(kept + F, c.n0, (int)F, lane, 0, v);
    }
    if (p.act == GMMGF_ACT_GEGLU) geglus(u, v, o);
    else swiglus(u, v, o);
    store_piece<ENC == kF16>((uint16_t*)p.y + at * F, c.n0, (int)F, lane, 0, o);
  };
  auto epilogue = [&](const Tile& c) {
    int lane = threadIdx.x & 63;  // opaque, as in set_sources
    asm volatile("" : "+v"(lane));
    // sum_at's asm reads products' results: past the 18 wait states that the
    // last of them may need
    if constexpr (IN_AGPRS) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    if constexpr (BACK) {
      // One loop over the blocks, whose sums are brought to the same registers:
      // unrolled it would be 30 KB of instructions that every wave fetches once
      // a tile.  What was kept is asked for three blocks ahead: loads and stores
      // are counted together and in order, so that a load is waited for with the
      // stores before it.
      constexpr int BLOCKS = FM * FN;
      auto ask = [&](int b) -> Kept<BACK8> {
        Kept<BACK8> k;
        if (b < BLOCKS) load_kept(c, lane, b / FN, b % FN, k);
        return k;
      };
      Kept<BACK8> k0 = ask(0), k1 = ask(1), k2 = ask(2);
#pragma unroll 1
      for (int b = 0; b < BLOCKS; ++b) {
        const Kept<BACK8> k3 = ask(b + 3);
        float sums[16];
        one_of<0, BLOCKS>(b, [&](auto b_) {
          constexpr int B = decltype(b_)::value;
#pragma unroll
          for (int r = 0; r < 16; ++r) sums[r] = sum_at(B / FN, B % FN, r);
        });
        back_block(c, lane, b / FN, b % FN, k0, sums);
        k0 = k1, k1 = k2, k2 = k3;
      }
      return;
    }
    if constexpr (GLU && BN == 32) {
      gated_half(c, lane, acc[0][0]);
      return;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (GLU) {
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
          float u[16], v[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) u[r] = sum_at(i, j, r), v[r] = sum_at(i, j + 1, r);
          if constexpr (FORM == kGated) {
            gated_block(c, lane, i, (wn * WTN + j * 32) / 2, u, v);
          } else {
            swiglus(u, v, v);
            store_block(c, lane, i, (wn * WTN + j * 32) / 2, v);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float v[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = sum_at(i, j, r);
          store_block(c, lane, i, wn * WTN + j * 32, v);
        }
      }
    }
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v16f{0};
  };

  const int t0 = tile_at(0);
  if (t0 < 0) return;
  Tile c = coord(t0);
  int steps = steps_of(c), jc = 0;
  int st = 0, slot = KWAVES ? STAGES - 1 : 0;  // computing: stage, slot of the scales in use
  set_sources(c);
  set_scale_sources(c);
  // A step of the computing stream has landed (its copies and all before
  // them): publish it.
  constexpr int YOUNGER = (STAGES - 2) * STEP_COPIES;  // copies that may be in flight then

  if constexpr (KWAVES) {
    // A stream of copies STAGES - 1 steps ahead that crosses the tiles' borders
    int jl = 0, lk = 0, lsteps = steps, sc_in = 0;  // tile count, k-step in it, slot of the next scales
    bool live = true;
    Tile ahead = c;
    auto feed = [&](int st) {
      issue_scales(lk, sc_in);
      if constexpr (MX) {
        if (lk % SPG == 0) sc_in = sc_in + 1 == STAGES ? 0 : sc_in + 1;
      }
      static_for<STEP_COPIES>([&](auto q_) { issue_copy(st, q_); });
      advance();
      if (++lk == lsteps && live) {
        lk = 0;
        const int t = tile_at(++jl);
        live = t >= 0;
        if (live) {
          ahead = coord(t);
          lsteps = steps_of(ahead);
          set_sources(ahead);
          set_scale_sources(ahead);
        } else {
          no_sources();  // what is still issued copies zeros
          no_scale_sources();
        }
      }
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) feed(s);
    while (true) {
      clear();
#pragma unroll 1
      for (int kt = 0; kt < steps; ++kt) {
        wait_vmcnt<YOUNGER>();
        if constexpr (MX) {
          if (kt % SPG == 0) slot = slot + 1 == STAGES ? 0 : slot + 1;
        }
        lds_barrier();
        feed(st == 0 ? STAGES - 1 : st - 1);
        XFrag xf[FM];
        WFrag wf[FN];
        read_scales(c, kt, slot);
        read_frags(st, wave, xf, wf);
        multiply(xf, wf, std::integral_constant<int, 0>{}, nothing);
        st = st + 1 == STAGES ? 0 : st + 1;
      }
      // The waves' sums meet in the first wave: (0 + 2) + (1 + 3).  Wave 3 gives
      // its own in the stage read last, free until the next copies: with 8 KB
      // of LDS more instead of 16 two workgroups fit a CU whatever the number
      // of experts, whose table takes up to 8 KB (1024 experts of 2048 x 1024,
      // 4 rows each: bf16 725 -> 682 us, FP4 407 -> 252; 256 of 2048 x 7168,
      // skewed, FP8: 479.6 -> 481.3).
      static_assert(!KWAVES || (NWAVES == 4 && W_BYTES >= FM * FN * 4 * 64 * 16), "two rounds, a wave's sums within a stage");
      constexpr int Q = FM * FN * 4;
      v4f* in_stage = (v4f*)(sW + (st == 0 ? STAGES - 1 : st - 1) * W_BYTES);
      auto give = [&](v4f* to) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const v16f& a = acc[q / 4 / FN][q / 4 % FN];
          to[q * 64 + lane] = v4f{a[q % 4 * 4], a[q % 4 * 4 + 1], a[q % 4 * 4 + 2], a[q % 4 * 4 + 3]};
        }
      };
      auto take = [&](const v4f* from) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const v4f o = from[q * 64 + lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[q / 4 / FN][q / 4 % FN][q % 4 * 4 + r] += o[r];
        }
      };
      lds_barrier();  // all have read that stage
      if (wave == 2) give(s_sum);
      if (wave == 3) give(in_stage);
      lds_barrier();
      if (wave == 0) take(s_sum);
      if (wave == 1) {
        take(in_stage);
        give(in_stage);
      }
      lds_barrier();
      if (wave == 0) take(in_stage);
      if (wave == 0) epilogue(c);
      const int t = tile_at(++jc);
      if (t < 0) break;
      // the copies are in the next tile already, and not past it if it has more
      // steps than they are ahead (all tiles have as many): it is not looked up
      // again (256 skewed experts, FP4: 525 -> 482 us)
      c = steps >= STAGES ? ahead : coord(t);
      steps = steps_of(c);
      // s_sum is written again only after the next tile's first barrier
    }
  } else {
    // After the barrier that publishes a step, the stage before it is refilled
    // with the step STAGES - 1 after it: in two halves, between the products
    // that follow the barrier and those of the next slice (all at once they
    // block the waves; later ones land too late: a quarter later cost 2-4%);
    // with two slices of microscaled operands, whose products take longer, all
    // between the former.  The first fragments of a step are read between the
    // last products of the one before.  Copies are issued under no condition
    // (past the last tile they copy zeros): the compiler would move the
    // products behind the branch.
    XFrag xf[2][FM];
    WFrag wf[2][FN];
    constexpr int PARTS = MX && NS == 2 ? 1 : 2, PRODUCTS = FM * FN;
    auto copies = [&](int to, auto part_, auto m_) {  // those of a part that follow product m
      constexpr int P = decltype(part_)::value, M = decltype(m_)::value;
      constexpr int FIRST = STEP_COPIES * P / PARTS, COUNT = STEP_COPIES * (P + 1) / PARTS - FIRST;
      constexpr int A = FIRST + COUNT * M / PRODUCTS, B = FIRST + COUNT * (M + 1) / PRODUCTS;
      if constexpr (B > A) {
        __builtin_amdgcn_sched_barrier(0);
        static_for<B - A>([&](auto q_) { issue_copy(to, std::integral_constant<int, A + decltype(q_)::value>{}); });
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;
    auto all_copies = [&](int to) {
      static_for<STEP_COPIES>([&](auto q_) { issue_copy(to, q_); });
      advance();
    };
    auto publish = [&](int nk) {  // step nk of a tile
      wait_vmcnt<YOUNGER>();
      slot ^= 1;
      hand_on(nk, slot);
      lds_barrier();
    };
    int t_next = 0, refill = STAGES - 1;
    Tile next = c;
    issue_scales(0, 0);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) all_copies(s);
    if constexpr (EIGHT != kNone8) {
      wait_vmcnt<YOUNGER>();
      asm volatile("" ::: "memory");
      e_odd = e_odd_next;
      fetch_codes(0);
      static_for<WIDEN>([&](auto w_) { widen(0, w_); });
    }
    publish(0);
    issue_scales(1, 0);
    static_for<STEP_COPIES / PARTS>([&](auto q_) { issue_copy(STAGES - 1, q_); });
    if constexpr (PARTS == 1) advance();
    fetch_scales(slot);
    read_frags(0, 0, xf[0], wf[0]);
    keep_scales();
    // The steps of a tile.  A wave whose rows all lie past the group's last
    // (ALIVE false) only copies: where half of a tile's rows exist the waves
    // that share its SIMDs have them alone (2% at 1024 rows an expert).
    auto run = [&](auto alive_) {
      constexpr bool ALIVE = decltype(alive_)::value;
      // the pieces of the coming step's FP8 operand that follow product m of the
      // first slice, in its second half: their codes are on their way till then
      auto widened = [&](auto part_, auto m_) {
        if constexpr (EIGHT && decltype(part_)::value == 1) {
          constexpr int M = decltype(m_)::value, H = PRODUCTS / 2;
          if constexpr (M >= H) {
            constexpr int A = WIDEN * (M - H) / H, B = WIDEN * (M - H + 1) / H;
            static_for<B - A>([&](auto w_) { widen(st + 1, std::integral_constant<int, A + decltype(w_)::value>{}); });
          }
        }
      };
      auto with_copies = [&](XFrag (&x)[FM], WFrag (&w)[FN], auto s_, auto part_, int to, auto t_) {
        constexpr int T = decltype(t_)::value;  // the slice whose fragments are read meanwhile, of stage `to`
        if constexpr (ALIVE) {
          if constexpr (EARLY) read_frags(to, T, xf[T & 1], wf[T & 1]);
          multiply(x, w, s_, [&](auto m_) {
            if constexpr (!EARLY) read_after(to, T, xf[T & 1], wf[T & 1], m_);
            copies(refill, part_, m_);
            widened(part_, m_);
          });
        } else static_for<PRODUCTS>([&](auto m_) { copies(refill, part_, m_); });
      };
#pragma unroll 1
      for (int kt = 0; kt < steps; ++kt) {
        static_for<NS - 1>([&](auto s_) {
          constexpr int S = decltype(s_)::value;
          if constexpr (EIGHT != kNone8) {
            // issued by now: this step's copies and the next two's, and half of
            // those of the one after; wanted: the next one's first EI + 1
            wait_vmcnt<STEP_COPIES * 2 + STEP_COPIES / 2 - EI - 1>();
            asm volatile("" ::: "memory");
            if (kt + 1 == steps) e_odd = e_odd_next;
            fetch_codes(st + 1 == STAGES ? 0 : st + 1);
          }
          if constexpr (S == 0 && PARTS == 2) {
            with_copies(xf[0], wf[0], s_, Second{}, st, std::integral_constant<int, S + 1>{});
            advance();
          } else if constexpr (ALIVE) {
            if constexpr (EARLY) read_frags(st, S + 1, xf[(S + 1) & 1], wf[(S + 1) & 1]);
            multiply(xf[S & 1], wf[S & 1], s_, [&](auto m_) {
              if constexpr (!EARLY) read_after(st, S + 1, xf[(S + 1) & 1], wf[(S + 1) & 1], m_);
            });
          }
        });
        publish(kt + 1 < steps ? kt + 1 : 0);
        refill = st;
        st = st + 1 == STAGES ? 0 : st + 1;
        if (kt + STAGES == steps) {  // the next copies are the next tile's
          t_next = tile_at(++jc);
          if (t_next >= 0) {
            next = coord(t_next);
            set_sources(next);
          } else {
            no_sources();  // what is still issued copies zeros
          }
        }
        if constexpr (MX) {  // scales are two steps ahead whatever the stages
          if (kt + 2 == steps) {
            if (t_next >= 0) set_scale_sources(next);
            else no_scale_sources();
          }
          issue_scales(kt + 2 < steps ? kt + 2 : kt + 2 - steps, 0);
        }
        if constexpr (ALIVE) fetch_scales(slot);
        with_copies(xf[(NS - 1) & 1], wf[(NS - 1) & 1], std::integral_constant<int, NS - 1>{}, First{}, st, First{});
        if constexpr (PARTS == 1) advance();
        if constexpr (ALIVE) keep_scales();
      }
      if constexpr (!ALIVE) {  // for the next tile
        fetch_scales(slot);
        read_frags(st, 0, xf[0], wf[0]);
        keep_scales();
      }
    };
    while (true) {
      clear();
      // (microscaled: the second form costs the first registers, and 8%)
      if constexpr (MX || WGRAD) {
        run(std::true_type{});
      } else {
        if (c.valid > wm * WTM) run(std::true_type{});
        else run(std::false_type{});
      }
      epilogue(c);
      if (t_next < 0) break;
      c = next;
      steps = steps_of(c);
      // the way back wants its registers for itself: the next tile's first
      // fragments are read again
      if constexpr (BACK) read_frags(st, 0, xf[0], wf[0]);
    }
  }
  wait_vmcnt<0>();  // no copy in flight when the workgroup ends
}

// ---------------------------------------------------------------- host side

inline bool given(const gmmfr_tensor& t) {
  if (t.data != nullptr) return true;
  for (int i = 0; i < t.ndim && i < 4; ++i)
    if (t.dims[i] == 0) return true;
  return false;
}
inline bool shape_is(const gmmfr_tensor& t, int nd, int64_t d0, int64_t d1 = 0, int64_t d2 = 0, int64_t d3 = 0) {
  const int64_t d[4] = {d0, d1, d2, d3};
  if (t.ndim != nd) return false;
  for (int i = 0; i < nd; ++i)
    if (t.dims[i] != d[i]) return false;
  return true;
}
inline int aligned(std::initializer_list<const gmmfr_tensor*> all) {
  for (const gmmfr_tensor* t : all)
    if (given(*t) && ((uintptr_t)t->data & 15u) != 0) return GMMFR_ERR_ALIGN;
  return GMMFR_OK;
}

enum Kind { kLarge = 0, kMiddle = 1, kSmall = 2, kThin = 3 };
constexpr int kTileM[4] = {256, 128, 32, 32}, kTileN[4] = {256, 128, 64, 32}, kPerCu[4] = {1, 2, 2, 2};

struct Plan {
  Params p;
  Kind kind;
  int enc, grid;
  bool glu, col;
  bool few;  // weight gradient: its groups are short
};

// tuning: [0] expected rows per expert, [1] forced tile height, [2] cap of the grid
inline int tuning(const int64_t* t, int64_t len, int64_t* rows, int64_t* height, int64_t* cap) {
  *rows = *height = *cap = 0;
  if (len < 0 || (len > 0 && !t)) return GMMFR_ERR_ATTR;
  if (len > 0) *rows = t[0];
  if (len > 1) *height = t[1];
  if (len > 2) *cap = t[2];
  if (*rows < 0 || *cap < 0) return GMMFR_ERR_ATTR;
  if (*height != 0 && *height != 32 && *height != 128 && *height != 256) return GMMFR_ERR_ATTR;
  return GMMFR_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 256-row tiles or 128-row ones, of which `large` and `middle` (in halves) lie
// along M: by the rounds of the chip that they make, a round of 512 small
// tiles (two a CU) taking 0.6 of a round of 256 large ones, 0.65 with
// microscaled operands (measured at 32768 x 2048 x 7168 over 32 experts, 16
// bit: 1.15 against 0.95 ms for the same work; FP4, 12000 x 7168 x 4096 over
// 64: 8 rounds in 0.41 ms against 5 in 0.34).  Other shapes have other factors:
// fp16 (e,n,k), 20011 x 7160 x 2040 over 64, falls to the 128-row tiles by it (4
// rounds against 6), 1011 us, where 256-row ones take 977.
inline Kind larger_kind(int64_t large, int64_t middle, int64_t columns, bool mx) {
  const int64_t l = ceil_div(large * ceil_div(columns, 256), 2 * 256), m = ceil_div(middle * ceil_div(columns, 128), 2 * 512);
  return l * 100 <= m * (mx ? 65 : 60) ? kLarge : kMiddle;
}

inline int grid_of(const Plan& pl, int64_t tiles, int64_t cap) {
  int64_t g = 256 * kPerCu[pl.kind];
  if (cap > 0 && cap < g) g = cap;
  // fewer workgroups than that only in whole rounds of the XCDs
  if (tiles < g) g = cap > 0 && cap < kXcds ? tiles : ceil_div(tiles, kXcds) * kXcds;
  if (cap > 0 && cap < g) g = cap;
  return (int)(g < 1 ? 1 : g);
}

// What the gated forms' plans may take beside the plain product's.
enum More { kThinGate = 1, kFewTiles = 2 };
inline int product_plan(const gmmgm_args* a, Plan* pl, int more = 0) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->x) || !given(a->w) || !given(a->group_list) || !given(a->y)) return GMMFR_ERR_NULLPTR;
  const int xt = a->x.dtype, wt = a->w.dtype, yt = a->y.dtype;
  const bool mx = xt == GMMFR_DT_FLOAT4_E2M1X2 || xt == GMMFR_DT_FLOAT8_E4M3FN;
  if (mx) {
    if (wt != GMMFR_DT_FLOAT4_E2M1X2) return GMMFR_ERR_DTYPE;
    if (!given(a->x_scale) || !given(a->w_scale)) return GMMFR_ERR_NULLPTR;
    if (a->x_scale.dtype != GMMFR_DT_FLOAT8_E8M0 || a->w_scale.dtype != GMMFR_DT_FLOAT8_E8M0) return GMMFR_ERR_DTYPE;
    if (yt != GMMFR_DT_BFLOAT16 && yt != GMMFR_DT_FLOAT16 && yt != GMMFR_DT_FLOAT32) return GMMFR_ERR_DTYPE;
  } else {
    if (xt != GMMFR_DT_BFLOAT16 && xt != GMMFR_DT_FLOAT16) return GMMFR_ERR_DTYPE;
    if (wt != xt || (yt != xt && yt != GMMFR_DT_FLOAT32)) return GMMFR_ERR_DTYPE;
    if (given(a->x_scale) || given(a->w_scale)) return GMMFR_ERR_UNSUPPORTED;
  }
  if (a->group_list.dtype != GMMFR_DT_INT64) return GMMFR_ERR_DTYPE;
  if (a->group_list_type != 0 && a->group_list_type != 1) return GMMFR_ERR_ATTR;
  if (a->transpose_w != 0 && a->transpose_w != 1) return GMMFR_ERR_ATTR;
  if (mx && a->transpose_w != 1) return GMMFR_ERR_ATTR;
  if (a->activation != GMMGM_ACT_NONE && a->activation != GMMGM_ACT_SWIGLU) return GMMFR_ERR_ATTR;
  int64_t rows, height, cap;
  if (tuning(a->tuning_config, a->tuning_config_len, &rows, &height, &cap) != GMMFR_OK) return GMMFR_ERR_ATTR;
  const bool glu = a->activation == GMMGM_ACT_SWIGLU;
  if (a->x.ndim != 2 || a->w.ndim != 3 || a->group_list.ndim != 1) return GMMFR_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if ((i < 2 && a->x.dims[i] >= (int64_t(1) << 31)) || a->w.dims[i] >= (int64_t(1) << 31)) return GMMFR_ERR_SHAPE;
  const int per = xt == GMMFR_DT_FLOAT4_E2M1X2 ? 2 : 1, wper = mx ? 2 : 1;  // values an element of the shape stands for
  const int64_t m = a->x.dims[0], k = a->x.dims[1] * per, e = a->w.dims[0];
  const int64_t n = a->w.dims[a->transpose_w ? 1 : 2], wk = a->w.dims[a->transpose_w ? 2 : 1] * wper;
  if (m < 0 || m >= (int64_t(1) << 31) || e < 1 || e > kMaxExperts) return GMMFR_ERR_SHAPE;
  const int64_t unit = mx ? 64 : 8;
  if (k < unit || k > 65536 || k % unit != 0 || wk != k) return GMMFR_ERR_SHAPE;
  const int64_t nunit = glu ? 16 : 8;
  if (n < nunit || n > 65536 || n % nunit != 0 || m * n >= (int64_t(1) << 40)) return GMMFR_ERR_SHAPE;
  // SwiGLU reaches n/2 weight columns away from a tile's own: 31-bit offsets
  if (glu && a->transpose_w && n * k * (mx ? 1 : 4) / 2 > (int64_t(1) << 31)) return GMMFR_ERR_SHAPE;
  if (a->group_list.dims[0] != e) return GMMFR_ERR_SHAPE;
  if (mx && (!shape_is(a->x_scale, 3, m, k / 64, 2) || !shape_is(a->w_scale, 4, e, n, k / 64, 2))) return GMMFR_ERR_SHAPE;
  if (!shape_is(a->y, 2, m, glu ? n / 2 : n)) return GMMFR_ERR_SHAPE;
  if (aligned({&a->x, &a->w, &a->x_scale, &a->w_scale, &a->group_list, &a->y}) != GMMFR_OK) return GMMFR_ERR_ALIGN;
  Params& p = pl->p;
  p.x = a->x.data;
  p.w = a->w.data;
  p.xs = (const uint8_t*)a->x_scale.data;
  p.ws = (const uint8_t*)a->w_scale.data;
  p.group_list = (const int64_t*)a->group_list.data;
  p.y = a->y.data;
  p.m = m;
  p.k = k;
  p.n = n;
  p.e = (int32_t)e;
  p.cumulative = a->group_list_type == 0;
  p.out = yt == GMMFR_DT_FLOAT32 ? kOutF32 : (yt == GMMFR_DT_FLOAT16 ? kOutF16 : kOutBf16);
  p.accumulate = 0;
  pl->enc = xt == GMMFR_DT_BFLOAT16 ? kBf16 : xt == GMMFR_DT_FLOAT16 ? kF16 : per == 2 ? kFp4 : kFp8;
  pl->glu = glu;
  pl->col = a->transpose_w == 0;
  // By the rows an expert is likely to have (experts without rows cost
  // nothing).  Few rows: the narrow tiles, which stream the weights (us, narrow
  // against 128-row; e experts, k = 7168):
  //   FP8, n = 4096      e = 64:   32 rows 275, 319   40 rows 328, 280
  //   FP4, n = 2048      e = 32:   12 rows  52,  56   24 rows  68,  57
  //   (e,n,k), n = 2048  e = 32:   12 rows 147, 166   24 rows 188, 169
  // While the 128-row tiles leave CUs idle, up to 32 rows in all of them:
  //   FP4, n = 2048      e = 16:   32 rows  39,  40   e = 8:  22,  35
  //   (e,n,k), n = 2048  e = 16:   24 rows 124, 128   e = 8:  63, 103
  // Weights (e,k,n), of which a narrow tile takes half as much of a row at a
  // time, only then:
  //   (e,k,n), n = 2048  e = 32:   12 rows 181, 168   e = 16: 91, 116
  //   (e,k,n), n = 2048  e = 16:   24 rows 147, 117   e = 8:  77,  98
  // Tiles along M, in halves, for the choice among the others: one an expert up
  // to three quarters of a tile, then half a tile of each cut short (bf16, 64
  // experts of 188 rows, 2048 x 7168: 606 us with half a tile cut always, 501 so;
  // FP8 315 and 258, and with much skewed groups 299 and 302).
  // With expected rows: as many experts as m has of them, each in whole tiles of
  // that many (2048 x 7168 bf16 (e,k,n), us under 128-row and 256-row tiles; the
  // one taken without them, and with):
  //   8 of 256 experts, 1024 rows each of m = 8192   298, 236   first, second
  //   32 of 256, 256 rows each of m = 8192           335, 272   first, second
  //   32 experts, 40 rows each of m = 32768          192, 216   second, first
  //   32 experts, 150 rows each of m = 32768         265, 245   second, second
  const int64_t parts = e < m ? e : m;
  if (rows > m) rows = m;
  int64_t avg = m / (parts > 0 ? parts : 1), busy = parts;
  if (rows > 0) {
    avg = rows;
    if (ceil_div(m, rows) < busy) busy = ceil_div(m, rows);
  }
  const int64_t middle = busy * ceil_div(n, kTileN[kMiddle]);  // 128-row tiles, one row of them an expert
  // The gated forms take the narrow tiles too where all of them are one round of
  // the chip, or two with weights (e,n,k): 128-row tiles leave most CUs idle then
  // (us, narrow against 128-row, 16 bits kept, (e,n,k) and (e,k,n); forward):
  //   1 of 7168 x 4096, 64 rows     128 tiles   26, 102    56,  99
  //   8 of 7168 x 2048, 40 rows     512         43,  77    65,  74
  //   6 of 6352 x 512, 269 rows     432         60,  92    60,  88
  //   2 of 7168 x 4096, 256 rows   1024         77,  81    95,  79
  // (way back, (e,f,d), the last two: 34, 97 and 45, 86).
  const int64_t few = busy * ceil_div(avg, 32) * ceil_div(n, 64);
  const bool narrow = ((more & kFewTiles) && few <= (pl->col ? 512 : 1024)) ||
                      (avg <= 16 ? !pl->col || middle <= 256
                                 : avg <= 32 && (pl->enc == kFp8 || middle <= (pl->col ? 128 : 256)));
  // One expert's rows are known but for those behind it: whole tiles of them
  // (4096 rows of 7168, us under 128-row and 256-row tiles; inputs not in the
  // caches, and in them):
  //   n = 4096   bf16 (e,n,k) 249, 205 and 216, 183   FP4 95, 76 and 89, 72   FP8 147, 118 and 124, 99
  //   n = 2048   bf16 (e,n,k) 148, 198 and 113, 146   FP4 54, 74 and 53, 65   FP8 81, 110 and 71, 92
  auto along = [&](int64_t t) {
    if (parts == 1) return 2 * ceil_div(rows > 0 ? rows : m, t);
    if (rows > 0) return 2 * busy * ceil_div(rows, t);
    return 4 * m <= 3 * t * busy ? 2 * busy : 2 * m / t + busy;
  };
  pl->kind = height ? (height == 256 ? kLarge : height == 128 ? kMiddle : kSmall)
                    : (narrow ? kSmall : larger_kind(along(256), along(128), n, mx));
  auto tiles_of = [&](Kind kind) -> int64_t {
    p.tiles_n = (int32_t)ceil_div(n, kTileN[kind]);
    // at most this many tiles: whole ones, and one part a non-empty expert
    return (m / kTileM[kind] + parts) * p.tiles_n;
  };
  p.tiles_m = 0;
  int64_t tiles = tiles_of(pl->kind);
  // Narrow tiles that leave CUs without one: a CU streams weights at 27 GB/s
  // whatever is in flight (stages twice as deep, or twice as long: slower), so
  // they are cut in two for twice as many.  Weights (e,n,k) of 16 bits only:
  // those of (e,k,n) would be read half a line at a time, and the scales of
  // microscaled ones are staged for 64 columns.  us, 64 columns against 32:
  //   7168 x 4096, 1 row    64 tiles  34, 24    16384 x 8192      128  74, 59
  //   8 of 2048 x 1024     128        14, 11    16 of 2048 x 1024 256  18, 18
  // (in the caches; not in them the first 40, 27 and 77, 63 with a launch's events)
  if (pl->kind == kSmall && !mx && (!glu || (more & kThinGate)) && !pl->col && tiles <= 256) tiles = tiles_of(pl->kind = kThin);
  if (tiles >= (int64_t(1) << 31)) return GMMFR_ERR_SHAPE;
  pl->grid = grid_of(*pl, tiles, cap);
  return GMMFR_OK;
}

// eight: one of the two is kept in FP8.
inline int wgrad_plan(const gmmgw_args* a, Plan* pl, bool eight = false) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->x) || !given(a->dy) || !given(a->group_list) || !given(a->dw)) return GMMFR_ERR_NULLPTR;
  const int xt = a->x.dtype, ot = a->dw.dtype;
  if (xt != GMMFR_DT_BFLOAT16 && xt != GMMFR_DT_FLOAT16) return GMMFR_ERR_DTYPE;
  if (a->dy.dtype != xt || (ot != xt && ot != GMMFR_DT_FLOAT32)) return GMMFR_ERR_DTYPE;
  if (a->group_list.dtype != GMMFR_DT_INT64) return GMMFR_ERR_DTYPE;
  if (a->group_list_type != 0 && a->group_list_type != 1) return GMMFR_ERR_ATTR;
  if (a->accumulate != 0 && (a->accumulate != 1 || ot != GMMFR_DT_FLOAT32)) return GMMFR_ERR_ATTR;
  int64_t rows, height, cap;
  if (tuning(a->tuning_config, a->tuning_config_len, &rows, &height, &cap) != GMMFR_OK || height == 32)
    return GMMFR_ERR_ATTR;
  if (a->x.ndim != 2 || a->dy.ndim != 2 || a->group_list.ndim != 1) return GMMFR_ERR_SHAPE;
  const int64_t m = a->x.dims[0], k = a->x.dims[1], n = a->dy.dims[1], e = a->group_list.dims[0];
  if (m < 0 || m >= (int64_t(1) << 31) || a->dy.dims[0] != m || e < 1 || e > kMaxExperts) return GMMFR_ERR_SHAPE;
  if (k < 8 || k > 65536 || k % 8 != 0 || n < 8 || n > 65536 || n % 8 != 0) return GMMFR_ERR_SHAPE;
  if (!shape_is(a->dw, 3, e, k, n)) return GMMFR_ERR_SHAPE;
  if (aligned({&a->x, &a->dy, &a->group_list, &a->dw}) != GMMFR_OK) return GMMFR_ERR_ALIGN;
  Params& p = pl->p;
  p.x = a->x.data;
  p.w = a->dy.data;
  p.xs = p.ws = nullptr;
  p.group_list = (const int64_t*)a->group_list.data;
  p.y = a->dw.data;
  p.m = m;
  p.k = k;
  p.n = n;
  p.e = (int32_t)e;
  p.cumulative = a->group_list_type == 0;
  p.out = ot == GMMFR_DT_FLOAT32 ? kOutF32 : (ot == GMMFR_DT_FLOAT16 ? kOutF16 : kOutBf16);
  p.accumulate = a->accumulate;
  pl->enc = xt == GMMFR_DT_BFLOAT16 ? kBf16 : kF16;
  pl->glu = false;
  pl->col = true;
  // Few rows an expert are a few steps: with results of 16 bits, which do not
  // fill the memory's time, two workgroups a CU hide the tiles' ends, but read
  // each row twice as often.  So the 128-row tiles are taken where the others
  // make two rounds of the chip at most, or a sixteenth more work at the ends of
  // rounds and matrices, or where the rows are fewest beside the columns (us
  // under 128-row and 256-row tiles, rows and results not in the caches):
  //   two rounds      4 of 2048 x 2048, 8 rows   15.3, 17.8   64 of 512 x 512, 64 rows    16.5, 18.7
  //   less work       4 of 7168 x 2048, 64 rows  40, 48       64 of 2880 x 2880, 64 rows  343, 379
  //   fewest rows     16 of 4096 x 8192, 8 rows  293, 330     64 of 2048 x 2048, 4 rows   165, 171
  //   none of them    64 of 2048 x 2048, 64 rows 188, 179     64 of 1024 x 4096, 64 rows  204, 174
  //                   16 of 2048 x 4096, 16 rows 94, 88       64 of 1024 x 1024, 64 rows  52.6, 48.5
  // (results in fp32, in the caches: 32 of 2048 x 2048, 8 rows 148, 110).  Rows
  // kept in FP8 cost half of that, and something a step of 32 of them: the
  // 128-row tiles for one step (64 of 1536 x 2048: 4 rows 129, 145, 32 rows 135,
  // 145, 48 rows 146, 145, 64 rows 152, 143; 64 of 1024 x 4096: 32 rows 190,
  // 183, 48 rows 206, 183).
  const int64_t large = e * ceil_div(k, 256) * ceil_div(n, 256), middle = e * ceil_div(k, 128) * ceil_div(n, 128);
  const int64_t rounds = ceil_div(large, 256);
  const bool fine = ot != GMMFR_DT_FLOAT32 &&
                    (eight ? m <= 32 * e
                           : m <= 64 * e && (rounds <= 2 || middle * 8 <= 15 * 512 * rounds || (k >= 2048 && 512 * m <= e * k)));
  pl->kind = height ? (height == 256 ? kLarge : kMiddle)
             : fine ? kMiddle
                    : larger_kind(2 * e * ceil_div(k, 256), 2 * e * ceil_div(k, 128), n, false);
  pl->few = m < 1024 * e;  // (fragments read early: see above; 375 rows 28.9 us, between 29 to 33; 1024: 45.7, 44.4)
  p.tiles_m = (int32_t)ceil_div(k, kTileM[pl->kind]);
  p.tiles_n = (int32_t)ceil_div(n, kTileN[pl->kind]);
  pl->grid = grid_of(*pl, e * p.tiles_m * p.tiles_n, cap);
  return GMMFR_OK;
}

// What the callers' plan queries give of a plan.
inline int describe(int status, const Plan& pl, gmmgm_plan_info* info) {
  if (status != GMMFR_OK) return status;
  if (!info) return GMMFR_ERR_NULLPTR;
  info->tile_m = kTileM[pl.kind];
  info->tile_n = kTileN[pl.kind];
  info->grid = pl.grid;
  return GMMFR_OK;
}

// (hipLaunchKernel gives this launch's own status, where the runtime's last
// error may be an earlier one of the program's)
template <int ENC, bool XCOL, bool WCOL, bool WGRAD, bool GLU, int FORM = kStore, bool EARLY = ENC == kFp8>
hipError_t launch(Plan& pl, hipStream_t s) {
  const size_t dyn = (size_t)(2 * pl.p.e + 1) * 4;
  constexpr int BK = ENC == kFp4 ? 256 : (ENC == kFp8 ? 128 : 64), BKS = ENC == kFp8 ? 256 : BK;
  constexpr int STS = ENC == kFp8 ? 3 : (ENC == kFp4 ? 4 : 5);
  constexpr bool FOUR = WGRAD || FORM == kBackFull || FORM == kBackFp8;  // waves of 128 x 128
  pl.p.grid = pl.grid;
  void* args[] = {&pl.p};
  if (pl.kind == kLarge)
    // The weight gradient's stages are whole rows of a tile whatever their
    // length: four short ones hide more of a copy's way than two long ones
    // (1.27 -> 1.20 ms at 32768 x 2048 x 7168); with rows along the reduction
    // short stages would take half a line at a time (2-7% slower).  Four waves
    // of 128 x 128 read a third less from LDS than eight of 64 x 128, which
    // transposing reads make up for (1.20 -> 1.12 ms; without them -1 .. +2%).
    return hipLaunchKernel((const void*)product_kernel<ENC, XCOL, WCOL, WGRAD, GLU, 256, 256, WGRAD ? BK / 2 : BK,
                                                       FOUR ? 2 : 4, 2, WGRAD ? 4 : 2, false, FOUR ? 1 : 2, FORM, kNone8, EARLY>,
                           dim3(pl.grid), dim3(FOUR ? 256 : 512), args, dyn, s);
  if constexpr (!WGRAD) {
    if constexpr ((ENC == kBf16 || ENC == kF16) && !WCOL && (!GLU || FORM == kGated)) {
      if (pl.kind == kThin)
        return hipLaunchKernel((const void*)product_kernel<ENC, XCOL, WCOL, WGRAD, GLU, 32, 32, BK, 2, 2, STS, true, 2, FORM>,
                               dim3(pl.grid), dim3(256), args, dyn, s);
    }
    if (pl.kind == kSmall)
      return hipLaunchKernel((const void*)product_kernel<ENC, XCOL, WCOL, WGRAD, GLU, 32, 64, BKS, 2, 2, STS, true, 2, FORM>,
                             dim3(pl.grid), dim3(256), args, dyn, s);
  }
  return hipLaunchKernel((const void*)product_kernel<ENC, XCOL, WCOL, WGRAD, GLU, 128, 128, BK, 2, 2, 2, false, 2, FORM>,
                         dim3(pl.grid), dim3(256), args, dyn, s);
}

}  // namespace gmmgm
