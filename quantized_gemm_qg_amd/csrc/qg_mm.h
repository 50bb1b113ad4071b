// Tiled matrix product of the int8 layers, the bf16 gated feed-forward block and the
// cross entropy of a head: Y[r][c] = sum_k A(r, k) B(c, k), int8 x int8 into int32 or bf16 x bf16
// into fp32, with three operand forms:
//
//   kRows    the operand's rows run along k ([row][pitch], k contiguous):
//            activations, bf16 weights, the gradient of the pre-activations
//   kPacked  int8 weights in the packed layout (1-KB pieces of 16 columns x 64 k)
//   kCols    k runs along the rows of the stored matrix ([k][pitch], the
//            operand's own index contiguous): the backward products contract
//            over tokens or over the feed-forward index, which no stored
//            matrix has contiguous, so the fragments are transposed on their
//            way out of LDS (ds_read_b64_tr_b16) instead of in memory
//
// A workgroup computes a BM x BN tile with WM x WN waves as blocks of 16 x 16
// (v_mfma_i32_16x16x64_i8 / v_mfma_f32_16x16x32_bf16: both take 64 bytes of k
// per row, 16 per lane).  The operands go through a ring of ST stages of 128
// bytes of k (a cache line per row; with 64 every line was fetched twice), filled by global_load_lds_dwordx4 (1 KB per wave and copy, no
// register staging), and from LDS into a second set of operand registers while
// the first one multiplies.  Bank conflicts: row chunks of 16 bytes sit at slot
// chunk ^ f(row), the 32-byte column units of kCols at unit ^ f(k); packed pieces
// are read in the order they are stored.  Past the last k both operands read a
// line of zeros (nothing is multiplied by what lies behind a row), past the last
// row or column the last valid one (never stored).
//
// The weights are the MFMA's first operand, so a lane holds four consecutive
// columns of one row: the epilogue packs them with one LDS write per block and
// stores 16 bytes per lane along the rows.
//
// Bounds and rates: large products by the matrix cores, which run into the power
// limit (1.65-1.75 GHz; busy 65-72 % of the cycles in bf16, 55 % in int8): int8 4096
// x 14336 x 4096 224 us (2.1 POP/s), bf16 4096 x 4096 x 28672 with one operand
// transposed 725 us (1.33 PFLOP/s), with both 750 us.  (The int8 256 x 256 shapes
// spill 14 to 20 registers, between the loop and the epilogue.)  128 x 128 tiles by LDS (96 KB
// read and 32 KB written per stage, 1024 clocks for 512 of products), small
// batches by the latency of their stages and of the join.
//
// Gated: the tile's B columns are half gate and half up columns of the same
// BN / 2 outputs, and every wave owns both halves of its outputs, so
// act(g) u is computed on the accumulators.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qg_device.h"
#include "qg_internal.h"

namespace qg {

enum { kRows = 0, kPacked = 1, kCols = 2 };

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // 16 bytes at any element

// bf16 bits, nearest-even (a NaN stays a NaN)
__device__ __forceinline__ uint32_t bf16_rne(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

// act(g) = g p(g) and its derivative, p = 1 / (1 + exp(-z)): z = g for SiLU; for
// GELU z = 2 sqrt(2 / pi) (g + 0.044715 g^3), as (1 + tanh(y)) / 2 = p(2 y), which
// costs an exponential and a reciprocal and keeps the relative accuracy where
// 1 + tanh cancels.  derivative: p + g p (1 - p) z'.
__device__ __forceinline__ float act_gate(float g, int act) {
  const float z = act == QG_ACT_SILU ? g : 1.5957691216057308f * g * (1.f + 0.044715f * g * g);
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
__device__ __forceinline__ float act_value(float g, int act) { return g * act_gate(g, act); }
__device__ __forceinline__ void act_both(float g, int act, float *v, float *dv) {
  const float p = act_gate(g, act), r = p * (1.f - p);
  const float dz = act == QG_ACT_SILU ? 1.f : 1.5957691216057308f * (1.f + 0.134145f * g * g);
  *v = g * p;
  *dv = r > 0.f ? p + g * r * dz : p;  // (r = 0: dz may have overflowed)
}

struct MmArgs {
  const uint8_t *a;  // kRows: [m][lda]; kCols: [kd][lda]
  int64_t lda;       // bytes
  const uint8_t *b;  // kRows: [columns][ldb]; kCols: [kd][ldb]; kPacked: the codes
  int64_t ldb;       // bytes; kPacked: bytes of one 16-column strip
  int32_t m, n;      // output rows and columns (gated: n = inter, B has 2 n columns)
  int32_t kd;        // contraction length
  void *y;
  int64_t ldy;       // elements
  int32_t otype;
  const float *sa;   // int8: scale of each row, of each B column
  const float *sb;
  void *gu;          // gated: the pre-activations, or NULL
  int64_t ldgu;
  int32_t gu_type;
  int32_t act;
  // bf16 backward of few tokens: the operand A is the sum of two bf16 parts, the
  // second one `halves` (0: there is none) rows behind the first.  kRows: both
  // are rows of one tile, m counts to the last, and output row r is r plus
  // r + halves; kCols: kd counts to the last (one stage), B's row repeats.
  int32_t halves;
  int32_t group_m;
  // split over k: `per` stages each; one arrival counter per tile and the
  // partial tiles [split][tile]
  int32_t splits, per;
  uint32_t *counters;
  uint64_t *partials;
};

// What the other epilogues need besides (apart: the longer arguments alone cost the
// int8 product of 333 rows 3 %).
struct MmMoreArgs : MmArgs {
  // cross entropy of a head (kXentStats, kXentGrad): y's columns are the logits of
  // tokens first_token ..; kXentStats leaves the largest logit and the sum of
  // exponentials of every row and tile in stats [tile][m] and the target's logit
  // in at_target; kXentGrad writes weight (softmax - target), weight the rows' dloss
  // over their largest, alpha_out = scale times that
  const int32_t *targets;
  int32_t first_token;
  float scale;
  float *stats, *at_target;
  const float *lse, *dloss, *dloss_most;  // (dloss_most: found before, or NULL)
  float *alpha_out;
  int32_t vocab;
  // kScaled: y = alpha[0] times the product.  kParts: split over k without a join,
  // part p's sums go to y + p part_stride (fp32), on top of what is there where p <
  // parts_there
  const float *alpha;
  int64_t part_stride;
  int32_t parts_there;
};

// What is done with a tile's sums besides storing them.
enum { kPlain = 0, kXentStats = 1, kXentGrad = 2, kScaled = 3, kParts = 4 };

// Partial tiles of a call take at most this much.
constexpr uint64_t kMmPartialBytes = 48u << 20;

// 16 zero bytes that copies past the last k read
static __device__ const uint32_t mm_zeros[4] = {0u, 0u, 0u, 0u};

// SPLIT: the tile's k may be shared by several workgroups.
template <bool I8_, int AF_, int BF_, bool GATED_, int BM_, int BN_, int WM_, int WN_, int ST_, bool SPLIT_,
          int EPI_ = kPlain>
struct MmCfg {
  static constexpr int EPI = EPI_;
  using Args = typename std::conditional<EPI == 0, MmArgs, MmMoreArgs>::type;
  static constexpr bool I8 = I8_, GATED = GATED_;
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int AF = AF_, BF = BF_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, KB = 128, ST = ST_;
  static constexpr int EL = I8 ? 1 : 2;
  static constexpr int KE = KB / EL;             // k per stage
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  static constexpr int SUB = KB / 64;            // MFMA steps per stage
  static constexpr int A = BM * KB, B = BN * KB, STAGE = A + B;
  static constexpr int A_COPIES = A / 1024, B_COPIES = B / 1024;
  static constexpr int A_LOADS = (A_COPIES + WAVES - 1) / WAVES, B_LOADS = (B_COPIES + WAVES - 1) / WAVES;
  static constexpr int LOADS = A_LOADS + B_LOADS;
  static constexpr int OUT_NB = GATED ? NB / 2 : NB;                  // 16-column blocks of a wave's output
  static constexpr int PITCH = 16 * OUT_NB * 4 + 16;                  // bytes of a slab row (fp32)
  static constexpr int SLAB = 16 * PITCH;
  static constexpr int OUT = WAVES * SLAB + (EPI == kXentGrad ? 16 * BM : 0);  // slabs, rows' values
  static constexpr int LDS = STAGE * ST > OUT ? STAGE * ST : OUT;
  static constexpr bool ROW_HALVES = !I8 && AF == kRows && BF == kCols && BM == 32, K_HALVES = AF == kCols;
  static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && (!GATED || NB % 2 == 0), "blocks");
  static_assert(!I8 || AF == kRows, "int8 activations are rows");
  static_assert(AF != kCols || BM >= 128, "column units for the swizzle");
  static_assert(BF != kCols || BN >= 128, "column units for the swizzle");
  static_assert(LDS <= 160 * 1024 && ST >= 2 && ST <= 4, "LDS ring");
  static_assert(EPI == kPlain || (!I8 && !GATED), "epilogues of the bf16 products");
};

// Waits until at most `stages` (0 .. 3) stages of LOADS loads each are out.
template <int LOADS>
__device__ __forceinline__ void wait_loads(int stages) {
  static_assert(3 * LOADS < 64, "outstanding loads");
  if (stages >= 3) {
    QG_WAIT_VMCNT(3 * LOADS);
  } else if (stages == 2) {
    QG_WAIT_VMCNT(2 * LOADS);
  } else if (stages == 1) {
    QG_WAIT_VMCNT(LOADS);
  } else {
    QG_WAIT_VMCNT(0);
  }
}

// Workgroup barrier that no memory access moves across and that no wave reaches
// with an LDS access out: s_barrier itself waits for none, and the compiler may
// sink the products that a read feeds (and its wait) below it, while other waves
// write the same LDS behind it.
__device__ __forceinline__ void mm_barrier() {
  asm volatile("" ::: "memory");
  QG_WAIT_LGKMCNT0();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Direct global -> LDS copies of 16 bytes per lane, at a lane offset from a
// uniform base or at a lane's own address; `lds` (uniform) receives the wave's
// 1 KB.  Written out because the builtin makes the compiler wait for every
// outstanding copy before each transposed LDS read (it cannot tell the stages
// of the ring apart there); the waits are wait_loads above.  The instruction
// has no destination register.  m0 is a reserved register, which the compiler
// does not preserve around such a clobber and warns about for every copy: these
// kernels name it nowhere else, so there is nothing to preserve.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void mm_copy16(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void mm_copy16_at(const uint8_t *src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop

// chunk order of a row's 16-byte chunks
__device__ __forceinline__ int row_swz(int row) { return row & 7; }
// unit order of a k row's 32-byte column units
__device__ __forceinline__ int col_swz(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

template <class C>
__global__ __launch_bounds__(C::THREADS) void mm_kernel(typename C::Args a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  typedef typename std::conditional<C::I8, i32x4, f32x4>::type Acc;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int q = lane >> 4, r16 = lane & 15;
  constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;  // output columns per tile

  const int m_tiles = (a.m + C::BM - 1) / C::BM, n_tiles = (a.n + OUT_BN - 1) / OUT_BN;
  int tm, tn, pid = blockIdx.x, split = 0;
  if constexpr (C::SPLIT) {
    const int grid1 = gridDim.x / a.splits;  // a multiple of the XCDs
    split = pid / grid1;
    pid -= split * grid1;
  }
  if (!tile_of(pid, m_tiles, n_tiles, a.group_m, &tm, &tn)) return;
  const int m0 = tm * C::BM, n0 = tn * OUT_BN;
  const int rows = min(C::BM, a.m - m0);
  static_assert(C::EPI != kXentGrad || C::THREADS >= C::BM, "a thread per row");
  f32x4 my_row = {0.f, 0.f, 0.f, 0.f};  // kXentGrad: what the epilogue needs of this thread's row
  float dloss_most = 0.f;  // the wave's, then the workgroup's
  if constexpr (C::EPI == kXentGrad) {
    // (every workgroup looks for the largest |dloss| of the rows that count: a launch
    // of its own for it took 5 us)
    auto dloss_of = [&](int r) { return (uint32_t)a.targets[r] < (uint32_t)a.vocab ? a.dloss[r] : 0.f; };
    if (a.dloss_most)
      dloss_most = a.dloss_most[0];
    else
      for (int r = threadIdx.x; r < a.m; r += C::THREADS) dloss_most = fmaxf(dloss_most, fabsf(dloss_of(r)));
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) dloss_most = fmaxf(dloss_most, __shfl_xor(dloss_most, off));
    dloss_most = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(dloss_most)));
    const int row = min(m0 + (int)threadIdx.x, a.m - 1);
    my_row = f32x4{dloss_of(row), a.lse[row] * 1.4426950408889634f, __int_as_float(a.targets[row] - a.first_token), 0.f};
  }

  // B column of block jb of the tile (the up half of a gated tile starts at
  // column n), not clamped; and the last valid one of its half
  auto b_col = [&](int jb, int r, bool *up) {
    if constexpr (C::GATED) {
      const int w = jb / C::NB, j = jb % C::NB;
      *up = j >= C::NB / 2;
      return n0 + (w * (C::NB / 2) + (j % (C::NB / 2))) * 16 + r;
    } else {
      *up = false;
      return n0 + jb * 16 + r;
    }
  };

  // source offset of each copy of this wave (from a 64-bit base per operand),
  // and the k, inside a stage, of the 16 bytes
  uint32_t a_off[C::A_LOADS], b_off[C::B_LOADS];
  int a_k[C::A_LOADS], b_k[C::B_LOADS];
  bool b_up[C::B_LOADS];
  auto a_copy = [&](int i) { return min(wave * C::A_LOADS + i, C::A_COPIES - 1); };
  auto b_copy = [&](int i) { return min(wave * C::B_LOADS + i, C::B_COPIES - 1); };
  constexpr int CPR = C::KB / 16;  // chunks per row
#pragma unroll
  for (int i = 0; i < C::A_LOADS; ++i) {
    if constexpr (C::AF == kRows) {
      const int row = a_copy(i) * (64 / CPR) + lane / CPR;
      const int c = (lane % CPR) ^ row_swz(row);
      a_off[i] = (uint32_t)((int64_t)min(row, rows - 1) * a.lda + 16 * c);
      a_k[i] = 16 * c / C::EL;
    } else {
      const int k = a_copy(i) * (512 / C::BM) + lane / (C::BM / 8), s = lane % (C::BM / 8);
      const int col = 16 * ((s >> 1) ^ col_swz(k)) + 8 * (s & 1);
      a_off[i] = (uint32_t)(k * a.lda + 2 * min(col, ((a.m + 7) & ~7) - 8 - m0));
      a_k[i] = k;
    }
  }
#pragma unroll
  for (int i = 0; i < C::B_LOADS; ++i) {
    if constexpr (C::BF == kRows) {
      const int row = b_copy(i) * (64 / CPR) + lane / CPR;
      const int c = (lane % CPR) ^ row_swz(row);
      const int col = b_col(row / 16, row % 16, &b_up[i]);
      b_off[i] = (uint32_t)((int64_t)(min(col, a.n - 1) - n0) * a.ldb + 16 * c);
      b_k[i] = 16 * c / C::EL;
    } else if constexpr (C::BF == kPacked) {
      const int jb = b_copy(i) / C::SUB, half = b_copy(i) % C::SUB;
      int col = min(b_col(jb, r16, &b_up[i]), a.n - 1);
      const int first = b_up[i] ? (a.n + n0) / 16 : n0 / 16;  // strip of the base below
      if (b_up[i]) col += a.n;
      b_off[i] = (uint32_t)((int64_t)(col / 16 - first) * a.ldb + half * 1024 + q * 256 + (col % 16) * 16);
      b_k[i] = 0;  // padded with zeros to whole 128-k blocks
    } else {
      const int k = b_copy(i) * (512 / C::BN) + lane / (C::BN / 8), s = lane % (C::BN / 8);
      const int col = 16 * ((s >> 1) ^ col_swz(k)) + 8 * (s & 1);
      const int row = C::K_HALVES && a.halves > 0 && k >= a.halves ? k - a.halves : k;
      b_off[i] = (uint32_t)(row * a.ldb + 2 * min(col, ((a.n + 7) & ~7) - 8 - n0));
      b_k[i] = k;
      b_up[i] = false;
    }
  }
  const uint8_t *a_base = a.a + (C::AF == kRows ? (int64_t)m0 * a.lda : (int64_t)m0 * 2);
  const uint8_t *b_base, *b_base_up;
  if constexpr (C::BF == kRows) {
    b_base = a.b + (int64_t)n0 * a.ldb;
    b_base_up = b_base + (int64_t)a.n * a.ldb;
  } else if constexpr (C::BF == kPacked) {
    b_base = a.b + (int64_t)(n0 / 16) * a.ldb;
    b_base_up = a.b + (int64_t)((a.n + n0) / 16) * a.ldb;
  } else {
    b_base = b_base_up = a.b + (int64_t)n0 * 2;
  }
  // bytes from one stage to the next
  const int64_t a_step = C::AF == kRows ? C::KB : (int64_t)C::KE * a.lda;
  const int64_t b_step = C::BF == kRows ? C::KB : C::BF == kPacked ? 1024 * C::SUB : (int64_t)C::KE * a.ldb;
  // stages first .. steps - 1 of k are this workgroup's
  const int all_steps = (a.kd + C::KE - 1) / C::KE;
  const int first = C::SPLIT ? split * a.per : 0;
  const int steps = C::SPLIT ? min(first + a.per, all_steps) : all_steps;

  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;
  auto issue = [&](int s) {
    const uint32_t st = ring + (s % C::ST) * C::STAGE;
    const uint8_t *as = a_base + s * a_step, *bs = b_base + s * b_step;
    const int64_t up = b_base_up - b_base;
    if ((s + 1) * C::KE <= a.kd) {
#pragma unroll
      for (int i = 0; i < C::A_LOADS; ++i) mm_copy16(as, a_off[i], st + a_copy(i) * 1024);
#pragma unroll
      for (int i = 0; i < C::B_LOADS; ++i)
        mm_copy16(bs + (b_up[i] ? up : 0), b_off[i], st + C::A + b_copy(i) * 1024);
    } else {
      const int left = a.kd - s * C::KE;
      // (between two halves nothing)
      auto in = [&](int k) { return k < left && !(C::K_HALVES && k >= left - a.halves && k < a.halves); };
#pragma unroll
      for (int i = 0; i < C::A_LOADS; ++i)
        mm_copy16_at(in(a_k[i]) ? as + a_off[i] : (const uint8_t *)mm_zeros, st + a_copy(i) * 1024);
#pragma unroll
      for (int i = 0; i < C::B_LOADS; ++i)
        mm_copy16_at(in(b_k[i]) ? bs + (b_up[i] ? up : 0) + b_off[i] : (const uint8_t *)mm_zeros,
                     st + C::A + b_copy(i) * 1024);
    }
  };

  // Fragments of one stage in registers.  kRows: row 16 blk + r16, its swizzle
  // depends on r16 alone.  kCols: k 32 u + 8 q + 0..3 and + 4..7 of column
  // 16 blk + r16; within 16 lanes, lane i names k row i / 4 and columns 4 (i % 4)
  // .. + 3 and receives column i; the unit swizzle depends on i / 4 and q alone.
  // So every address is a lane offset per operand (kCols: per block) plus
  // constants.
  uint32_t a_at[C::AF == kCols ? C::MB : C::SUB], b_at[C::BF == kCols ? C::NB : C::SUB];
  const int ksw = (r16 >> 2) | ((q & 1) << 2);
  if constexpr (C::AF == kCols) {
#pragma unroll
    for (int i = 0; i < C::MB; ++i)
      a_at[i] = (8 * q + (r16 >> 2)) * (2 * C::BM) + 32 * ((wm * C::MB + i) ^ ksw) + 8 * (r16 & 3);
  } else {
#pragma unroll
    for (int u = 0; u < C::SUB; ++u)
      a_at[u] = (wm * C::MB * 16 + r16) * C::KB + 16 * ((4 * u + q) ^ row_swz(r16));
  }
  if constexpr (C::BF == kCols) {
#pragma unroll
    for (int j = 0; j < C::NB; ++j)
      b_at[j] = C::A + (8 * q + (r16 >> 2)) * (2 * C::BN) + 32 * ((wn * C::NB + j) ^ ksw) + 8 * (r16 & 3);
  } else {
#pragma unroll
    for (int u = 0; u < C::SUB; ++u)
      b_at[u] = C::A + (C::BF == kRows ? (wn * C::NB * 16 + r16) * C::KB + 16 * ((4 * u + q) ^ row_swz(r16))
                                       : (wn * C::NB * C::SUB + u) * 1024 + 16 * lane);
  }
  auto cols_frag = [&](const uint8_t *p, int width, int u) {
    u32x4 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4 *)(p + (32 * u + 4 * h) * (2 * width)));
      const uint2 w = __builtin_bit_cast(uint2, t);
      v[2 * h] = w.x;
      v[2 * h + 1] = w.y;
    }
    return v;
  };
  struct Frags {
    u32x4 a[C::MB], b[C::NB];
  };
  auto read = [&](int s, int u, Frags &f) {
    const uint8_t *st = smem + (s % C::ST) * C::STAGE;
#pragma unroll
    for (int j = 0; j < C::NB; ++j) {
      if constexpr (C::BF == kCols)
        f.b[j] = cols_frag(st + b_at[j], C::BN, u);
      else
        f.b[j] = *(const u32x4 *)(st + b_at[u] + j * (C::BF == kRows ? 16 * C::KB : 1024 * C::SUB));
    }
#pragma unroll
    for (int i = 0; i < C::MB; ++i) {
      if constexpr (C::AF == kCols)
        f.a[i] = cols_frag(st + a_at[i], C::BM, u);
      else
        f.a[i] = *(const u32x4 *)(st + a_at[u] + i * 16 * C::KB);
    }
  };

  Acc acc[C::MB][C::NB];
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int j = 0; j < C::NB; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  auto multiply = [&](const Frags &f) {
#pragma unroll
    for (int i = 0; i < C::MB; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) {
        if constexpr (C::I8)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, f.b[j]),
                                                            __builtin_bit_cast(i32x4, f.a[i]), acc[i][j], 0, 0, 0);
        else
          acc[i][j] = mfma_bf16(f.b[j], f.a[i], acc[i][j]);
      }
  };
  // one LDS read, then its share of the products, and so on
  auto interleave = [&] {
    constexpr int READS = C::NB * (C::BF == kCols ? 2 : 1) + C::MB * (C::AF == kCols ? 2 : 1);
    constexpr int MULS = C::NB * C::MB, PER = MULS / READS > 0 ? MULS / READS : 1;
#pragma unroll
    for (int r = 0; r < READS; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    }
    if constexpr (MULS > READS * PER) __builtin_amdgcn_sched_group_barrier(0x008, MULS - READS * PER, 0);
  };

  // While one half of a stage multiplies, the fragments of the next half are
  // read, so no product waits for LDS.  A stage's buffer is free once the
  // fragments of its second half are in registers; stage s + ST follows into it.
#pragma unroll
  for (int s = 0; s < C::ST; ++s)
    if (first + s < steps) issue(first + s);
  wait_loads<C::LOADS>(min(C::ST - 1, steps - 1 - first));
  mm_barrier();  // the first stage is in LDS for every wave
  Frags f[2];
  read(first, 0, f[0]);
  for (int s = first; s + 1 < steps; ++s) {
    read(s, 1, f[1]);
    multiply(f[0]);
    interleave();
    // stages s + 2 .. s + ST - 1 may still be out
    wait_loads<C::LOADS>(min(C::ST - 2, steps - 2 - s));
    mm_barrier();  // stage s + 1 is in LDS, stage s free
    if (s + C::ST < steps) issue(s + C::ST);
    read(s + 1, 0, f[0]);
    multiply(f[1]);
    interleave();
  }
  read(steps - 1, 1, f[1]);
  multiply(f[0]);
  multiply(f[1]);

  if constexpr (C::SPLIT && C::EPI != kParts) {
    if (a.splits > 1) {
      // Publish this part of k (agent-scope stores, complete before the counter
      // moves); the last workgroup of the tile adds the parts in their order,
      // its own from memory like the others, and leaves the counter at zero.
      const int tile = tm * n_tiles + tn;
      constexpr int WORDS = C::MB * C::NB * 2 * C::THREADS;  // 8-byte words of a tile
      auto at = [&](int p) {
        return a.partials + ((int64_t)p * m_tiles * n_tiles + tile) * WORDS + threadIdx.x;
      };
      uint64_t *mine = at(split);
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) {
          const u32x4 w = __builtin_bit_cast(u32x4, acc[i][j]);
          uint64_t *d = mine + (i * C::NB + j) * 2 * C::THREADS;
          __hip_atomic_store(d, w.x | ((uint64_t)w.y << 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(d + C::THREADS, w.z | ((uint64_t)w.w << 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      __builtin_amdgcn_s_waitcnt(0);
      mm_barrier();  // every wave's parts are in memory, and the ring is free
      int *last = (int *)smem;
      if (threadIdx.x == 0)
        *last = __hip_atomic_fetch_add(a.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (uint32_t)(a.splits - 1);
      __syncthreads();
      if (!*last) return;  // uniform over the workgroup
      __syncthreads();     // (the flag's place is written again below)
      if (threadIdx.x == 0) __hip_atomic_store(a.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) acc[i][j] = Acc{0, 0, 0, 0};
      // (the loads of GO parts go out together: one part's latency, not each's)
      constexpr int GO = C::MB * C::NB <= 4 ? 4 : 2;
      for (int p0 = 0; p0 < a.splits; p0 += GO) {
        uint64_t w[GO][C::MB * C::NB][2];
#pragma unroll
        for (int g = 0; g < GO; ++g) {
          const uint64_t *src = at(min(p0 + g, a.splits - 1));
#pragma unroll
          for (int b = 0; b < C::MB * C::NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[g][b][h] = __hip_atomic_load(src + (2 * b + h) * C::THREADS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int g = 0; g < GO; ++g) {
          if (p0 + g >= a.splits) continue;
#pragma unroll
          for (int b = 0; b < C::MB * C::NB; ++b) {
            const u32x4 v = {(uint32_t)w[g][b][0], (uint32_t)(w[g][b][0] >> 32), (uint32_t)w[g][b][1],
                             (uint32_t)(w[g][b][1] >> 32)};
            acc[b / C::NB][b % C::NB] += __builtin_bit_cast(Acc, v);
          }
        }
      }
    }
  }

  if constexpr (C::ROW_HALVES) {
    if (a.halves > 0) {
#pragma unroll
      for (int j = 0; j < C::NB; ++j) acc[0][j] += acc[1][j];
    }
  }
  const int m_out = C::ROW_HALVES && a.halves > 0 ? a.m - a.halves : a.m;

  // ---- epilogue: 16-row slabs through a wave-private part of the ring ----
  mm_barrier();  // the last fragments are in registers for every wave, the ring is free
  uint8_t *slab = smem + wave * C::SLAB;
  const int row_w = m0 + wm * C::MB * 16;           // first row of the wave
  const int col_w = n0 + wn * C::OUT_NB * 16;       // first output column of the wave
  if constexpr (C::EPI == kXentStats) {
    // Largest logit and sum of exp(scale (z - largest)) of every row over the wave's
    // columns, over its 4 quarters of lanes, then over the waves side by side.  (z -
    // largest) before the product with the scale: the difference is exact where it
    // counts.
    float *red = (float *)smem;  // [WN][BM][2]
    const float base2 = a.scale * 1.4426950408889634f;
    const bool edge = col_w + 16 * C::NB > a.n;
#pragma unroll
    for (int i = 0; i < C::MB; ++i) {
      if (edge) {
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col_w + 16 * j + 4 * q + e >= a.n) acc[i][j][e] = -INFINITY;
      }
      float most = -INFINITY;
#pragma unroll
      for (int j = 0; j < C::NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) most = fmaxf(most, acc[i][j][e]);
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      const float from = most == -INFINITY ? 0.f : most;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < C::NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f((acc[i][j][e] - from) * base2);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (q == 0) *(float2 *)(red + 2 * ((wn * C::BM) + (wm * C::MB + i) * 16 + r16)) = float2{most, sum};
      const int row = row_w + 16 * i + r16;
      const int at = row < a.m && a.targets ? a.targets[row] - a.first_token - col_w : -1;
      if (__any(at >= 0 && at < 16 * C::NB)) {
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at == 16 * j + 4 * q + e && col_w + at < a.n) a.at_target[row] = acc[i][j][e];
      }
    }
    mm_barrier();
    for (int r = threadIdx.x; r < rows; r += C::THREADS) {
      float2 v[C::WN];
      float most = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < C::WN; ++w) {
        v[w] = *(const float2 *)(red + 2 * (w * C::BM + r));
        most = fmaxf(most, v[w].x);
      }
      const float from = most == -INFINITY ? 0.f : most;
#pragma unroll
      for (int w = 0; w < C::WN; ++w) sum += v[w].y * __builtin_amdgcn_exp2f((v[w].x - from) * base2);
      *(float2 *)(a.stats + 2 * ((int64_t)tn * a.m + m0 + r)) = float2{most, sum};
    }
    return;
  }
  // columns that are stored (the gradient of the logits is padded with zeros to
  // whole 16-byte units: the products that read it take units whole)
  const int n_out = C::EPI == kXentGrad ? (a.n + 7) & ~7 : a.n;
  // kXentGrad: per row its weight, the logarithm (base 2) of its sum and its target
  float *row_info = (float *)(smem + C::WAVES * C::SLAB);  // [BM][4]
  if constexpr (C::EPI == kXentGrad) {
    // (in the slabs' place, not in LDS of its own: 32 bytes more left one workgroup of
    // 32 x 128 on a CU instead of two; backward pass of 16 tokens, 100003 x 2048: 263 us
    // against 273)
    float *most_of = (float *)smem;
    if (lane == 0) most_of[wave] = dloss_most;
    mm_barrier();
    for (int w = 0; w < C::WAVES; ++w) dloss_most = fmaxf(dloss_most, most_of[w]);
    const float c = dloss_most >= 0x1p-126f && dloss_most < INFINITY ? dloss_most : 1.f;
    my_row[0] /= c;
    if (tm == 0 && tn == 0 && threadIdx.x == 0) a.alpha_out[0] = a.scale * c;
    if (threadIdx.x < C::BM) *(f32x4 *)(row_info + 4 * threadIdx.x) = my_row;
    mm_barrier();
  }
  float alpha = 1.f;
  if constexpr (C::EPI == kScaled) alpha = a.alpha[0];
  if constexpr (C::EPI == kParts) a.y = (float *)a.y + split * a.part_stride;
  // fp32 values of block (i, j), scales applied
  auto value = [&](int i, int j) {
    f32x4 v;
    if constexpr (C::EPI == kXentGrad) {
      const float base2 = a.scale * 1.4426950408889634f;
      const int col = col_w + 16 * j + 4 * q;
      const f32x4 info = *(const f32x4 *)(row_info + 4 * ((wm * C::MB + i) * 16 + r16));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], base2, -info[1]));
        // (a weight of 0: nothing, whatever the logits are)
        v[e] = info[0] == 0.f || col + e >= a.n ? 0.f : info[0] * (col + e == __float_as_int(info[2]) ? p - 1.f : p);
      }
      return v;
    }
    if constexpr (C::EPI == kScaled) {
      v = acc[i][j] * alpha;
      return v;
    }
    if constexpr (C::EPI == kParts) {
      v = acc[i][j];
      const int row = row_w + 16 * i + r16, col = col_w + 16 * j + 4 * q;
      if (split < a.parts_there && row < m_out && col < a.n) v += *(const f32x4 *)((const float *)a.y + row * a.ldy + col);
      return v;
    }
    if constexpr (C::I8) {
      bool up;
      int col = b_col(wn * C::NB + j, 4 * q, &up);
      const float s = a.sa[min(row_w + 16 * i + r16, a.m - 1)];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = (float)acc[i][j][e] * s * a.sb[min(col + e, a.n - 1) + (up ? a.n : 0)];
    } else {
      v = acc[i][j];
    }
    return v;
  };
  // writes slab i of `at(j)` to out columns col_w .. of a matrix whose column
  // 0 is at element `shift` of its rows; the element type is a constant, so the
  // addresses need no division and the copies unroll
  auto store_as = [&](auto f32, int i, auto &at, void *out, int64_t ld, int64_t shift) {
    constexpr bool F32 = decltype(f32)::value;
    constexpr int EL = F32 ? 4 : 2, CHUNKS = 16 * C::OUT_NB * EL / 16, PER = 16 / EL;
    constexpr int ROWS = 64 / CHUNKS > 16 ? 16 : 64 / CHUNKS;  // rows per pass of the wave
#pragma unroll
    for (int j = 0; j < C::OUT_NB; ++j) {
      const f32x4 v = at(j);
      uint8_t *p = slab + r16 * C::PITCH + (16 * j + 4 * q) * EL;
      if constexpr (F32)
        *(f32x4 *)p = v;
      else
        *(uint2 *)p = uint2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own writes, before its reads
    const int c = (lane % CHUNKS) * PER, col = col_w + c;
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += ROWS) {
      const int rr = r0 + lane / CHUNKS, row = row_w + 16 * i + rr;
      if (lane >= ROWS * CHUNKS || row >= m_out || col >= n_out) continue;
      const u32x4 v = *(const u32x4 *)(slab + rr * C::PITCH + c * EL);
      uint8_t *dst = (uint8_t *)out + (row * ld + shift + col) * EL;
      if (col + PER <= n_out) {
        // (a weight gradient, of any size, is read once, much later: past the caches.
        // Backward us through / past them, gradients in turn that no cache holds: 257
        // tokens of 2817 x 1032 35.4 / 33.4 (11.6 MB bf16) and 37.0 / 35.3 (fp32), one
        // of 4096 x 4096 44.1 / 43.0 and 62.9 / 58.0, of 14336 x 4096 126 / 106 and 171
        // / 143; 257 of 4096 x 4096 75.6 / 76.6 and 86.3 / 89.9.  The forward's
        // outputs, read next, lose: 790 -> 810 us at 4096 tokens)
        if constexpr (C::AF == kCols)
          __builtin_nontemporal_store(v, (u32x4_any *)dst);
        else
          *(u32x4_any *)dst = v;
      } else {
#pragma unroll
        for (int b = 0; b < PER; ++b) {
          if (b >= a.n - col) continue;
          if constexpr (F32)
            ((uint32_t *)dst)[b] = v[b];
          else
            ((uint16_t *)dst)[b] = (uint16_t)(v[b >> 1] >> (16 * (b & 1)));
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads, before the slab's next writes
  };
  auto store = [&](int i, auto &&at, void *out, int64_t ld, int otype, int64_t shift) {
    if (otype == QG_O_F32)
      store_as(std::true_type{}, i, at, out, ld, shift);
    else
      store_as(std::false_type{}, i, at, out, ld, shift);
  };
#pragma unroll
  for (int i = 0; i < C::MB; ++i) {
    if constexpr (C::GATED) {
      constexpr int H = C::NB / 2;
      if (a.gu) {
        store(i, [&](int j) { return value(i, j); }, a.gu, a.ldgu, a.gu_type, 0);
        store(i, [&](int j) { return value(i, H + j); }, a.gu, a.ldgu, a.gu_type, a.n);
      }
      if (a.y)
        store(i,
              [&](int j) {
                const f32x4 g = value(i, j), u = value(i, H + j);
                f32x4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = act_value(g[e], a.act) * u[e];
                return h;
              },
              a.y, a.ldy, a.otype, 0);
    } else {
      store(i, [&](int j) { return value(i, j); }, a.y, a.ldy, a.otype, 0);
      if constexpr (C::EPI == kXentGrad && C::BM == 32) {
        if (a.halves > 0)  // what the rounding left
          store(i,
                [&](int j) {
                  f32x4 v = value(i, j);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float rest = v[e] - bf16_bits_to_f32(bf16_rne(v[e]));
                    v[e] = fabsf(v[e]) <= 3.3e38f ? rest : 0.f;  // (nothing of an infinity or a NaN)
                  }
                  return v;
                },
                (uint16_t *)a.y + a.halves * a.ldy, a.ldy, a.otype, 0);
      }
    }
  }
}

// What a tile shape and a split of k would cost, in clocks of the busiest CU:
// its workgroups' stages (matrix or LDS time, which workgroups of a CU share, or
// one stage's latency where they are few) beside the operands' way from memory,
// each workgroup's start and end, and the sum over the parts.  The latencies,
// the fixed parts and the factor 1.7 over the matrix instructions' own time are
// measured.  What the shapes are for: 256 x 256 where its tiles fill the CUs; 192
// rows where a batch is little more than a whole number of them (gated int8,
// 322 rows of 14004 x 2528: 39.5 us, 50 in 128 x 128, 42 in 256 x 256); 128 x 128,
// with two stages two workgroups share a CU, with four one has more in flight;
// 64 and 32 rows for small batches (bf16, 128 rows of 2816 x 1024: 10.0 and 8.7
// us).  Workgroups are counted per XCD, where all parts of a tile run (28
// tiles in 9 parts, 36 on some XCDs' 32 CUs, took 36 us, in 8 parts 29).
struct MmPlan {
  int splits = 1, per = 0;
  double cost = 0;
};
// Workgroups of a shape that a CU holds (the kernels have no LDS but what the launch
// asks for).
template <class C>
constexpr int64_t kMmResident = 160 * 1024 / C::LDS;
constexpr int64_t kMmMostSplits = 32;
// Parts without a join in the kernel (kParts) cost their way to memory and back, by
// all CUs, and a launch.
template <class C>
static MmPlan mm_plan(int64_t m, int64_t n, int64_t kd, uint64_t budget) {
  constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;
  const int64_t m_tiles = (m + C::BM - 1) / C::BM, n_tiles = (n + OUT_BN - 1) / OUT_BN, tiles = m_tiles * n_tiles;
  const int64_t steps = (kd + C::KE - 1) / C::KE;
  constexpr int64_t mfma = (int64_t)C::BM * C::BN * C::KE / (C::I8 ? 4096 : 2048) * 17 / 10;
  constexpr int64_t lds = (C::WAVES * (C::MB + C::NB) * 16 * C::KB + C::STAGE) / 128 * 21 / 20;
  // (kParts: what one operand with k across its rows takes, measured in long
  // contractions: 256 x 256 5070 clocks a stage, 128 x 128 1760)
  constexpr int64_t matrix = (mfma > lds ? mfma : lds) * (C::EPI != kParts ? 10 : C::BM > 128 ? 14 : 16) / 10;
  constexpr int64_t latency = C::BM <= 64 ? 700 : C::ST == 2 ? 1170 : 900;
  constexpr int64_t resident = kMmResident<C>;
  constexpr int64_t partial = (int64_t)C::BM * C::BN * 4;
  const double memory = (double)(m + (C::GATED ? 2 * n : n)) * kd * C::EL / 2100;
  MmPlan best;
  const bool parts = C::EPI == kParts;
  const int64_t most = parts ? (int64_t)(budget / (uint64_t)(4 * m * n))
                       : C::SPLIT && tiles <= kMaxSplitCounters ? (int64_t)(budget / (uint64_t)(partial * tiles)) : 1;
  for (int64_t want = 1; want <= std::min<int64_t>(std::min<int64_t>(std::max<int64_t>(most, 1), steps), kMmMostSplits); ++want) {
    const int64_t per = (steps + want - 1) / want, splits = (steps + per - 1) / per;
    if (splits != want) continue;  // the same as a smaller number of parts
    const int64_t wgs = ((tiles + kXcds - 1) / kXcds * splits + 31) / 32, rounds = (wgs + resident - 1) / resident;
    if (splits > 1 && rounds > 1) break;  // (more parts than places: slower than fewer)
    const double stages = (double)per * std::max(wgs * matrix, rounds * latency);
    double cost = std::sqrt(stages * stages + memory * memory) + 4000. * wgs;
    if (parts)
      cost += splits > 1 ? 8000 + (double)splits * m * n * 8 / 2100 : 0;
    else if (splits > 1)
      cost += 6000 + splits * partial / 24;
    if (best.per == 0 || cost < best.cost) best = MmPlan{(int)splits, (int)per, cost};
  }
  return best;
}

template <class C>
static uint64_t mm_partial_bytes(int64_t m, int64_t n, const MmPlan &p) {
  constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;
  if (C::EPI == kParts) return p.splits > 1 ? (uint64_t)p.splits * m * n * 4 : 0;
  return p.splits > 1 ? (uint64_t)p.splits * ((m + C::BM - 1) / C::BM) * ((n + OUT_BN - 1) / OUT_BN) * C::BM * C::BN * 4
                      : 0;
}

// The most that mm_partial_bytes comes to for up to m x n outputs and contractions of
// up to kd, whichever of the shapes is taken: parts times tiles are at most the
// places on all CUs.
template <class C0, class... Cs>
static uint64_t mm_most_partial_bytes(int64_t m, int64_t n, int64_t kd, uint64_t budget) {
  auto one = [&](auto *cfg) -> uint64_t {
    using C = std::remove_pointer_t<decltype(cfg)>;
    constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;
    const int64_t steps = (kd + C::KE - 1) / C::KE, tiles = ((m + C::BM - 1) / C::BM) * ((n + OUT_BN - 1) / OUT_BN);
    if (!C::SPLIT || steps < 2) return 0;
    const int64_t places = 256 * kMmResident<C>, most = std::min(steps, kMmMostSplits);
    return std::min<uint64_t>((uint64_t)std::min(tiles * most, places) * C::BM * C::BN * 4, budget);
  };
  uint64_t most = one((C0 *)nullptr);
  ((most = std::max(most, one((Cs *)nullptr))), ...);
  return most;
}

template <class C>
static hipError_t launch_mm(const typename C::Args &args, const MmPlan &p, hipStream_t s) {
  constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;
  typename C::Args a = args;
  a.splits = p.splits;
  a.per = p.per;
  if (p.splits > 1 && C::EPI != kParts && (!a.counters || !a.partials)) return hipErrorInvalidValue;
  const int64_t total = (int64_t)((a.m + C::BM - 1) / C::BM) * ((a.n + OUT_BN - 1) / OUT_BN);
  const int64_t grid = (total + kXcds - 1) / kXcds * kXcds * p.splits;
  auto kern = mm_kernel<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(C::THREADS), C::LDS, s, a);
  return hipGetLastError();
}

// Whether the 32-bit offsets of the copies, from the 64-bit base of a tile and a
// stage, reach all of a stage's rows at these pitches.
template <class C>
static bool mm_reaches(const MmArgs &a) {
  constexpr int OUT_BN = C::GATED ? C::BN / 2 : C::BN;
  const int64_t far_a = (C::AF == kRows ? C::BM - 1 : C::KE - 1) * a.lda + (C::AF == kRows ? C::KB : 2 * C::BM);
  const int64_t far_b = C::BF == kRows   ? (OUT_BN - 1) * a.ldb + C::KB
                        : C::BF == kCols ? (C::KE - 1) * a.ldb + 2 * C::BN
                                         : (int64_t)(OUT_BN / 16 + 1) * a.ldb;
  return far_a <= (1ll << 32) && far_b <= (1ll << 32);
}

// The cheapest of the compiled shapes that reach their operands' rows: launches
// it, or (info; the pitches count here too) only says which it is and what
// partial tiles it needs.
template <class C0, class... Cs>
static hipError_t mm_dispatch(const typename C0::Args &a, uint64_t budget, hipStream_t s, MmInfo *info) {
  const MmPlan plans[] = {mm_plan<C0>(a.m, a.n, a.kd, budget), mm_plan<Cs>(a.m, a.n, a.kd, budget)...};
  const bool reach[] = {mm_reaches<C0>(a), mm_reaches<Cs>(a)...};
  int best = -1;
  for (int i = 0; i <= (int)sizeof...(Cs); ++i)
    if (reach[i] && (best < 0 || plans[i].cost < plans[best].cost)) best = i;
  int i = 0;
  hipError_t e = hipErrorInvalidValue;
  auto one = [&](auto *cfg) {
    using C = std::remove_pointer_t<decltype(cfg)>;
    if (i++ != best) return;
    if (info) {
      *info = MmInfo{mm_partial_bytes<C>(a.m, a.n, plans[best]), C::BM, C::BN, plans[best].splits, C::ST};
      e = hipSuccess;
    } else {
      e = launch_mm<C>(a, plans[best], s);
    }
  };
  one((C0 *)nullptr);
  (one((Cs *)nullptr), ...);
  return e;
}

// The compiled shapes of one product.
template <class... Cs>
struct MmShapes {
  template <class Args>
  static hipError_t dispatch(const Args &a, uint64_t budget, hipStream_t s, MmInfo *info) {
    return mm_dispatch<Cs...>(a, budget, s, info);
  }
  static uint64_t most_bytes(int64_t m, int64_t n, int64_t kd, uint64_t budget) {
    return mm_most_partial_bytes<Cs...>(m, n, kd, budget);
  }
  static constexpr int narrowest = std::min({Cs::BN...});  // columns of a tile
};

}  // namespace qg
