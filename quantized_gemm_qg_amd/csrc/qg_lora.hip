// Low-rank adapters of many requests added to the output of a shared projection:
//   y[r] += scale_a (x[r] A_a^T) B_a^T   for the rows r of adapter a,
// A_a [rank][k], B_a [n][rank], rows grouped by adapter (qg_moe_sort's lists).
// Two launches: the first leaves t = x A^T of every listed row in fp32 (k in parts
// where there are few rows), the second adds scale t B^T; the smallest calls are one
// launch.  Both work on items of up to 16 (second: 16, 32 or 64) rows of one adapter;
// a workgroup finds its item from the offsets by itself, so nothing is planned on the
// host and no list is written.
// t goes into the second product as a sum of bf16 numbers, two for a bf16 y (2^-16
// of t is left, against 2^-8 of y's own rounding), three for an fp32 y (2^-24): the
// parts stand side by side along the contraction, so a rank of 16 in two parts is
// one matrix instruction, as one part would be.
// Bound by bytes: the adapters in use once, x, and y read and written.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"
#include "qg_quant.h"

namespace qg {

namespace {

struct LoraItem {
  int adapter;  // < 0: none
  int pos, rows;  // sorted positions pos .. pos + rows - 1
};

// Item `item` of the list that has, adapter by adapter, one for every ROWS of its
// positions (or what is left of them).  Every wave finds it for itself: a lane takes
// `per` adapters, a scan over the lanes gives the first item of each.  Offsets out
// of 0 .. m or falling count as empty.
template <int ROWS>
__device__ __forceinline__ LoraItem lora_item(const LoraArgs &a, int item) {
  const int lane = threadIdx.x & 63;
  const int per = (a.adapters + 63) / 64, first = lane * per, last = min(first + per, a.adapters);
  auto span = [&](int e, int *begin) {
    *begin = min(max(a.offsets[e], 0), a.m);
    return max(min(a.offsets[e + 1], a.m) - *begin, 0);
  };
  int mine = 0, begin = 0, count = 0;
  for (int e = first; e < last; ++e) {
    count = span(e, &begin);
    mine += (count + ROWS - 1) / ROWS;
  }
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off);
    if (lane >= off) upto += o;
  }
  const uint64_t behind = __ballot(upto > item);
  if (behind == 0) return LoraItem{-1, 0, 0};
  const int owner = __ffsll((unsigned long long)behind) - 1;
  int at = item - (upto - mine), e = first;
  if (per > 1 && lane == owner)  // (with one adapter per lane its offsets are at hand)
    for (; e + 1 < last; ++e) {
      count = span(e, &begin);
      const int items = (count + ROWS - 1) / ROWS;
      if (at < items) break;
      at -= items;
      count = span(e + 1, &begin);
    }
  return LoraItem{__builtin_amdgcn_readlane(e, owner), __builtin_amdgcn_readlane(begin + at * ROWS, owner),
                  __builtin_amdgcn_readlane(min(ROWS, count - at * ROWS), owner)};
}

// acc = x A^T of an item's 16 rows over stages begin .. end - 1 of 64 k, by one wave.
// The operand layout of the matrix instruction has neighbouring lanes in different
// rows, which the memory path takes at 16 bytes per clock and CU (51 with four lanes
// to 64 bytes of a row; L1 hits, 4 waves per SIMD), and every workgroup reads its
// whole adapter: so whole cache lines go to a ring of ST stages in LDS (16-byte chunks
// of a row at slot chunk ^ row % 8), one ring per wave, without barriers.
template <int NB, int ST>
__device__ __forceinline__ void lora_low_rank(const LoraArgs &a, const LoraItem &it, int begin, int end,
                                              const uint8_t *mine, f32x4 (&acc)[NB]) {
  constexpr int COPIES = 2 * (1 + NB), STAGE = COPIES * 1024;
  const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15;
  // a copy: 8 rows of 128 bytes, this lane's 16 of row 8 c + lane / 8
  const int chunk = (lane & 7) ^ ((lane >> 3) & 7);
  const uint8_t *src[COPIES];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int row = a.sorted[it.pos + min(8 * c + (lane >> 3), it.rows - 1)];
    src[c] = (const uint8_t *)(a.x + (row >= 0 && row < a.m ? row : 0) * a.ldx) + 16 * chunk;
  }
#pragma unroll
  for (int c = 2; c < COPIES; ++c)
    src[c] = (const uint8_t *)(a.a + ((int64_t)it.adapter * a.rank + min(8 * (c - 2) + (lane >> 3), a.rank - 1)) * a.lda) +
             16 * chunk;
  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)mine;
  auto issue = [&](int s) {
    const uint32_t st = ring + (s - begin) % ST * STAGE;
    const bool in = 64 * s + 8 * chunk < a.k;  // (behind k: zeros)
#pragma unroll
    for (int c = 0; c < COPIES; ++c)
      mm_copy16_at(in ? src[c] + 128 * (int64_t)s : (const uint8_t *)mm_zeros, st + c * 1024);
  };
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < ST - 1; ++s)
    if (begin + s < end) issue(begin + s);
  for (int s = begin; s < end; ++s) {
    // (into the stage that was read last time: its reads are in registers)
    if (s + ST - 1 < end) issue(s + ST - 1);
    // stage s is there when at most the later ones are out
    static_assert(ST >= 2 && ST <= 4 && (ST - 1) * COPIES < 64, "outstanding loads");
    const int out = min(ST - 1, end - 1 - s);
    if (ST == 4 && out == 3)
      QG_WAIT_VMCNT(ST == 4 ? 3 * COPIES : 0);
    else if (ST >= 3 && out == 2)
      QG_WAIT_VMCNT(ST >= 3 ? 2 * COPIES : 0);
    else if (out >= 1)
      QG_WAIT_VMCNT(COPIES);
    else
      QG_WAIT_VMCNT(0);
    asm volatile("" ::: "memory");
    const uint8_t *st = mine + (s - begin) % ST * STAGE;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = r16 * 128 + 16 * ((4 * u + q) ^ (r16 & 7));
      const u32x4 xv = *(const u32x4 *)(st + at);
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] = mfma_bf16(*(const u32x4 *)(st + 2048 * (1 + j) + at), xv, acc[j]);
    }
    QG_WAIT_LGKMCNT0();
    asm volatile("" ::: "memory");
  }
}

// The second product of one workgroup: 16 RB rows, 64 columns per wave and chunk.
// The parts of scale t stand in LDS as units of 8 along the contraction, [unit][row].
// SD x 32 of the rank are in registers at a time, used for every part in turn; ranks
// of 8 and 16 have their parts side by side in one step.  y is loaded and stored along
// its rows, 16 bytes per lane (the sums go through LDS for that).
template <int RB, int SD, bool F32>
struct LoraColumns {
  static constexpr int ROWS = 16 * RB, PARTS = F32 ? 3 : 2, EL = F32 ? 4 : 2;
  // columns per lane, lanes per row, rows per pass, passes
  static constexpr int VC = 16 / EL, LPR = 64 / VC, RPP = 64 / LPR, PASSES = 16 / RPP;
  static constexpr int UNIT = ROWS + 1;        // 16-byte rows of a unit (one more: banks)
  static constexpr int PITCH = 64 * 4 + 16;    // bytes of a row of the sums
  typedef u32x4 Rows[RB][PASSES];

  const LoraArgs &a;
  const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15, ycol = lane % LPR * VC;
  const int units, groups, pitch, lds_steps;  // pitch: units of a part
  const bool side;                            // parts side by side
  u32x4 *parts;                               // [lds_steps * pitch][UNIT]
  uint8_t *slab;                              // the wave's 16 rows of sums
  const uint8_t *bbase;
  int row[RB][PASSES];                        // this lane's row in each pass of each 16 rows, or -1
  u32x4 bv[SD][4];

  __device__ __forceinline__ LoraColumns(const LoraArgs &args, const LoraItem &it, uint8_t *lds, int wave)
      : a(args),
        units(args.rank / 8),
        groups((units + 4 * SD - 1) / (4 * SD)),
        pitch(units <= 2 ? 4 : groups * 4 * SD),
        lds_steps(units <= 2 ? (PARTS * units + 3) / 4 : PARTS),
        side(units <= 2),
        parts((u32x4 *)lds),
        slab(lds + lds_steps * pitch * UNIT * 16 + wave * 16 * PITCH),
        bbase((const uint8_t *)(args.b + (int64_t)it.adapter * args.n * args.ldb)) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int at = 16 * i + p * RPP + lane / LPR, r = a.sorted[it.pos + min(at, it.rows - 1)];
        row[i][p] = at < it.rows && r >= 0 && r < a.m ? r : -1;
      }
  }
  __device__ __forceinline__ void load_b(int col0, int group) {
    const uint8_t *p = bbase + (int64_t)col0 * a.ldb * 2;
    uint32_t boff[4];  // (64 rows of B span less than 4 GiB; columns behind the last one bring it)
#pragma unroll
    for (int j = 0; j < 4; ++j) boff[j] = (uint32_t)(min(16 * j + r16, a.n - 1 - col0) * a.ldb * 2);
#pragma unroll
    for (int d = 0; d < SD; ++d) {
      const int unit = side ? q % units : 4 * (group * SD + d) + q;
      const uint32_t at = 16 * min(unit, units - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bv[d][j] = *(const u32x4 *)(p + (boff[j] + at));
        if (unit >= units) bv[d][j] = u32x4{0u, 0u, 0u, 0u};
      }
    }
  }
  __device__ __forceinline__ uint8_t *y_at(int i, int p, int col0) const {
    return (uint8_t *)a.y + (max(row[i][p], 0) * a.ldy + col0 + ycol) * EL;
  }
  __device__ __forceinline__ bool whole(int col0) const { return a.y_vectors && col0 + 64 <= a.n; }
  // (rows that are not on 16 bytes, and the last columns: element by element, all of
  // them asked for before the first is stored)
  __device__ __forceinline__ void load_y(int col0, Rows &yv) const {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const uint8_t *src = y_at(i, p, col0);
        if (whole(col0)) {
          yv[i][p] = *(const u32x4 *)src;
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          auto at = [&](int c) -> uint32_t {
            if (col0 + ycol + c >= a.n) return 0;
            return F32 ? ((const uint32_t *)src)[c] : ((const uint16_t *)src)[c];
          };
          yv[i][p][e] = F32 ? at(e) : at(2 * e) | at(2 * e + 1) << 16;
        }
      }
  }
  // the parts of 8 values of row r (scaled)
  __device__ __forceinline__ void put(int r, int unit, float (&v)[8]) const {
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
      parts[(part * (side ? units : pitch) + unit) * UNIT + r] = w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // what the part left (nothing of an infinity or a NaN)
        const float f = __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        v[e] = fabsf(f) <= 3.4e38f ? v[e] - f : 0.f;
      }
    }
  }
  // zeros in the units that no part fills
  __device__ __forceinline__ void put_zeros() const {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    if (side) {
      for (int u = PARTS * units * UNIT + threadIdx.x; u < lds_steps * 4 * UNIT; u += blockDim.x) parts[u] = zero;
    } else {
      for (int u = threadIdx.x; u < PARTS * (pitch - units) * ROWS; u += blockDim.x) {
        const int r = u % ROWS, unit = u / ROWS;
        parts[(unit / (pitch - units) * pitch + units + unit % (pitch - units)) * UNIT + r] = zero;
      }
    }
  }
  // y of columns col0 .. col0 + 63 (a whole wave; col0 < n) from the parts, bv (col0's
  // first group) and yv; next >= 0: asks for the operands of those columns
  __device__ __forceinline__ void columns(int col0, int next, Rows &yv) {
    Rows later;
    if (next >= 0) load_y(next, later);
    f32x4 acc[RB][4];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int group = 0; group < groups; ++group) {
      if (group > 0) load_b(col0, group);
      for (int st = 0; st < lds_steps; ++st)
#pragma unroll
        for (int d = 0; d < SD; ++d)
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            const u32x4 tv = parts[(st * pitch + 4 * (group * SD + d) + q) * UNIT + 16 * i + r16];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(bv[d][j], tv, acc[i][j]);
          }
    }
    if (next >= 0) load_b(next, 0);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4 *)(slab + r16 * PITCH + (16 * j + 4 * q) * 4) = acc[i][j];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own writes, before its reads
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const f32x4 *sum = (const f32x4 *)(slab + (p * RPP + lane / LPR) * PITCH + ycol * 4);
        float d[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) d[e] = sum[e / 4][e % 4];
        if (row[i][p] < 0) continue;
        uint8_t *dst = y_at(i, p, col0);
        u32x4 w = yv[i][p];
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + d[e]);
        } else {
          float v[8];
          unpack8(w, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = bf16_pair(v[2 * e] + d[2 * e], v[2 * e + 1] + d[2 * e + 1]);
        }
        if (whole(col0)) {
          *(u32x4 *)dst = w;
          continue;
        }
#pragma unroll
        for (int e = 0; e < VC; ++e) {
          if (col0 + ycol + e >= a.n) continue;
          if constexpr (F32)
            ((uint32_t *)dst)[e] = w[e];
          else
            ((uint16_t *)dst)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads, before the slab's next writes
    }
    if (next >= 0) {
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int p = 0; p < PASSES; ++p) yv[i][p] = later[i][p];
    }
  }
};

}  // namespace

// t[split][position][rank] = x A^T over the split's part of k, for an item of 16
// rows: KW waves share the part of k and join in LDS.  4096 rows, rank 64, k 4096: 16
// us (operands straight to registers 24), 44 rows of 35 adapters of rank 16: 4.1 us
// (6.2).
template <int NB, int KW, int ST>
__global__ __launch_bounds__(64 * KW) void lora_down_kernel(LoraArgs a) {
  constexpr int RING = ST * 2 * (1 + NB) * 1024;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const LoraItem it = lora_item<16>(a, blockIdx.x);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  // stages of 64 k: of the split, then of the wave
  const int steps = (a.k + 63) / 64, per_split = (steps + a.splits - 1) / a.splits;
  const int s0 = min((int)blockIdx.y * per_split, steps), s1 = min(s0 + per_split, steps);
  const int per_wave = (s1 - s0 + KW - 1) / KW;
  const int begin = min(s0 + kw * per_wave, s1), end = min(begin + per_wave, s1);
  f32x4 acc[NB];
  lora_low_rank<NB, ST>(a, it, begin, end, smem + kw * RING, acc);
  f32x4 *join = (f32x4 *)smem;
  __syncthreads();  // every wave is done with its ring
  if (kw > 0) {
#pragma unroll
    for (int j = 0; j < NB; ++j) join[((kw - 1) * NB + j) * 64 + lane] = acc[j];
  }
  __syncthreads();
  if (kw > 0 || r16 >= it.rows) return;
#pragma unroll
  for (int o = 0; o < KW - 1; ++o)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[j] += join[(o * NB + j) * 64 + lane];
  float *t = a.t + ((int64_t)blockIdx.y * a.m + it.pos + r16) * a.rank;
#pragma unroll
  for (int j = 0; j < NB; ++j)
    if (16 * j + 4 * q < a.rank) *(f32x4 *)(t + 16 * j + 4 * q) = acc[j];
}

// y += scale t B^T for one item and `chunks` times 256 columns, a stride apart so that
// workgroups side by side work on neighbouring columns.  4096 rows of 14336 bf16
// outputs, rank 64: 55 us, 4.3 TB/s of y (90 with y in the operand's layout, rows of
// neighbouring lanes 28 KB apart); 333 fp32 rows of 8187: 9.2 us.
template <int RB, int SD, bool F32>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  typedef LoraColumns<RB, SD, F32> Columns;
  const LoraItem it = lora_item<Columns::ROWS>(a, blockIdx.y);
  if (it.adapter < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Columns c(a, it, smem, wave);
  typename Columns::Rows yv;
  const int first_col = blockIdx.x * 256 + 64 * wave, stride = gridDim.x * 256;
  if (first_col < a.n) {
    c.load_b(first_col, 0);
    c.load_y(first_col, yv);
  }

  const float scale = a.scales ? a.scales[it.adapter] : 1.f;
  for (int u = threadIdx.x; u < c.units * Columns::ROWS; u += 256) {
    const int r = u / c.units, unit = u % c.units;
    const float *t = a.t + ((int64_t)it.pos + min(r, it.rows - 1)) * a.rank + 8 * unit;
    f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    for (int s0 = 0; s0 < a.splits; s0 += 4) {  // (the loads of four parts go out together)
      f32x4 w[4][2];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 *p = (const f32x4 *)(t + (int64_t)min(s0 + g, a.splits - 1) * a.m * a.rank);
        w[g][0] = p[0];
        w[g][1] = p[1];
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (s0 + g >= a.splits) continue;
        v0 += w[g][0];
        v1 += w[g][1];
      }
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * scale;
    c.put(r, unit, v);
  }
  c.put_zeros();
  __syncthreads();
  for (int chunk = 0; chunk < a.chunks; ++chunk) {
    const int col0 = first_col + stride * chunk;
    if (col0 >= a.n) break;  // (whole waves: the matrix instructions take every lane)
    c.columns(col0, chunk + 1 < a.chunks && col0 + stride < a.n ? col0 + stride : -1, yv);
  }
}

// Both products in one launch, for the smallest calls: every workgroup computes t of
// its item for itself (8 waves share k), then 512 columns of y.
template <int NB, int ST, bool F32>
__global__ __launch_bounds__(512) void lora_small_kernel(LoraArgs a) {
  constexpr int RING = ST * 2 * (1 + NB) * 1024;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  typedef LoraColumns<1, (NB + 1) / 2, F32> Columns;
  const LoraItem it = lora_item<16>(a, blockIdx.y);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Columns c(a, it, smem + 8 * NB * 1024, wave);
  typename Columns::Rows yv;
  const int col0 = blockIdx.x * 512 + 64 * wave;
  if (col0 < a.n) {
    c.load_b(col0, 0);
    c.load_y(col0, yv);
  }
  const float scale = a.scales ? a.scales[it.adapter] : 1.f;
  const int steps = (a.k + 63) / 64, per_wave = (steps + 7) / 8;
  const int begin = min(wave * per_wave, steps), end = min(begin + per_wave, steps);
  f32x4 acc[NB];
  lora_low_rank<NB, ST>(a, it, begin, end, smem + wave * RING, acc);
  __syncthreads();  // every wave is done with its ring
  f32x4 *join = (f32x4 *)smem;  // [wave][16 columns][lane]
#pragma unroll
  for (int j = 0; j < NB; ++j) join[(wave * NB + j) * 64 + lane] = acc[j];
  __syncthreads();
  for (int u = threadIdx.x; u < c.units * 16; u += 512) {
    const int r = u % 16, unit = u / 16;  // columns 8 unit ..: two lanes' four of block unit / 2
    const f32x4 *p = join + unit / 2 * 64 + unit % 2 * 32 + r;
    f32x4 v0 = p[0], v1 = p[16];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      v0 += p[w * NB * 64];
      v1 += p[w * NB * 64 + 16];
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * scale;
    c.put(r, unit, v);
  }
  c.put_zeros();
  __syncthreads();
  if (col0 < a.n) c.columns(col0, -1, yv);
}

template <int V>
using Int = std::integral_constant<int, V>;

// Items at most: one per adapter with rows, and one more for every `rows` rows.
static int64_t lora_items(int64_t m, int adapters, int rows) { return std::min<int64_t>(adapters, m) + m / rows; }

// Parts of k: workgroups for the CUs, of about 8 stages of 64 or more (the last one has
// what is left).
static int64_t lora_most_splits(int64_t k) { return std::min<int64_t>((k + 511) / 512, 16); }
static int lora_splits(int64_t m, int64_t k, int adapters) {
  return (int)std::min(std::max<int64_t>(256 / lora_items(m, adapters, 16), 1), lora_most_splits(k));
}
// Parts times rows of any call of up to m rows: s > 1 parts of r rows have s items <=
// 256 and r < 16 items, so s r < 4096.
int64_t lora_most_rows(int64_t m, int64_t k) {
  return std::max(m, std::min<int64_t>(lora_most_splits(k) * m, 4096));
}

// Calls of one launch: a round of workgroups, each of which reads all of A for
// itself.  us a call one after another in one / in two launches (and of a program
// that makes the calls): k 4096, one row, n 4096, rank 16 6.5 / 7.6 (7.7 / 10.3), 16
// rows of 8 adapters, n 14336, rank 16 7.5 / 8.3 (8.0 / 10.1), 4 rows, rank 32 8.2 /
// 8.4 (8.1 / 10.1), rank 64 10.5 / 9.4; k 14336, rank 16 11.6 / 9.1; 64 rows, k 1024
// 5.1 / 7.3.
static bool lora_small(int64_t m, int64_t k, int64_t n, int adapters, int rank) {
  return rank <= 64 && rank * k <= 32 * 4096 && lora_items(m, adapters, 16) * ((n + 511) / 512) <= 256;
}

LoraPlan lora_plan(int64_t m, int64_t k, int64_t n, int adapters, int rank, bool y_f32) {
  const int units = rank / 8;
  LoraPlan p = {};
  p.small = lora_small(m, k, n, adapters, rank);
  p.nb = units <= 2 ? 1 : units <= 4 ? 2 : units <= 8 ? 4 : units <= 16 ? 8 : 16;
  if (p.small) return p;
  p.splits = lora_splits(m, k, adapters);
  p.sd = units <= 4 ? 1 : units <= 8 ? 2 : 4;
  // Second product: rows of an item as many as the adapters have on average, as long
  // as workgroups are left for the CUs.
  const int64_t columns = (n + 255) / 256;
  p.rb = 4;
  while (p.rb > 1 && (m < 8ll * p.rb * adapters || lora_items(m, adapters, 16 * p.rb) * columns < 1024)) p.rb /= 2;
  // Chunks of a workgroup: rounds of the CUs times the chunks and what comes ahead
  // of them (of the items that may be, half of the adapters' last ones are there).
  // Many rows: workgroups side by side a multiple of the XCDs, each of which then
  // reads its own columns of B (4096 rows, n 14336, rank 64: 8 side by side 54.9 us,
  // 10 67.5, 19 62.3, 56 64.4; 44 rows of 35 adapters: 56 11.4, 28 8.3, 19 9.1).
  // `places` are those of ranks up to 64.  Above, the parts of t take up to 117 KB and
  // leave one workgroup of 64 rows to a CU; the same chunks were kept there without a
  // measurement of others (4096 rows, n 14336, both launches, bf16 and fp32 y: rank 64 104
  // and 138 us, 128 162 and 192, 256 273 and 318).
  const double expected = (double)m / (16 * p.rb) + 0.5 * (double)std::min<int64_t>(adapters, m);
  const int places = 256 * (p.rb == 4 ? (y_f32 ? 2 : 3) : p.rb == 2 ? (y_f32 ? 3 : 4) : 5);
  double best = 0;
  for (int64_t c = 1; c <= std::min<int64_t>(columns, 32); ++c) {
    const int64_t side = (columns + c - 1) / c;
    const double cost = std::ceil(expected * side / places) * (c + 1) * (p.rb > 1 && side % kXcds != 0 ? 1.25 : 1.);
    if (c > 1 && cost >= best) continue;
    best = cost;
    p.chunks = (int32_t)c;
  }
  return p;
}

hipError_t launch_lora(LoraArgs a, const LoraPlan &p, bool y_f32, hipStream_t s) {
  hipError_t e = hipSuccess;
  auto launch = [&](auto kern, const dim3 &grid, int threads, int lds) {
    if (lds > 64 * 1024) e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, grid, dim3(threads), lds, s, a);
    e = hipGetLastError();
  };
  if (p.small) {
    const dim3 grid((unsigned)((a.n + 511) / 512), (unsigned)lora_items(a.m, a.adapters, 16));
    auto small = [&](auto blocks, auto stages) {
      constexpr int NB = decltype(blocks)::value, ST = decltype(stages)::value, LDS = 8 * ST * (1 + NB) * 2048;
      y_f32 ? launch(lora_small_kernel<NB, ST, true>, grid, 512, LDS) : launch(lora_small_kernel<NB, ST, false>, grid, 512, LDS);
    };
    if (p.nb == 1)
      small(Int<1>(), Int<4>());
    else if (p.nb == 2)
      small(Int<2>(), Int<3>());
    else
      small(Int<4>(), Int<2>());
    return e;
  }
  a.splits = p.splits;
  a.chunks = p.chunks;
  auto down = [&](auto blocks, auto waves, auto stages) {
    constexpr int NB = decltype(blocks)::value, KW = decltype(waves)::value, ST = decltype(stages)::value;
    launch(lora_down_kernel<NB, KW, ST>, dim3((unsigned)lora_items(a.m, a.adapters, 16), a.splits), 64 * KW,
           KW * ST * (1 + NB) * 2048);
  };
  // (rings of 3 stages where two workgroups of them fit a CU)
  if (p.nb == 1)
    down(Int<1>(), Int<4>(), Int<3>());
  else if (p.nb == 2)
    down(Int<2>(), Int<4>(), Int<3>());
  else if (p.nb == 4)
    down(Int<4>(), Int<4>(), Int<2>());
  else if (p.nb == 8)
    down(Int<8>(), Int<4>(), Int<2>());
  else
    down(Int<16>(), Int<2>(), Int<2>());
  if (e != hipSuccess) return e;

  const int64_t columns = (a.n + 255) / 256;
  const int units = a.rank / 8, parts = y_f32 ? 3 : 2;
  const int lds_units = units <= 2 ? (parts * units + 3) / 4 * 4 : parts * ((units + 4 * p.sd - 1) / (4 * p.sd)) * 4 * p.sd;
  const int lds = lds_units * (16 * p.rb + 1) * 16 + 4 * 16 * (64 * 4 + 16);
  const dim3 grid((unsigned)((columns + a.chunks - 1) / a.chunks), (unsigned)lora_items(a.m, a.adapters, 16 * p.rb));
  auto up = [&](auto blocks, auto steps) {
    constexpr int RB = decltype(blocks)::value, SD = decltype(steps)::value;
    y_f32 ? launch(lora_up_kernel<RB, SD, true>, grid, 256, lds) : launch(lora_up_kernel<RB, SD, false>, grid, 256, lds);
  };
  auto with_rows = [&](auto blocks) {
    if (p.sd == 1)
      up(blocks, Int<1>());
    else if (p.sd == 2)
      up(blocks, Int<2>());
    else
      up(blocks, Int<4>());
  };
  if (p.rb == 4)
    with_rows(Int<4>());
  else if (p.rb == 2)
    with_rows(Int<2>());
  else
    with_rows(Int<1>());
  return e;
}

}  // namespace qg
