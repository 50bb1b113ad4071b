// Low-rank adapters of many requests added to the output of a shared projection:
//   y[r] += scale_a (x[r] A_a^T) B_a^T   for the rows r of adapter a,
// A_a [rank][k], B_a [n][rank], rows grouped by adapter (qg_moe_sort's lists).
// Two launches: the first leaves t = x A^T of every listed row in fp32 (k in parts
// where there are few rows), the second adds scale t B^T.  Both work on items of up
// to 16 or 64 rows of one adapter; a workgroup finds its item from the offsets by
// itself, so nothing is planned on the host and no list is written.
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
    for (;; ++e) {
      count = span(e, &begin);
      const int items = (count + ROWS - 1) / ROWS;
      if (at < items) break;
      at -= items;
    }
  return LoraItem{__builtin_amdgcn_readlane(e, owner), __builtin_amdgcn_readlane(begin + at * ROWS, owner),
                  __builtin_amdgcn_readlane(min(ROWS, count - at * ROWS), owner)};
}

// The row of sorted position pos, -1 for an entry that names none
__device__ __forceinline__ int lora_row(const LoraArgs &a, int pos) {
  const int r = a.sorted[pos];
  return r >= 0 && r < a.m ? r : -1;
}

}  // namespace

// t[split][position][rank] = x A^T over the split's part of k, for an item of 16
// rows: KW waves share the part of k and join in LDS.  The operand layout of the
// matrix instruction has neighbouring lanes in different rows, which the memory path
// takes at 16 bytes per clock and CU (51 with four lanes to 64 bytes of a row; L1
// hits, 4 waves per SIMD), and every workgroup reads its whole adapter: so whole
// cache lines go to a ring of ST stages of 64 k in LDS (16-byte chunks of a row at
// slot chunk ^ row % 8), one ring per wave, without barriers.  4096 rows, rank 64, k
// 4096: 16 us (operands straight to registers 24), 44 rows of 35 adapters of rank
// 16: 4.1 us (6.2), one row 3.7 us (5.4).
template <int NB, int KW, int ST>
__global__ __launch_bounds__(64 * KW) void lora_down_kernel(LoraArgs a) {
  constexpr int COPIES = 2 * (1 + NB), STAGE = COPIES * 1024, RING = ST * STAGE;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const LoraItem it = lora_item<16>(a, blockIdx.x);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
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
  // stages of 64 k: of the split, then of the wave
  const int steps = (a.k + 63) / 64, per_split = (steps + a.splits - 1) / a.splits;
  const int s0 = min((int)blockIdx.y * per_split, steps), s1 = min(s0 + per_split, steps);
  const int per_wave = (s1 - s0 + KW - 1) / KW;
  const int begin = min(s0 + kw * per_wave, s1), end = min(begin + per_wave, s1);
  const uint8_t *mine = smem + kw * RING;
  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)mine;
  auto issue = [&](int s) {
    const uint32_t st = ring + (s - begin) % ST * STAGE;
    const bool in = 64 * s + 8 * chunk < a.k;  // (behind k: zeros)
#pragma unroll
    for (int c = 0; c < COPIES; ++c)
      mm_copy16_at(in ? src[c] + 128 * (int64_t)s : (const uint8_t *)mm_zeros, st + c * 1024);
  };
  f32x4 acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < ST - 1; ++s)
    if (begin + s < end) issue(begin + s);
  for (int s = begin; s < end; ++s) {
    // (into the stage that was read last time: its reads are in registers)
    if (s + ST - 1 < end) {
      issue(s + ST - 1);
      QG_WAIT_VMCNT((ST - 1) * COPIES);
    } else if (ST > 2 && s + 1 < end) {
      QG_WAIT_VMCNT(COPIES);
    } else {
      QG_WAIT_VMCNT(0);
    }
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

// y += scale t B^T for one item of 16 RB rows and `chunks` times 256 columns, 64 of
// them per wave.  The parts of t stand in LDS as units of 8 along the contraction,
// [unit][row].  SD x 32 of the rank are in registers at a time, used for every part
// in turn; ranks of 8 and 16 have their parts side by side in one step.  y is loaded
// and stored along its rows, 16 bytes per lane (the sums go through LDS for that),
// and asked for before t.
template <int RB, int SD, bool F32>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int ROWS = 16 * RB, PARTS = F32 ? 3 : 2, EL = F32 ? 4 : 2;
  constexpr int VC = 16 / EL, LPR = 64 / VC, RPP = 64 / LPR, PASSES = 16 / RPP;  // columns per lane, lanes per row, rows per pass
  constexpr int UNIT = ROWS + 1;           // 16-byte rows of a unit (one more: banks)
  constexpr int PITCH = 64 * 4 + 16;       // bytes of a row of the sums
  const LoraItem it = lora_item<ROWS>(a, blockIdx.y);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int units = a.rank / 8;
  const bool side = units <= 2;  // parts side by side
  const int groups = (units + 4 * SD - 1) / (4 * SD), pitch = side ? 4 : groups * 4 * SD;  // units of a part
  const int lds_steps = side ? (PARTS * units + 3) / 4 : PARTS;
  u32x4 *parts = (u32x4 *)smem;  // [lds_steps * pitch][UNIT]
  uint8_t *slab = smem + lds_steps * pitch * UNIT * 16 + wave * 16 * PITCH;

  // this lane's row in each pass of each block of 16 rows, and its first column
  int row[RB][PASSES];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int at = 16 * i + p * RPP + lane / LPR, r = a.sorted[it.pos + min(at, it.rows - 1)];
      row[i][p] = at < it.rows && r >= 0 && r < a.m ? r : -1;
    }
  const int ycol = lane % LPR * VC;

  const uint8_t *bbase = (const uint8_t *)(a.b + (int64_t)it.adapter * a.n * a.ldb);
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 bv[SD][4];
  auto load_b = [&](int col0, int group) {
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
        if (unit >= units) bv[d][j] = zero;
      }
    }
  };
  u32x4 yv[RB][PASSES], next[RB][PASSES];
  auto y_at = [&](int i, int p, int col0) {
    return (uint8_t *)a.y + (max(row[i][p], 0) * a.ldy + col0 + ycol) * EL;
  };
  auto load_y = [&](int col0, u32x4 (&yv)[RB][PASSES]) {
    if (!a.y_vectors || col0 + 64 > a.n) return;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) yv[i][p] = *(const u32x4 *)y_at(i, p, col0);
  };
  const int first_col = blockIdx.x * 256 + 64 * wave, stride = gridDim.x * 256;
  if (first_col < a.n) load_b(first_col, 0);
  load_y(first_col, yv);

  const float scale = a.scales ? a.scales[it.adapter] : 1.f;
  for (int u = threadIdx.x; u < units * ROWS; u += 256) {
    const int r = u / units, unit = u % units;
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
  if (side) {
    for (int u = PARTS * units * UNIT + threadIdx.x; u < lds_steps * 4 * UNIT; u += 256) parts[u] = zero;
  } else {
    for (int u = threadIdx.x; u < PARTS * (pitch - units) * ROWS; u += 256) {
      const int r = u % ROWS, unit = u / ROWS;
      parts[(unit / (pitch - units) * pitch + units + unit % (pitch - units)) * UNIT + r] = zero;
    }
  }
  __syncthreads();

  for (int chunk = 0; chunk < a.chunks; ++chunk) {
    const int col0 = first_col + stride * chunk;
    if (col0 >= a.n) break;  // (whole waves: the matrix instructions take every lane)
    const bool whole = a.y_vectors && col0 + 64 <= a.n, more = chunk + 1 < a.chunks && col0 + stride < a.n;
    if (more) load_y(col0 + stride, next);
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
    if (more) load_b(col0 + stride, 0);
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
        if (whole) {
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
          *(u32x4 *)dst = w;
        } else {
#pragma unroll
          for (int e = 0; e < VC; ++e) {
            if (col0 + ycol + e >= a.n) continue;
            if constexpr (F32)
              ((float *)dst)[e] += d[e];
            else
              ((uint16_t *)dst)[e] = (uint16_t)bf16_pair(bf16_bits_to_f32(((uint16_t *)dst)[e]) + d[e], 0.f);
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads, before the slab's next writes
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) yv[i][p] = next[i][p];
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

// Items at most: one per adapter with rows, and one more for every `rows` rows.
static int64_t lora_items(int64_t m, int adapters, int rows) { return std::min<int64_t>(adapters, m) + m / rows; }

// Parts of k: workgroups for the CUs, of at least 8 stages of 64 each.
int lora_splits(int64_t m, int64_t k, int adapters) {
  const int64_t want = std::max<int64_t>(256 / lora_items(m, adapters, 16), 1), most = std::max<int64_t>((k + 511) / 512, 1);
  return (int)std::min<int64_t>(std::min(want, most), 16);
}

hipError_t launch_lora(LoraArgs a, bool y_f32, hipStream_t s) {
  hipError_t e = hipSuccess;
  auto launch = [&](auto kern, const dim3 &grid, int threads, int lds) {
    if (lds > 64 * 1024) e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, grid, dim3(threads), lds, s, a);
    e = hipGetLastError();
  };
  auto down = [&](auto blocks, auto waves, auto stages) {
    constexpr int NB = decltype(blocks)::value, KW = decltype(waves)::value, ST = decltype(stages)::value;
    launch(lora_down_kernel<NB, KW, ST>, dim3((unsigned)lora_items(a.m, a.adapters, 16), a.splits), 64 * KW,
           KW * ST * (1 + NB) * 2048);
  };
  // (rings of 3 stages where two workgroups of them fit a CU)
  if (a.rank <= 16)
    down(Int<1>(), Int<4>(), Int<3>());
  else if (a.rank <= 32)
    down(Int<2>(), Int<4>(), Int<3>());
  else if (a.rank <= 64)
    down(Int<4>(), Int<4>(), Int<2>());
  else if (a.rank <= 128)
    down(Int<8>(), Int<4>(), Int<2>());
  else
    down(Int<16>(), Int<2>(), Int<2>());
  if (e != hipSuccess) return e;

  // Second product: rows of an item as many as the adapters have on average, as long
  // as workgroups are left for the CUs.
  const int64_t columns = (a.n + 255) / 256;
  int rb = 4;
  while (rb > 1 && (a.m < 8ll * rb * a.adapters || lora_items(a.m, a.adapters, 16 * rb) * columns < 1024)) rb /= 2;
  const int64_t rows = lora_items(a.m, a.adapters, 16 * rb);
  // Chunks of a workgroup: rounds of the CUs times the chunks and what comes ahead
  // of them (of the items that may be, half of the adapters' last ones are there).
  // Many rows: workgroups side by side a multiple of the XCDs, each of which then
  // reads its own columns of B (4096 rows, n 14336, rank 64: 8 side by side 54.9 us,
  // 10 67.5, 19 62.3, 56 64.4; 44 rows of 35 adapters: 56 11.4, 28 8.3, 19 9.1).
  const double expected = (double)a.m / (16 * rb) + 0.5 * (double)std::min<int64_t>(a.adapters, a.m);
  const int places = 256 * (rb == 4 ? (y_f32 ? 2 : 3) : rb == 2 ? (y_f32 ? 3 : 4) : 5);
  double best = 0;
  for (int64_t c = 1; c <= std::min<int64_t>(columns, 32); ++c) {
    const int64_t side = (columns + c - 1) / c;
    const double cost = std::ceil(expected * side / places) * (c + 1) * (rb > 1 && side % kXcds != 0 ? 1.25 : 1.);
    if (c > 1 && cost >= best) continue;
    best = cost;
    a.chunks = (int32_t)c;
  }
  const int units = a.rank / 8, parts = y_f32 ? 3 : 2;
  const int sd = units <= 4 ? 1 : units <= 8 ? 2 : 4;
  const int lds_units = units <= 2 ? (parts * units + 3) / 4 * 4 : parts * ((units + 4 * sd - 1) / (4 * sd)) * 4 * sd;
  const int lds = lds_units * (16 * rb + 1) * 16 + 4 * 16 * (64 * 4 + 16);
  const dim3 grid((unsigned)((columns + a.chunks - 1) / a.chunks), (unsigned)rows);
  auto up = [&](auto blocks, auto steps) {
    constexpr int RB = decltype(blocks)::value, SD = decltype(steps)::value;
    y_f32 ? launch(lora_up_kernel<RB, SD, true>, grid, 256, lds) : launch(lora_up_kernel<RB, SD, false>, grid, 256, lds);
  };
  auto with_rows = [&](auto blocks) {
    if (sd == 1)
      up(blocks, Int<1>());
    else if (sd == 2)
      up(blocks, Int<2>());
    else
      up(blocks, Int<4>());
  };
  if (rb == 4)
    with_rows(Int<4>());
  else if (rb == 2)
    with_rows(Int<2>());
  else
    with_rows(Int<1>());
  return e;
}

}  // namespace qg
