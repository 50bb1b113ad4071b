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
  int mine = 0, begin;
  for (int e = first; e < last; ++e) mine += (span(e, &begin) + ROWS - 1) / ROWS;
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off);
    if (lane >= off) upto += o;
  }
  const uint64_t behind = __ballot(upto > item);
  if (behind == 0) return LoraItem{-1, 0, 0};
  const int owner = __ffsll((unsigned long long)behind) - 1;
  LoraItem found = {-1, 0, 0};
  if (lane == owner) {
    int at = item - (upto - mine);
    for (int e = first; e < last; ++e) {
      const int count = span(e, &begin), items = (count + ROWS - 1) / ROWS;
      if (at < items) {
        found = LoraItem{e, begin + at * ROWS, min(ROWS, count - at * ROWS)};
        break;
      }
      at -= items;
    }
  }
  found.adapter = __builtin_amdgcn_readlane(found.adapter, owner);
  found.pos = __builtin_amdgcn_readlane(found.pos, owner);
  found.rows = __builtin_amdgcn_readlane(found.rows, owner);
  return found;
}

// The row of sorted position pos, -1 for an entry that names none
__device__ __forceinline__ int lora_row(const LoraArgs &a, int pos) {
  const int r = a.sorted[pos];
  return r >= 0 && r < a.m ? r : -1;
}

}  // namespace

// t[split][position][rank] = x A^T over the split's part of k.  A wave computes 16
// rows x 16 NB columns with operands straight from memory (16 bytes per lane, U
// steps of 32 k in flight).  RW waves take 16 rows each; the KW waves of a row block
// share the part of k and join in LDS.
template <int NB, int RW, int KW>
__global__ __launch_bounds__(64 * RW *KW) void lora_down_kernel(LoraArgs a) {
  constexpr int U = NB <= 2 ? 8 : NB <= 4 ? 4 : 2;
  __shared__ f32x4 join[KW > 1 ? RW * (KW - 1) * NB * 64 : 1];
  const LoraItem it = lora_item<16 * RW>(a, blockIdx.x);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int q = lane >> 4, r16 = lane & 15;
  const bool any = 16 * rw < it.rows;
  const int pos = it.pos + min(16 * rw + r16, it.rows - 1);
  const int row = max(lora_row(a, pos), 0);
  const uint16_t *xp = a.x + row * a.ldx + 8 * q;
  const uint16_t *ap[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    ap[j] = a.a + ((int64_t)it.adapter * a.rank + min(16 * j + r16, a.rank - 1)) * a.lda + 8 * q;
  // steps of 32 k: of the split, then of the wave
  const int steps = (a.k + 31) / 32, per_split = (steps + a.splits - 1) / a.splits;
  const int s0 = blockIdx.y * per_split, s1 = min(s0 + per_split, steps);
  const int per_wave = (max(s1 - s0, 0) + KW - 1) / KW;
  const int begin = s0 + kw * per_wave, end = any ? min(begin + per_wave, s1) : begin;
  f32x4 acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int s = begin; s < end; s += U) {
    u32x4 xv[U], av[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (steps behind the wave's last one are loaded again and multiplied by zeros;
      // so are the units behind k)
      const int at = min(s + u, end - 1);
      const bool in = 32 * at + 8 * q < a.k;
      const int64_t off = in ? 32 * (int64_t)at : 0;
      xv[u] = *(const u32x4 *)(xp + (in ? off : -8 * q));
#pragma unroll
      for (int j = 0; j < NB; ++j) av[u][j] = *(const u32x4 *)(ap[j] + (in ? off : -8 * q));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = s + u < end && 32 * (s + u) + 8 * q < a.k;
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] = mfma_bf16(in ? av[u][j] : zero, in ? xv[u] : zero, acc[j]);
    }
  }
  if constexpr (KW > 1) {
    if (kw > 0) {
#pragma unroll
      for (int j = 0; j < NB; ++j) join[((rw * (KW - 1) + kw - 1) * NB + j) * 64 + lane] = acc[j];
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int o = 0; o < KW - 1; ++o)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] += join[((rw * (KW - 1) + o) * NB + j) * 64 + lane];
  }
  if (16 * rw + r16 >= it.rows) return;
  float *t = a.t + ((int64_t)blockIdx.y * a.m + it.pos + 16 * rw + r16) * a.rank;
#pragma unroll
  for (int j = 0; j < NB; ++j)
    if (16 * j + 4 * q < a.rank) *(f32x4 *)(t + 16 * j + 4 * q) = acc[j];
}

// y += scale t B^T for one item and 256 columns, 64 per wave.  Which column of B a
// lane brings is arbitrary: block j's column c is 16 (c / 4) + 4 j + c % 4, so a lane
// ends with 16 neighbouring columns of one row, and four lanes with a cache line.
// The parts of t stand in LDS as units of 8 along the contraction: [unit][row].
template <int RB, bool F32>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int ROWS = 16 * RB, PARTS = F32 ? 3 : 2, EL = F32 ? 4 : 2;
  const LoraItem it = lora_item<ROWS>(a, blockIdx.y);
  if (it.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int col0 = blockIdx.x * 256 + 64 * wave;
  const int units = a.rank / 8, steps = (PARTS * units + 3) / 4;
  u32x4 *parts = (u32x4 *)smem;  // [4 steps][ROWS]

  // this lane's 16 columns of its row in each block of 16 rows
  const int col = col0 + 16 * q;
  uint8_t *yp[RB];
  bool store[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int p = 16 * i + r16, row = lora_row(a, it.pos + min(p, it.rows - 1));
    store[i] = p < it.rows && row >= 0 && col < a.n;
    yp[i] = (uint8_t *)a.y + (max(row, 0) * a.ldy + min(col, a.n - 1)) * EL;
  }
  const bool whole = a.y_vectors && col + 16 <= a.n;
  u32x4 yv[RB][EL];
  if (whole) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int h = 0; h < EL; ++h) yv[i][h] = ((const u32x4 *)yp[i])[h];
  }

  const float scale = a.scales ? a.scales[it.adapter] : 1.f;
  for (int u = threadIdx.x; u < units * ROWS; u += 256) {
    const int row = u % ROWS, unit = u / ROWS;
    const float *t = a.t + ((int64_t)it.pos + min(row, it.rows - 1)) * a.rank + 8 * unit;
    f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    for (int s = 0; s < a.splits; ++s) {
      const f32x4 *p = (const f32x4 *)(t + (int64_t)s * a.m * a.rank);
      v0 += p[0];
      v1 += p[1];
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * scale;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
      parts[(part * units + unit) * ROWS + row] = w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // what the part left (nothing of an infinity or a NaN)
        const float f = __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        v[e] = fabsf(f) <= 3.4e38f ? v[e] - f : 0.f;
      }
    }
  }
  for (int u = PARTS * units * ROWS + threadIdx.x; u < 4 * steps * ROWS; u += 256) parts[u] = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();

  const uint16_t *bp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    bp[j] = a.b + ((int64_t)it.adapter * a.n + min(col0 + 16 * (r16 >> 2) + 4 * j + (r16 & 3), a.n - 1)) * a.ldb;
  f32x4 acc[RB][4];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (col0 < a.n)  // (whole waves only: the matrix instructions take every lane)
    for (int s = 0; s < steps; ++s) {
      const int unit = 4 * s + q;
      // (units behind the last part: zeros in LDS, any finite or not values of B must not meet them)
      const int at = unit % units;
      u32x4 bv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bv[j] = *(const u32x4 *)(bp[j] + 8 * at);
        if (unit >= PARTS * units) bv[j] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const u32x4 tv = parts[unit * ROWS + 16 * i + r16];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(bv[j], tv, acc[i][j]);
      }
    }
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (!store[i]) continue;
    if (whole) {
#pragma unroll
      for (int h = 0; h < EL; ++h) {
        u32x4 w = yv[i][h];
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + acc[i][h][e]);
        } else {
          float v[8];
          unpack8(w, v);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = bf16_pair(v[2 * e] + acc[i][2 * h + e / 2][2 * (e % 2)], v[2 * e + 1] + acc[i][2 * h + e / 2][2 * (e % 2) + 1]);
        }
        ((u32x4 *)yp[i])[h] = w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (col + c >= a.n) continue;
        if constexpr (F32) {
          ((float *)yp[i])[c] += acc[i][c / 4][c % 4];
        } else {
          uint16_t *p = (uint16_t *)yp[i] + c;
          *p = (uint16_t)bf16_pair(bf16_bits_to_f32(*p) + acc[i][c / 4][c % 4], 0.f);
        }
      }
    }
  }
}

// Rows of an item: 64 where the adapters have that many on average, so that a
// workgroup reads its adapter's columns once for more rows.
static int lora_rows(int64_t m, int adapters) { return m >= 32ll * adapters ? 64 : 16; }
static int64_t lora_items(int64_t m, int adapters) {
  return std::min<int64_t>(adapters, m) + m / lora_rows(m, adapters);
}

// Parts of k: workgroups for the CUs, of at least 16 steps of 32 each.
int lora_splits(int64_t m, int64_t k, int adapters) {
  const int64_t want = std::max<int64_t>(256 / lora_items(m, adapters), 1), most = std::max<int64_t>((k + 511) / 512, 1);
  return (int)std::min<int64_t>(std::min(want, most), 16);
}

hipError_t launch_lora(const LoraArgs &a, bool y_f32, hipStream_t s) {
  const int rows = lora_rows(a.m, a.adapters);
  const unsigned items = (unsigned)lora_items(a.m, a.adapters);
  auto down = [&](auto kern, int threads) { hipLaunchKernelGGL(kern, dim3(items, a.splits), dim3(threads), 0, s, a); };
  if (rows == 64)
    a.rank <= 16    ? down(lora_down_kernel<1, 4, 1>, 256)
    : a.rank <= 32  ? down(lora_down_kernel<2, 4, 1>, 256)
    : a.rank <= 64  ? down(lora_down_kernel<4, 4, 1>, 256)
    : a.rank <= 128 ? down(lora_down_kernel<8, 4, 1>, 256)
                    : down(lora_down_kernel<16, 4, 1>, 256);
  else
    a.rank <= 16    ? down(lora_down_kernel<1, 1, 8>, 512)
    : a.rank <= 32  ? down(lora_down_kernel<2, 1, 8>, 512)
    : a.rank <= 64  ? down(lora_down_kernel<4, 1, 8>, 512)
    : a.rank <= 128 ? down(lora_down_kernel<8, 1, 4>, 256)
                    : down(lora_down_kernel<16, 1, 4>, 256);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = y_f32 ? 3 : 2, lds = (parts * a.rank / 8 + 3) / 4 * 4 * rows * 16;
  auto up = [&](auto kern) {
    e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.n + 255) / 256), items), dim3(256), lds, s, a);
    e = hipGetLastError();
  };
  if (rows == 64)
    y_f32 ? up(lora_up_kernel<4, true>) : up(lora_up_kernel<4, false>);
  else
    y_f32 ? up(lora_up_kernel<1, true>) : up(lora_up_kernel<1, false>);
  return e;
}

}  // namespace qg
