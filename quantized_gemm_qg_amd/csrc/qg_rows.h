// Products of few rows (up to 16 MT): int8 layers and the bf16 gated block, bound
// by the weight bytes.  A workgroup computes NT strips of 16 columns (gated: one
// gate strip and its up strip) for all rows and all of K; its waves split K in
// runs of KR blocks of 128 bytes per row and join their 16 x 16 partial blocks
// in LDS.  Weights go from memory straight into the MFMA's operand registers,
// 16 bytes per lane and load, all loads of a run in flight before its first
// product, so nothing is staged and no barrier stands between loads.
//
// One token of 14336 x 4096: int8 14.3 us from memory (4.1 TB/s of weights) and
// 12.9 from the last-level cache (256 MB), int8 gated 20.8 us (5.6 TB/s), bf16
// gated 43.2 us (5.4 TB/s); a copy reaches 5.1 TB/s.
//
// PAST (int8 weights of up to 16 rows, from 64 MB on): loads past the caches.  us
// through the caches / past them, of layers in turn that no cache holds, and in
// brackets of three layers in turn:
//   1 row     8192 x 4096   10.1 / 9.6   [9.4 / 9.0]
//             14336 x 4096  14.3 / 13.6  [12.9 / 12.9]
//             28672 x 4096  23.9 / 21.8  [23.9 / 21.4], gated 23.0 / 21.1 [23.0 / 20.7]
//   16 rows   8192 x 4096   9.6 / 9.3    [8.0 / 8.8]
//             14336 x 4096  16.9 / 15.8  [13.1 / 15.1]
//             28672 x 4096  30.6 / 29.0  [30.4 / 28.4]
// What comes from memory gains 2 to 10 % at every size, what the last-level cache
// holds loses up to 16 %.  From 64 MB on a few layers fill that cache; below,
// whether they are found there is the program's, and the loads go through it.
// Not 17 rows and more (23 rows of 4096 x 14336 17.1 / 16.5 [14.3 / 16.1]), nor
// bf16, whose lines take two loads each (45.3 -> 48.2).
//
// FUSEQ (int8, the rows' codes fit in LDS): x is bf16 and every workgroup
// quantizes it for itself while its first weights are on their way, which
// costs it a read of x from L2 and saves a launch.  Otherwise the rows come
// from L2 in the operand's layout.
#pragma once

#include "qg_mm.h"
#include "qg_quant.h"

namespace qg {

// Bytes of a row's codes in LDS: whole blocks (what lies behind K meets zero
// weights), and 16 more so that rows start on different banks.
__host__ __device__ constexpr int rows_pitch(int k) { return (k + 127) / 128 * 128 + 16; }
// LDS: codes of the quantized rows and their scales (FUSEQ), partial blocks
template <int MT, int NT>
constexpr int64_t rows_lds_bytes(bool fuseq, int64_t m, int64_t k, int waves) {
  return (fuseq ? m * rows_pitch((int)k) + 256 : 0) + (int64_t)waves * NT * MT * 1024;
}

// Waves of a workgroup: eight at most (two workgroups per CU, so one's joining
// and writing is behind the other's loads: the bf16 block at one token 45.7 us
// against 52.1 with one workgroup of 16 waves), four for the int8 gated form
// (23.9 against 25.2).
template <bool I8, bool GATED>
constexpr int rows_waves() { return I8 && GATED ? 4 : 8; }

template <bool I8, bool GATED, int MT, int NT, int KR, bool FUSEQ, bool PAST>
__global__ __launch_bounds__((I8 && GATED) ? 256 : 512, MT == 1 ? 4 : 3) void rows_kernel(MmArgs a) {
  static_assert(!FUSEQ || (I8 && MT == 1), "quantized rows in LDS");
  static_assert(!GATED || NT == 2, "a gate strip and its up strip");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ float row_max[16];
  typedef typename std::conditional<I8, i32x4, f32x4>::type Acc;
  constexpr int KE = I8 ? 128 : 64;  // k per block
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int q = lane >> 4, r16 = lane & 15;
  const int strip0 = blockIdx.x * (GATED ? 1 : NT);
  // whole blocks are split over the waves in contiguous runs; the last wave
  // also takes the block that K ends in
  const int blocks = a.kd / KE, run = (blocks + waves - 1) / waves;
  const int b_begin = min(wave * run, blocks), b_end = min(b_begin + run, blocks);

  // 64-bit bases per strip (uniform), 32-bit lane offsets: this lane's weight
  // column of each strip, and its row of each 16 rows of x
  const uint8_t *bp[NT];
  uint32_t bo[NT], ao[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int first = min((GATED ? strip0 : strip0 + t) * 16, a.n - 1) + (GATED && t == 1 ? a.n : 0);
    const int col = min((GATED ? strip0 : strip0 + t) * 16 + r16, a.n - 1) + (GATED && t == 1 ? a.n : 0);
    if constexpr (I8) {
      bp[t] = a.b + (int64_t)(first / 16) * a.ldb;
      bo[t] = (uint32_t)((col / 16 - first / 16) * a.ldb) + q * 256 + (col % 16) * 16;
    } else {
      bp[t] = a.b + (int64_t)first * a.ldb;
      bo[t] = (uint32_t)((col - first) * a.ldb) + 16 * q;
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) ao[i] = (uint32_t)(min(16 * i + r16, a.m - 1) * a.lda) + 16 * q;

  u32x4 bw[KR][NT][2], aw[FUSEQ ? 1 : KR][MT][2];
  auto load = [&](int b, int r) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint8_t *u = bp[t] + (int64_t)b * (I8 ? 2048 : 128);  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 *p = (const u32x4 *)(u + bo[t] + (I8 ? 1024 : 64) * h);
        bw[r][t][h] = PAST ? __builtin_nontemporal_load(p) : *p;
      }
    }
    if constexpr (!FUSEQ) {
      const uint8_t *u = a.a + (int64_t)b * 128;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) aw[r][i][h] = *(const u32x4 *)(u + ao[i] + 64 * h);
    }
  };
  // one row to quantize: its first 16-byte units per thread, asked for ahead of
  // the weights (loads return in order, so behind them they would wait for all)
  constexpr int XV = FUSEQ ? 4 : 1;
  u32x4 xv[XV];
  if constexpr (FUSEQ) {
#pragma unroll
    for (int i = 0; i < XV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      xv[i] = a.m == 1 && c < a.kd / 8 ? *(const u32x4 *)(a.a + 16 * c) : u32x4{0u, 0u, 0u, 0u};
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // (where a run ends inside KR blocks its last one is loaded again: under a
  // condition of its own a load would leave the compiler no count to wait by,
  // and it would wait for all of them)
  const bool any = b_begin < b_end;
  if (any) {
#pragma unroll
    for (int r = 0; r < KR; ++r) load(min(b_begin + r, b_end - 1), r);
  }
  __builtin_amdgcn_sched_barrier(0);

  const int pitch = rows_pitch(a.kd);
  float *row_scale = nullptr;
  uint8_t *red = smem;
  if constexpr (FUSEQ) {
    row_scale = (float *)(smem + a.m * pitch);
    red = (uint8_t *)row_scale + 256;
    auto largest_of = [](const u32x4 &w, float most) {
      float v[8];
      unpack8(w, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
      return most;
    };
    auto largest = [&](const uint8_t *xr, int c0, int step, float most) {
      for (int c = c0; c < a.kd / 8; c += step) most = largest_of(*(const u32x4 *)(xr + 16 * c), most);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) most = fmaxf(most, __shfl_xor(most, off));
      return most;
    };
    auto put = [&](int r, int c, const u32x4 &w, float s) {
      float v[8];
      unpack8(w, v);
      *(uint2 *)(smem + r * pitch + 8 * c) = uint2{i8_codes4(v, s), i8_codes4(v + 4, s)};
    };
    auto codes = [&](int r, const uint8_t *xr, float s, int c0, int step) {
      for (int c = c0; c < a.kd / 8; c += step) put(r, c, *(const u32x4 *)(xr + 16 * c), s);
    };
    if (a.m == 1) {  // one row: the whole workgroup
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < XV; ++i) most = largest_of(xv[i], most);
      most = largest(a.a, threadIdx.x + XV * blockDim.x, blockDim.x, most);
      if (lane == 0) row_max[wave] = most;
      __syncthreads();
      for (int w = 0; w < waves; ++w) most = fmaxf(most, row_max[w]);
      const float s = i8_scale(most);
#pragma unroll
      for (int i = 0; i < XV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < a.kd / 8) put(0, c, xv[i], s);
      }
      codes(0, a.a, s, threadIdx.x + XV * blockDim.x, blockDim.x);
      if (threadIdx.x == 0) row_scale[0] = s;
    } else {  // a row per wave, without barriers between them
      for (int r = wave; r < a.m; r += waves) {
        const uint8_t *xr = a.a + (int64_t)r * a.lda;
        const float s = i8_scale(largest(xr, lane, 64, 0.f));
        codes(r, xr, s, lane, 64);
        if (lane == 0) row_scale[r] = s;
      }
    }
    __syncthreads();
  }

  Acc acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = Acc{0, 0, 0, 0};
  auto multiply = [&](int b, int r) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        u32x4 av;
        if constexpr (FUSEQ)
          av = *(const u32x4 *)(smem + min(r16, a.m - 1) * pitch + b * 128 + 64 * h + 16 * q);
        else
          av = aw[r][i][h];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (I8)
            acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, bw[r][t][h]),
                                                              __builtin_bit_cast(i32x4, av), acc[i][t], 0, 0, 0);
          else
            acc[i][t] = mfma_bf16(bw[r][t][h], av, acc[i][t]);
        }
      }
  };
  if (any) {
    int b = b_begin;
    for (; b + KR < b_end; b += KR) {
#pragma unroll
      for (int r = 0; r < KR; ++r) {
        multiply(b + r, r);
        load(min(b + KR + r, b_end - 1), r);
      }
    }
#pragma unroll
    for (int r = 0; r < KR; ++r)
      if (b + r < b_end) multiply(b + r, r);
  }
  if (wave == waves - 1 && blocks * KE < a.kd) {
    // the block that K ends in: lanes behind the end read zeros for both
    // operands (int8 weights are padded with zeros: the rows read their first
    // bytes instead)
    const uint8_t *zeros = (const uint8_t *)mm_zeros;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = blocks * KE + (I8 ? 64 : 32) * h + (I8 ? 16 : 8) * q < a.kd;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        bw[0][t][h] = I8 ? *(const u32x4 *)(bp[t] + (int64_t)blocks * 2048 + bo[t] + 1024 * h)
                         : *(const u32x4 *)(in ? bp[t] + (int64_t)blocks * 128 + bo[t] + 64 * h : zeros);
      if constexpr (!FUSEQ) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
          aw[0][i][h] = *(const u32x4 *)(in ? a.a + (int64_t)blocks * 128 + ao[i] + 64 * h : zeros);
      }
    }
    multiply(blocks, 0);
  }
  // partial blocks [wave][strip][row tile][row][16 columns]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i) *(Acc *)(red + ((wave * NT + t) * MT + i) * 1024 + r16 * 64 + q * 16) = acc[i][t];
  __syncthreads();
  // outputs, 4 columns per thread
  constexpr int OUT_T = GATED ? 1 : NT;
  for (int o = threadIdx.x; o < OUT_T * a.m * 4; o += blockDim.x) {
    const int t = o / (a.m * 4), row = (o / 4) % a.m, c4 = 4 * (o % 4);
    const int col = (strip0 + t) * 16 + c4;
    if (col >= a.n) continue;
    auto total = [&](int strip) {
      Acc s = {0, 0, 0, 0};
      for (int w = 0; w < waves; ++w)
        s += *(const Acc *)(red + ((w * NT + strip) * MT + row / 16) * 1024 + (row % 16) * 64 + c4 * 4);
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)s[e];
        if constexpr (I8)
          v[e] = v[e] * (FUSEQ ? row_scale[row] : a.sa[row]) * a.sb[min(col + e, a.n - 1) + (GATED && strip ? a.n : 0)];
      }
      return v;
    };
    auto store = [&](void *out, int64_t at, int otype, const f32x4 &v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col + e >= a.n) continue;
        if (otype == QG_O_F32)
          ((float *)out)[at + e] = v[e];
        else
          ((uint16_t *)out)[at + e] = (uint16_t)bf16_rne(v[e]);
      }
    };
    if constexpr (GATED) {
      const f32x4 g = total(0), u = total(1);
      if (a.gu) {
        store(a.gu, row * a.ldgu + col, a.gu_type, g);
        store(a.gu, row * a.ldgu + a.n + col, a.gu_type, u);
      }
      if (a.y) {
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_value(g[e], a.act) * u[e];
        store(a.y, row * a.ldy + col, a.otype, h);
      }
    } else {
      store(a.y, row * a.ldy + col, a.otype, total(t));
    }
  }
}

template <bool I8, bool GATED, int MT, int NT, int KR, bool FUSEQ>
static hipError_t launch_rows(const MmArgs &a, hipStream_t s) {
  constexpr int KE = I8 ? 128 : 64;
  const int runs = a.kd / KE > 0 ? (a.kd / KE + KR - 1) / KR : 1;
  const int waves = runs < rows_waves<I8, GATED>() ? runs : rows_waves<I8, GATED>();
  const int strips = (a.n + 15) / 16, per = GATED ? 1 : NT;
  const int64_t lds = rows_lds_bytes<MT, NT>(FUSEQ, a.m, a.kd, waves);
  auto kern = rows_kernel<I8, GATED, MT, NT, KR, FUSEQ, false>;
  if constexpr (I8 && MT == 1) {
    if ((int64_t)a.n * a.kd * (GATED ? 2 : 1) >= (64 << 20)) kern = rows_kernel<I8, GATED, MT, NT, KR, FUSEQ, true>;
  }
  hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((strips + per - 1) / per), dim3(64 * waves), lds, s, a);
  return hipGetLastError();
}

}  // namespace qg
