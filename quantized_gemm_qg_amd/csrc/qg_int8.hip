// int8 x int8 products with one fp32 scale per token and per output channel,
// and the quantization of bf16 rows that feeds them:
//   s_r = max_k |x_rk| / 127 (1 for a row of zeros),  q_rk = rint(x_rk / s_r)
//   y_rn = (float)(sum_k q_rk c_nk) * s_r * t_n
// The sum is exact in 32 bits (K < 2^17), so a row's result does not depend
// on the kernel, the tile or the split that computed it.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"
#include "qg_rows.h"

namespace qg {

// One row per workgroup, held in registers (VEC x 16 bytes per thread) between
// its maximum and its codes, so it is read once; longer rows are read a second
// time from L2.  The scale and the quotient are IEEE fp32 divisions, the code
// the nearest integer, ties to even.  4096 x 4096: 50 MB in 13.4 us from memory
// (10.0 at the copy's rate), 16384 rows 42.3 us (0.94 of it), 64 rows 2.9 us: a
// launch of one round of rows and one read's latency, which only more rows hide.
template <int THREADS, int VEC, bool LONG>
__global__ __launch_bounds__(THREADS) void quantize_int8_kernel(const uint16_t *x, int64_t ldx, int64_t k, uint8_t *q,
                                                                int64_t ldq, float *qs, int64_t rows) {
  __shared__ float wave_max[THREADS / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k8 = k / 8;  // units of 8 values
  auto largest = [](const u32x4 &w, float m) {
    float v[8];
    unpack8(w, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
  };
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const u32x4 *xr = (const u32x4 *)(x + row * ldx);
    uint2 *qr = (uint2 *)(q + row * ldq);
    u32x4 keep[VEC];
    float m = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int64_t c = v * THREADS + (int)threadIdx.x;
      keep[v] = c < k8 ? xr[c] : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) m = largest(keep[v], m);
    if constexpr (LONG)
      for (int64_t c = VEC * THREADS + (int)threadIdx.x; c < k8; c += THREADS) m = largest(xr[c], m);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
    if (lane == 0) wave_max[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) m = fmaxf(m, wave_max[w]);
    __syncthreads();  // wave_max is rewritten for the next row
    const float s = i8_scale(m);
    auto codes = [&](const u32x4 &w) {
      float v[8];
      unpack8(w, v);
      return uint2{i8_codes4(v, s), i8_codes4(v + 4, s)};
    };
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int64_t c = v * THREADS + (int)threadIdx.x;
      if (c < k8) qr[c] = codes(keep[v]);
    }
    if constexpr (LONG)
      for (int64_t c = VEC * THREADS + (int)threadIdx.x; c < k8; c += THREADS) qr[c] = codes(xr[c]);
    if (threadIdx.x == 0) qs[row] = s;
  }
}

hipError_t launch_quantize_int8(const void *x, int64_t rows, int64_t k, int64_t ldx, void *q, int64_t ldq, float *qs,
                                hipStream_t s) {
  if (rows == 0 || k == 0) return hipSuccess;
  auto go = [&](auto kern, int threads) {
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min<int64_t>(rows, 256 * 16)), dim3(threads), 0, s, (const uint16_t *)x,
                       ldx, k, (uint8_t *)q, ldq, qs, rows);
  };
  if (k <= 256 * 2 * 8)
    go(quantize_int8_kernel<256, 2, false>, 256);
  else if (k <= 1024 * 2 * 8)
    go(quantize_int8_kernel<1024, 2, false>, 1024);
  else
    go(quantize_int8_kernel<1024, 2, true>, 1024);
  return hipGetLastError();
}

static MmArgs i8_args(const I8Call &c) {
  MmArgs a = {};
  a.a = (const uint8_t *)c.x;
  a.lda = c.ldx;
  a.b = c.codes;
  a.ldb = (int64_t)c.k_blocks * 2048;
  a.m = (int32_t)c.m;
  a.n = c.n;
  a.kd = c.k;
  a.y = c.y;
  a.ldy = c.ldy;
  a.otype = c.otype;
  a.sa = c.x_scales;
  a.sb = c.scales;
  a.act = c.act;
  a.group_m = 4;
  a.counters = c.counters;
  a.partials = (uint64_t *)c.partials;
  return a;
}

// Rows that the few-rows kernel quantizes for itself: one (14336 x 4096: 3.9 us
// less than with a launch of its own for the quantization), or a few short ones
// (2 x 1024: 5.7 against 7.6 us; 2 x 4096: 10.6 against 8.5).
bool i8_quantizes_in_kernel(int64_t m, int64_t k) {
  return m == 1 ? rows_pitch((int)k) <= 64 * 1024 : m <= 4 && m * k <= 2048;
}

template <bool G, int BM, int BN, int WM, int WN, int ST, bool SPLIT>
using I8Cfg = MmCfg<true, kRows, kPacked, G, BM, BN, WM, WN, ST, SPLIT>;

// info: see mm_dispatch
static hipError_t i8_tiled(const I8Call &c, hipStream_t s, MmInfo *info) {
  const MmArgs a = i8_args(c);
  // (the static scratch of qg_gemm_noalloc holds less)
  const uint64_t budget = c.small_scratch ? (8u << 20) - (128u << 10) : kMmPartialBytes;
  if (c.gated)
    return mm_dispatch<I8Cfg<true, 256, 256, 4, 2, 2, false>, I8Cfg<true, 192, 256, 4, 2, 2, false>,
                       I8Cfg<true, 128, 128, 4, 2, 2, true>, I8Cfg<true, 128, 128, 4, 2, 4, true>,
                       I8Cfg<true, 64, 128, 2, 4, 4, true>, I8Cfg<true, 32, 128, 1, 4, 4, true>>(a, budget, s, info);
  // (224 columns, where the cost has fewer rounds of the CUs with them than with 256:
  // 14336 of them in 4096 rows are four whole ones)
  return mm_dispatch<I8Cfg<false, 256, 256, 4, 2, 2, false>, I8Cfg<false, 256, 224, 4, 2, 2, false>,
                     I8Cfg<false, 192, 256, 4, 2, 2, false>, I8Cfg<false, 128, 128, 4, 2, 2, true>,
                     I8Cfg<false, 128, 128, 4, 2, 4, true>, I8Cfg<false, 64, 128, 2, 4, 4, true>,
                     I8Cfg<false, 32, 128, 1, 8, 4, true>>(a, budget, s, info);
}

// Calls of the few-rows kernel: up to 8 rows, and up to 32 as long as the rows
// that every workgroup reads (m k bytes) are not too long beside its 16 columns of
// weights.  The bounds are where the two kernels cross, by N: with few columns the
// tiled kernel's parts of k occupy more CUs; up to 4096 columns every workgroup
// has a CU to itself; above, some CUs have a second one and the others wait for
// them, which brings the crossing down.  us here / tiled, weights of layers in turn that no cache
// holds (bytes m k in brackets):
//   N 1000   16 x 11264 [180 K] 11.0 / 11.0, 16 x 14336 [229 K] 13.4 / 12.0
//   N 1536   24 x 8192 [197 K] 10.4 / 10.6, 28 x 8192 [229 K] 11.0 / 10.6
//   N 4096   20 x 14336 [287 K] 16.2 / 17.2, 24 x 14336 [344 K] 17.3 / 17.3, 32 x
//            14336 [459 K] 19.5 / 17.3
//   N 5120   20 x 4096 [82 K] 10.0 / 10.3, 32 x 4096 [131 K] 12.2 / 10.5; 12 x 8192
//            [98 K] 13.7 / 14.1, 16 x 14336 [229 K] 25.2 / 19.1
//   N 7168   24 x 4096 [98 K] 11.0 / 11.6, 24 x 14336 [344 K] 31.0 / 23.2; 16 x 8192
//            [131 K] 16.2 / 16.6, 12 x 14336 [172 K] 23.6 / 23.0
// 17 rows and more of 8192 columns and more: tiled (32 rows of 14336 x 4096: 21.7
// here, 18.2 tiled).  Gated, from 2 rows on, not with many columns (4 rows: 8192 x
// 4096 15.5 us against 18.0, 12288 x 4096 22.0 against 20.9, 14336 x 4096 26.0
// against 23.6).
static bool i8_few_rows(const I8Call &c) {
  if (c.gated) return c.m == 1 || (c.m <= 16 && c.n < 10000);
  if (c.m <= 8 || c.m > 32) return c.m <= 8;
  const int64_t read = c.m * c.k;
  if (c.n <= 1536) return read <= 200000;
  if (c.n <= 4096) return read <= 24 * 14336;
  return c.m <= 16 ? read <= 32 * 4096 : c.n < 8192 && read <= 24 * 4096;
}

hipError_t launch_i8(const I8Call &c, hipStream_t s) {
  MmArgs a = i8_args(c);
  if (c.quantize) {
    a.lda = c.ldx * 2;
    return c.gated ? launch_rows<true, true, 1, 2, 4, true>(a, s) : launch_rows<true, false, 1, 1, 8, true>(a, s);
  }
  if (!i8_few_rows(c)) return i8_tiled(c, s, nullptr);
  if (c.m > 16) return launch_rows<true, false, 2, 1, 2, false>(a, s);
  // (gated: two blocks a trip; with four the registers spill, one row of 14336 x
  // 4096 25.2 us against 23.1)
  return c.gated ? launch_rows<true, true, 1, 2, 2, false>(a, s) : launch_rows<true, false, 1, 1, 4, false>(a, s);
}

MmInfo i8_info(const I8Call &c) {
  MmInfo info;
  if (c.quantize || i8_few_rows(c))
    info.bm = c.m > 16 ? 32 : 16;
  else
    (void)i8_tiled(c, nullptr, &info);
  return info;
}

}  // namespace qg
