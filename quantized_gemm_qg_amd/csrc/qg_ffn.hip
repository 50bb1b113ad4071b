// Gated feed-forward block in bf16, forward and backward:
//   g = x Wg^T, u = x Wu^T, h = act(g) u
//   du = dh act(g), dg = dh u act'(g), dx = dg Wg + du Wu, dW = [dg du]^T x
// The forward is one launch (both projections, the activation and the
// product, the pre-activations saved on request); the backward is one
// elementwise pass that leaves [dg du] in bf16 and one product per gradient.
// [dg du] is rounded to bf16 once because the matrix cores take bf16 operands
// (fp32 ones run at 1/16 of the rate): the rounding errors of its elements are
// independent, so each gradient's relative error grows from the output
// rounding's 1.7e-3 (2-norm) to sqrt(2) times that, and an fp32 dW has 1.7e-3 from
// it.  (Two parts for all tokens would double the products.)  With few tokens single
// elements decide and nothing is bound by the matrix cores, so there [dg du] is
// kept as the sum of two bf16 numbers (dx up to 16 tokens, dW up to 32: as far
// as one tile or stage holds both parts).
// 4096 tokens, 14336 x 4096: forward with pre-activations 794 us (1.21 PFLOP/s), the
// elementwise pass 158, dx 725, dW 750.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"
#include "qg_rows.h"

namespace qg {

// [dg du] ([m][ldd] bf16, ldd >= 2 inter, zeros from 2 inter to ldd) from the
// pre-activations and dh.  One pass, bound by its bytes: 822 MB for 4096 x 14336
// with fp32 pre-activations in 158 us.  A thread takes VEC consecutive elements
// of a row: 4 where their bf16 quadruples are 8-byte aligned (inter and the
// pitches multiples of 4), else 1 -- accesses of 8 bytes at odd elements are
// split by the hardware and took three times as long as single ones (257 x
// 2817: 17.2 against 5.1 us).
template <bool F32, int VEC>
__global__ __launch_bounds__(256) void ffn_dgu_kernel(const void *gu, int64_t ldgu, const uint16_t *dh, int64_t lddh,
                                                      int64_t inter, int act, uint16_t *dgu, int64_t ldd,
                                                      int64_t halves) {
  struct alignas(2 * VEC) Bf {
    uint16_t v[VEC];
  };
  struct alignas(4) Fp {  // (rows of the pre-activations start at any fp32)
    float v[VEC];
  };
  const int64_t row = blockIdx.y, c = VEC * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  uint16_t *d = dgu + row * ldd, *d2 = d + halves * ldd;
  if (c >= inter) {  // padding columns
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (inter + c + e < ldd) {
        d[inter + c + e] = 0;
        if (halves > 0) d2[inter + c + e] = 0;
      }
    return;
  }
  float g[VEC], u[VEC];
  if constexpr (F32) {
    const float *p = (const float *)gu + row * ldgu + c;
    const Fp gv = *(const Fp *)p, uv = *(const Fp *)(p + inter);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = gv.v[e], u[e] = uv.v[e];
  } else {
    const uint16_t *p = (const uint16_t *)gu + row * ldgu + c;
    const Bf gv = *(const Bf *)p, uv = *(const Bf *)(p + inter);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = bf16_bits_to_f32(gv.v[e]), u[e] = bf16_bits_to_f32(uv.v[e]);
  }
  const Bf hv = *(const Bf *)(dh + row * lddh + c);
  // what the first part's rounding left (nothing of an infinity or a NaN)
  auto rest = [](float v, uint16_t first) {
    return (uint16_t)((first & 0x7F80u) == 0x7F80u ? 0 : bf16_rne(v - bf16_bits_to_f32(first)));
  };
  Bf dg, du, dg2, du2;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float h = bf16_bits_to_f32(hv.v[e]);
    float v, dv;
    act_both(g[e], act, &v, &dv);
    const float g1 = h * u[e] * dv, u1 = h * v;
    dg.v[e] = (uint16_t)bf16_rne(g1);
    du.v[e] = (uint16_t)bf16_rne(u1);
    dg2.v[e] = rest(g1, dg.v[e]);
    du2.v[e] = rest(u1, du.v[e]);
  }
  *(Bf *)(d + c) = dg;
  *(Bf *)(d + inter + c) = du;
  if (halves > 0) {
    *(Bf *)(d2 + c) = dg2;
    *(Bf *)(d2 + inter + c) = du2;
  }
}

__global__ __launch_bounds__(256) void ffn_zero_kernel(uint8_t *p, int64_t ld_bytes, int64_t row_bytes, int64_t rows) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = 2 * (int64_t)threadIdx.x; c < row_bytes; c += 512) *(uint16_t *)(p + r * ld_bytes + c) = 0;
}

// (info: nothing is launched, see mm_dispatch)
hipError_t launch_ffn_forward(const FfnCall &c, hipStream_t s, MmInfo *info) {
  if (info) *info = MmInfo();
  MmArgs a = {};
  a.a = (const uint8_t *)c.x;
  a.lda = c.ldx * 2;
  a.b = (const uint8_t *)c.w;
  a.ldb = c.ldw * 2;
  a.m = (int32_t)c.m;
  a.n = (int32_t)c.inter;
  a.kd = (int32_t)c.k;
  a.y = c.h;
  a.ldy = c.ldh;
  a.otype = QG_O_BF16;
  a.gu = c.gu;
  a.ldgu = c.ldgu;
  a.gu_type = c.gu_type;
  a.act = c.act;
  a.group_m = 4;
  a.counters = c.counters;
  a.partials = (uint64_t *)c.partials;
  // Few rows: a workgroup per 16 columns with all of K, unless long rows meet few
  // columns, where the tiled kernel's parts of k occupy more CUs (8 rows: 400 x
  // 2560 8.6 us against 10.8, 1700 x 8192 17.1 against 23.6, 2400 x 8192 20.6
  // against 26.1; 4000 x 8192 34.7 against 27.5, 1500 x 2048 8.3 against 7.8; 2
  // rows of 3000 x 8192 24.3 against 22.7).  From 17 rows on tiled (24 rows of
  // 14336 x 4096: 51.9 us, 71.4 with two row blocks here).
  if (c.m <= 16 && (c.k < 2560 || c.inter > (c.m <= 4 ? 2048 : 3000)))
    return info ? hipSuccess : launch_rows<false, true, 1, 2, 4, false>(a, s);
  return mm_dispatch<MmCfg<false, kRows, kRows, true, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kRows, kRows, true, 192, 256, 4, 2, 2, false>,
                     MmCfg<false, kRows, kRows, true, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kRows, kRows, true, 128, 128, 4, 2, 4, true>,
                     MmCfg<false, kRows, kRows, true, 64, 128, 2, 4, 4, true>,
                     MmCfg<false, kRows, kRows, true, 32, 128, 1, 4, 4, true>>(a, kMmPartialBytes, s, info);
}

// Rows from the first to the second part of [dg du], 0: there is no second one.
static int64_t ffn_halves(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 0; }
int64_t ffn_dgu_rows(int64_t m) { return m + ffn_halves(m); }

hipError_t launch_ffn_dgu(const FfnCall &c, const void *dh, int64_t lddh, void *dgu, int64_t ldd, hipStream_t s) {
  const bool f32 = c.gu_type == QG_O_F32;
  const bool four = c.inter % 4 == 0 && lddh % 4 == 0 && ((uintptr_t)dh & 7) == 0 && (f32 || c.ldgu % 4 == 0);
  const int64_t per = four ? 1024 : 256;
  for (int64_t r0 = 0; r0 < c.m; r0 += 65535) {
    const dim3 grid((unsigned)((ldd - c.inter + per - 1) / per), (unsigned)std::min<int64_t>(c.m - r0, 65535));
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, grid, dim3(256), 0, s,
                         (const void *)((const uint8_t *)c.gu + r0 * c.ldgu * (f32 ? 4 : 2)), c.ldgu,
                         (const uint16_t *)dh + r0 * lddh, lddh, c.inter, c.act, (uint16_t *)dgu + r0 * ldd, ldd, ffn_halves(c.m));
    };
    if (four)
      f32 ? go(ffn_dgu_kernel<true, 4>) : go(ffn_dgu_kernel<false, 4>);
    else
      f32 ? go(ffn_dgu_kernel<true, 1>) : go(ffn_dgu_kernel<false, 1>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// dx = [dg du] W: contraction over the 2 inter rows of W
hipError_t launch_ffn_dx(const FfnCall &c, const void *dgu, int64_t ldd, void *dx, int64_t lddx, hipStream_t s,
                         MmInfo *info) {
  MmArgs a = {};
  a.a = (const uint8_t *)dgu;
  a.lda = ldd * 2;
  a.b = (const uint8_t *)c.w;
  a.ldb = c.ldw * 2;
  a.m = (int32_t)c.m;
  a.n = (int32_t)c.k;
  a.kd = (int32_t)(2 * c.inter);
  a.y = dx;
  a.ldy = lddx;
  a.otype = QG_O_BF16;
  a.group_m = 4;
  a.counters = c.counters;
  a.partials = (uint64_t *)c.partials;
  using Few = MmCfg<false, kRows, kCols, false, 32, 128, 1, 8, 4, true>;
  if (c.m <= 16) {
    a.halves = (int32_t)ffn_halves(c.m);
    a.m += a.halves;
    return mm_dispatch<Few>(a, kMmPartialBytes, s, info);
  }
  return mm_dispatch<MmCfg<false, kRows, kCols, false, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 4, true>,
                     MmCfg<false, kRows, kCols, false, 64, 128, 2, 4, 4, true>,
                     Few>(a, kMmPartialBytes, s, info);
}

// dW = [dg du]^T x: contraction over the tokens
hipError_t launch_ffn_dw(const FfnCall &c, const void *dgu, int64_t ldd, void *dw, int dw_type, int64_t lddw,
                         hipStream_t s, MmInfo *info) {
  MmArgs a = {};
  a.a = (const uint8_t *)dgu;
  a.lda = ldd * 2;
  a.b = (const uint8_t *)c.x;
  a.ldb = c.ldx * 2;
  a.m = (int32_t)(2 * c.inter);
  a.n = (int32_t)c.k;
  a.kd = (int32_t)c.m;
  a.y = dw;
  a.ldy = lddw;
  a.otype = dw_type;
  a.group_m = 4;
  a.counters = c.counters;
  a.partials = (uint64_t *)c.partials;
  a.halves = (int32_t)ffn_halves(c.m);
  a.kd += a.halves;
  return mm_dispatch<MmCfg<false, kCols, kCols, false, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 4, true>>(a, kMmPartialBytes, s, info);
}

hipError_t launch_ffn_zero(void *p, int64_t ld_bytes, int64_t row_bytes, int64_t rows, hipStream_t s) {
  hipLaunchKernelGGL(ffn_zero_kernel, dim3((unsigned)std::min<int64_t>(rows, 4096)), dim3(256), 0, s, (uint8_t *)p,
                     ld_bytes, row_bytes, rows);
  return hipGetLastError();
}

}  // namespace qg
