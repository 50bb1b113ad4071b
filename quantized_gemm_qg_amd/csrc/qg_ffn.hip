// Gated feed-forward block in bf16, forward and backward:
//   g = x Wg^T, u = x Wu^T, h = act(g) u
//   du = dh act(g), dg = dh u act'(g), dx = dg Wg + du Wu, dW = [dg du]^T x
// The forward is one launch (both projections, the activation and the
// product, the pre-activations saved on request); the backward is one
// elementwise pass that leaves [dg du] in bf16 and one product per gradient.
// [dg du] is rounded to bf16 once because the matrix cores take bf16 operands
// (fp32 ones run at 1/16 of the rate): the rounding errors of its elements are
// independent, so each gradient's relative error grows from the output
// rounding's 1.7e-3 (2-norm) to sqrt(2) times that.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"
#include "qg_rows.h"

namespace qg {

// [dg du] ([m][ldd] bf16, ldd >= 2 inter, zeros from 2 inter to ldd) from the
// pre-activations and dh, 4 consecutive elements of a row per thread.  One
// pass, bound by its bytes.
template <bool F32>
__global__ __launch_bounds__(256) void ffn_dgu_kernel(const void *gu, int64_t ldgu, const uint16_t *dh, int64_t lddh,
                                                      int64_t inter, int act, uint16_t *dgu, int64_t ldd) {
  typedef f32x4 f32x4_any __attribute__((aligned(4)));
  struct __attribute__((packed, aligned(2))) Half4 {  // 4 bf16 at any element
    uint16_t v[4];
  };
  const int64_t row = blockIdx.y, c = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  uint16_t *d = dgu + row * ldd;
  const uint16_t *t = dh + row * lddh + c;
  if (c >= inter) {
    for (int64_t p = inter + c; p < ldd && p < inter + c + 4; ++p)
      if (p >= 2 * inter) d[p] = 0;
    return;
  }
  const int n = (int)min((int64_t)4, inter - c);
  float g[4], u[4], h[4];
  if (n == 4) {
    const Half4 hv = *(const Half4 *)t;
    if constexpr (F32) {
      const float *p = (const float *)gu + row * ldgu + c;
      const f32x4 gv = *(const f32x4_any *)p, uv = *(const f32x4_any *)(p + inter);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = gv[e], u[e] = uv[e];
    } else {
      const uint16_t *p = (const uint16_t *)gu + row * ldgu + c;
      const Half4 gv = *(const Half4 *)p, uv = *(const Half4 *)(p + inter);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = bf16_bits_to_f32(gv.v[e]), u[e] = bf16_bits_to_f32(uv.v[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = bf16_bits_to_f32(hv.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = min(e, n - 1);
      if constexpr (F32) {
        const float *p = (const float *)gu + row * ldgu + c + k;
        g[e] = p[0], u[e] = p[inter];
      } else {
        const uint16_t *p = (const uint16_t *)gu + row * ldgu + c + k;
        g[e] = bf16_bits_to_f32(p[0]), u[e] = bf16_bits_to_f32(p[inter]);
      }
      h[e] = bf16_bits_to_f32(t[k]);
    }
  }
  Half4 dg, du;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v, dv;
    act_both(g[e], act, &v, &dv);
    dg.v[e] = (uint16_t)bf16_rne(h[e] * u[e] * dv);
    du.v[e] = (uint16_t)bf16_rne(h[e] * v);
  }
  if (n == 4) {
    *(Half4 *)(d + c) = dg;
    *(Half4 *)(d + inter + c) = du;
  } else {
    for (int e = 0; e < n; ++e) {
      d[c + e] = dg.v[e];
      d[inter + c + e] = du.v[e];
    }
    // the padding that this thread's 4 elements reach into
    for (int e = n; e < 4 && inter + c + e < ldd; ++e) d[inter + c + e] = 0;
  }
}

__global__ __launch_bounds__(256) void ffn_zero_kernel(uint8_t *p, int64_t ld_bytes, int64_t row_bytes, int64_t rows) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = 2 * (int64_t)threadIdx.x; c < row_bytes; c += 512) *(uint16_t *)(p + r * ld_bytes + c) = 0;
}

// (bytes: only says what partial tiles the launch needs, see mm_dispatch)
hipError_t launch_ffn_forward(const FfnCall &c, hipStream_t s, uint64_t *bytes) {
  if (bytes) *bytes = 0;
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
  if (bytes && c.m <= 64) return hipSuccess;
  if (c.m <= 16) return launch_rows<false, true, 1, 2, 4, false>(a, s);
  if (c.m <= 32) return launch_rows<false, true, 2, 2, 4, false>(a, s);
  if (c.m <= 64) return launch_rows<false, true, 4, 2, 2, false>(a, s);
  return mm_dispatch<MmCfg<false, kRows, kRows, true, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kRows, kRows, true, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kRows, kRows, true, 128, 128, 4, 2, 4, true>,
                     MmCfg<false, kRows, kRows, true, 64, 128, 2, 4, 4, true>>(a, kMmPartialBytes, s, bytes);
}

hipError_t launch_ffn_dgu(const FfnCall &c, const void *dh, int64_t lddh, void *dgu, int64_t ldd, hipStream_t s) {
  const unsigned gx = (unsigned)((ldd - c.inter + 1023) / 1024);
  for (int64_t r0 = 0; r0 < c.m; r0 += 65535) {
    const unsigned rows = (unsigned)std::min<int64_t>(c.m - r0, 65535);
    auto go = [&](auto kern, int el) {
      hipLaunchKernelGGL(kern, dim3(gx, rows), dim3(256), 0, s,
                         (const void *)((const uint8_t *)c.gu + r0 * c.ldgu * el), c.ldgu,
                         (const uint16_t *)dh + r0 * lddh, lddh, c.inter, c.act, (uint16_t *)dgu + r0 * ldd, ldd);
    };
    c.gu_type == QG_O_F32 ? go(ffn_dgu_kernel<true>, 4) : go(ffn_dgu_kernel<false>, 2);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// dx = [dg du] W: contraction over the 2 inter rows of W
hipError_t launch_ffn_dx(const FfnCall &c, const void *dgu, int64_t ldd, void *dx, int64_t lddx, hipStream_t s,
                         uint64_t *bytes) {
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
  return mm_dispatch<MmCfg<false, kRows, kCols, false, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 4, true>,
                     MmCfg<false, kRows, kCols, false, 64, 128, 2, 4, 4, true>>(a, kMmPartialBytes, s, bytes);
}

// dW = [dg du]^T x: contraction over the tokens
hipError_t launch_ffn_dw(const FfnCall &c, const void *dgu, int64_t ldd, void *dw, int dw_type, int64_t lddw,
                         hipStream_t s, uint64_t *bytes) {
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
  return mm_dispatch<MmCfg<false, kCols, kCols, false, 256, 256, 4, 2, 2, false>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 2, true>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 4, true>>(a, kMmPartialBytes, s, bytes);
}

hipError_t launch_ffn_zero(void *p, int64_t ld_bytes, int64_t row_bytes, int64_t rows, hipStream_t s) {
  hipLaunchKernelGGL(ffn_zero_kernel, dim3((unsigned)std::min<int64_t>(rows, 4096)), dim3(256), 0, s, (uint8_t *)p,
                     ld_bytes, row_bytes, rows);
  return hipGetLastError();
}

}  // namespace qg
