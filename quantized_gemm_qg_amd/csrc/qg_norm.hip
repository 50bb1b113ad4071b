// Root-mean-square norm with the residual's addition, to bf16 and to 8 bits with
// scales, and its backward pass:
//   s = x + residual (rounded to the residual's type where there is one)
//   r = 1 / sqrt(mean_j s_j^2 + eps),  y_j = (s_j w_j) r
//   ds_j = r (g_j - s_j r^2 mean(g s)) + dsum_j  with g = dy w,
//   dw_j = sum over the rows of dy_j s_j r
// One pass over the data: a row is held in registers between its sums and its
// outputs, by a wave (rows of up to 1024 values) or by a workgroup.  y is (s w) r
// in that order, so the largest |y| of a row is r max |s w| exactly, and one
// reduction gives the sum of squares and the per-token scale.  Sums are fp32; y
// is rounded once, to bf16 and from fp32 to the codes.
// Bound by HBM from about 100 MB on: 16384 x 4096 with the residual, bf16 and MXFP8 out
// 117 us (606 MB, 5.2 TB/s); 4096 x 4096 forward 26 and backward 25 us; below, by a
// launch and two memory latencies (one row of 4096 3.5 us, 1001 x 2080 8.1 us).  Rows of
// other lengths, bf16 with the residual, 268 MB, TB/s forward and backward with dw (a
// copy 5.2): 256 4.8 and 3.1, 512 and 1024 5.0 and 4.8, 2048 5.1 and 4.2, 4096 5.3 and
// 4.7, 8192 5.4 and 4.4, 12288 5.2 and 4.1, 14336 4.5 and 3.8, 16384 4.3 and 3.8, 32768 and
// 65536 3.8 and 2.2.  Above 12288 values a workgroup of 13 to 16 waves has a CU for
// itself and asks for nothing of the next row while it stores one; longer rows are read
// twice, and their backward kernels spill 17 (bf16) and 34 (fp32) registers.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_quant.h"

namespace qg {

namespace {

// smallest scale of codes: below, a / 127 and a / 448 would lose their own bits
constexpr float kLeastScale = 0x1p-126f;

// 8 consecutive values of a row as loaded, and as fp32
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *row, int64_t c) {
    w[0] = ((const u32x4 *)row)[F32 ? 2 * c : c];
    if constexpr (F32) w[1] = ((const u32x4 *)row)[2 * c + 1];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i / 4][i % 4]);
    } else {
      unpack8(w[0], v);
    }
  }
};
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}
template <bool F32>
__device__ __forceinline__ void store8(void *row, int64_t c, const float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      ((u32x4 *)row)[2 * c + h] = u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                        __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
  } else {
    ((u32x4 *)row)[c] = pack8(v);
  }
}

// e4m3 codes of 8 values times 1 / scale
__device__ __forceinline__ uint2 e4m3_8(const float (&v)[8], float inv) {
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    c[h] = e4m3_pair(v[4 * h] * inv, v[4 * h + 1] * inv) | (e4m3_pair(v[4 * h + 2] * inv, v[4 * h + 3] * inv) << 16);
  return uint2{c[0], c[1]};
}

// Sum of a and, MAX, maximum of b (else its sum) over the threads of a row.
// red: 2 x 2 x 16 floats, of which rows in turn use one half each: the barrier of
// one row lies between another's reads and the next writes of its half.
template <bool WAVE, bool MAX>
__device__ __forceinline__ void team_reduce(float &a, float &b, float (*red)[2][16], int half) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    a += __shfl_xor(a, off);
    const float o = __shfl_xor(b, off);
    b = MAX ? fmaxf(b, o) : b + o;
  }
  if constexpr (!WAVE) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[half][0][wave] = a;
      red[half][1][wave] = b;
    }
    __syncthreads();
    a = red[half][0][0];
    b = red[half][1][0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) {
      a += red[half][0][w];
      b = MAX ? fmaxf(b, red[half][1][w]) : b + red[half][1][w];
    }
  }
}

}  // namespace

// The threads of a row (a wave, or TEAMS 1: the workgroup) hold VEC x 8 values each
// (rows of 4096 on 512 threads with 8 values each: one row 3.3 us instead of 3.5, 333
// rows of 5128 6.8 instead of 6.2);
// LONG: what lies behind them is read twice.  RES: 0 no residual and no sum, 1 bf16,
// 2 fp32.
template <int TEAMS, int VEC, bool LONG, bool XF32, int RES>
__global__ __launch_bounds__(TEAMS > 1 ? 64 * TEAMS : 1024) void rmsnorm_kernel(NormArgs a) {
  __shared__ float red[2][2][16];
  const int team_size = TEAMS > 1 ? 64 : blockDim.x;
  const int t = TEAMS > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int k8 = (int)(a.k / 8);
  u32x4 wv[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) wv[v] = ((const u32x4 *)a.w)[min(v * team_size + t, k8 - 1)];
  int half = 0;
  for (int64_t row = blockIdx.x * TEAMS + (TEAMS > 1 ? threadIdx.x >> 6 : 0); row < a.rows;
       row += (int64_t)gridDim.x * TEAMS, half ^= 1) {
    const uint8_t *xr = (const uint8_t *)a.x + row * a.ldx * (XF32 ? 4 : 2);
    const uint8_t *rr = (const uint8_t *)a.res + row * a.ldr * (RES == 2 ? 4 : 2);
    uint8_t *sr = (uint8_t *)a.sum + row * a.lds * (RES == 2 ? 4 : 2);
    // s of chunk c, kept in `sum` (a caller may want it, later passes of a long row do)
    auto total = [&](int c, bool ok, const Raw8<XF32> &x, const Raw8<RES == 2> &res, float (&s)[8]) {
      x.values(s);
      if constexpr (RES != 0) {
        if (a.res) {
          float o[8];
          res.values(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] += o[i];
        }
        if constexpr (RES == 1) unpack8(pack8(s), s);
        if (a.sum && ok) store8<RES == 2>(sr, c, s);
      }
    };
    float ss = 0.f, most = 0.f;
    auto count = [&](bool ok, const float (&s)[8], const u32x4 &w) {
      float wf[8];
      unpack8(w, wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = ok ? s[i] : 0.f;
        ss = __builtin_fmaf(v, v, ss);
        most = fmaxf(most, fabsf(v * wf[i]));
      }
    };
    Raw8<XF32> x[VEC];
    Raw8<RES == 2> res[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int c = min(v * team_size + t, k8 - 1);
      x[v].load(xr, c);
      if constexpr (RES != 0)
        if (a.res) res[v].load(rr, c);
    }
    float s[VEC][8];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int c = v * team_size + t;
      total(c, c < k8, x[v], res[v], s[v]);
      count(c < k8, s[v], wv[v]);
    }
    // a chunk behind the registers; again: from what the first time left in `sum`,
    // which may be x's or the residual's own memory
    auto later = [&](int c, bool again, float (&s8)[8]) {
      if constexpr (RES != 0) {
        if (again && a.sum) {
          Raw8<RES == 2> kept;
          kept.load(sr, c);
          kept.values(s8);
          return;
        }
      }
      Raw8<XF32> xl;
      Raw8<RES == 2> rl;
      xl.load(xr, c);
      if constexpr (RES != 0)
        if (a.res) rl.load(rr, c);
      total(c, !again, xl, rl, s8);
    };
    if constexpr (LONG)
      for (int c = VEC * team_size + t; c < k8; c += team_size) {
        float s8[8];
        later(c, false, s8);
        count(true, s8, ((const u32x4 *)a.w)[c]);
      }
    team_reduce<(TEAMS > 1), true>(ss, most, red, half);
    const float r = 1.f / sqrtf(ss / (float)a.k + a.eps);
    most *= r;
    float scale = 1.f;
    if (most > 0.f && a.q_type == QG_A_INT8_TOKEN) scale = fmaxf(most / 127.f, kLeastScale);
    if (most > 0.f && a.q_type == QG_A_FP8_TOKEN) scale = fmaxf(most / 448.f, kLeastScale);
    if (t == 0 && (a.q_type == QG_A_INT8_TOKEN || a.q_type == QG_A_FP8_TOKEN)) ((float *)a.qs)[row] = scale;
    const float inv_scale = 1.f / scale;
    uint8_t *qr = a.q + row * a.ldq;
    // outputs of chunk c (every lane of the wave comes here: blocks are reduced over lanes)
    auto emit = [&](int c, bool ok, const float (&s8)[8], const u32x4 &w) {
      float y[8];
      unpack8(w, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (s8[i] * y[i]) * r;
      if (a.y && ok) ((u32x4 *)(a.y + row * a.ldy))[c] = pack8(y);
      if (a.q_type == QG_A_BF16) return;
      uint2 codes;
      if (a.q_type == QG_A_INT8_TOKEN) {
        uint32_t c8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c8[i] = (uint32_t)(int)rintf(y[i] * inv_scale) & 255u;
        codes = uint2{c8[0] | c8[1] << 8 | c8[2] << 16 | c8[3] << 24, c8[4] | c8[5] << 8 | c8[6] << 16 | c8[7] << 24};
      } else if (a.q_type == QG_A_FP8_TOKEN) {
        codes = e4m3_8(y, inv_scale);
      } else {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
        m = ok ? m : 0.f;
        if (a.q_type == QG_A_FP8_BLOCK) {  // 128 values: 16 lanes
#pragma unroll
          for (int off = 1; off < 16; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
          const float bs = m > 0.f ? fmaxf(m / 448.f, kLeastScale) : 1.f;
          codes = e4m3_8(y, 1.f / bs);
          if (ok && (t & 15) == 0) ((float *)a.qs)[row * ((k8 + 15) / 16) + c / 16] = bs;
        } else {  // MXFP8, 32 values: 4 lanes
          const int e = mx_block_exp(quad_max(__float_as_uint(m)));
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
          codes = e4m3_8(y, inv);
          if (ok && (t & 3) == 0) ((uint8_t *)a.qs)[row * (k8 / 4) + c / 4] = (uint8_t)(e + 127);
        }
      }
      if (ok) *(uint2 *)(qr + 8 * (int64_t)c) = codes;
    };
#pragma unroll
    for (int v = 0; v < VEC; ++v) emit(v * team_size + t, v * team_size + t < k8, s[v], wv[v]);
    if constexpr (LONG)
      for (int c0 = VEC * team_size; c0 < k8; c0 += team_size) {
        const int c = c0 + t;
        float s8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        u32x4 w = {0u, 0u, 0u, 0u};
        if (c < k8) {
          later(c, true, s8);
          w = ((const u32x4 *)a.w)[c];
        }
        emit(c, c < k8, s8, w);
      }
  }
}

// Backward pass: every workgroup sums dy s r of its rows, in registers, and leaves
// one row of `partial` ([gridDim.x][k] fp32), which rmsnorm_dw_kernel adds up in
// order.  LONG: what lies behind the registers is summed in `partial` itself.
template <int TEAMS, int VEC, bool LONG, bool SF32>
__global__ __launch_bounds__(TEAMS > 1 ? 64 * TEAMS : 1024) void rmsnorm_backward_kernel(NormBackArgs a) {
  __shared__ float red[2][2][16];
  __shared__ float join[TEAMS > 1 ? TEAMS * VEC * 64 * 8 : 1];
  const int team_size = TEAMS > 1 ? 64 : blockDim.x;
  const int t = TEAMS > 1 ? threadIdx.x & 63 : threadIdx.x, team = TEAMS > 1 ? threadIdx.x >> 6 : 0;
  const int k8 = (int)(a.k / 8);
  constexpr int EL = SF32 ? 4 : 2;
  float *mine = a.partial ? a.partial + (int64_t)blockIdx.x * a.k : nullptr;
  u32x4 wv[VEC];
  float dw[VEC][8];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    wv[v] = ((const u32x4 *)a.w)[min(v * team_size + t, k8 - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  int half = 0;
  bool first = true;
  for (int64_t row = (int64_t)blockIdx.x * TEAMS + team; row < a.rows;
       row += (int64_t)gridDim.x * TEAMS, half ^= 1, first = false) {
    const uint8_t *sr = (const uint8_t *)a.s + row * a.lds * EL;
    const uint16_t *dyr = a.dy + row * a.lddy;
    const uint8_t *dsr = (const uint8_t *)a.dsum + row * a.ldds * EL;
    uint8_t *dxr = (uint8_t *)a.dx + row * a.lddx * EL;
    Raw8<SF32> s[VEC], ds[VEC];
    Raw8<false> dy[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int c = min(v * team_size + t, k8 - 1);
      s[v].load(sr, c);
      dy[v].load(dyr, c);
      if (a.dsum) ds[v].load(dsr, c);
    }
    float ss = 0.f, gs = 0.f;
    auto count = [&](bool ok, const Raw8<SF32> &s8, const Raw8<false> &d8, const u32x4 &w) {
      float sf[8], df[8], wf[8];
      s8.values(sf);
      d8.values(df);
      unpack8(w, wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = ok ? sf[i] : 0.f;
        ss = __builtin_fmaf(v, v, ss);
        gs = __builtin_fmaf(ok ? df[i] * wf[i] : 0.f, v, gs);
      }
    };
#pragma unroll
    for (int v = 0; v < VEC; ++v) count(v * team_size + t < k8, s[v], dy[v], wv[v]);
    if constexpr (LONG)
      for (int c = VEC * team_size + t; c < k8; c += team_size) {
        Raw8<SF32> sl;
        Raw8<false> dl;
        sl.load(sr, c);
        dl.load(dyr, c);
        count(true, sl, dl, ((const u32x4 *)a.w)[c]);
      }
    team_reduce<(TEAMS > 1), false>(ss, gs, red, half);
    const float r = 1.f / sqrtf(ss / (float)a.k + a.eps);
    const float back = r * r * (gs / (float)a.k);
    auto emit = [&](int c, bool ok, const Raw8<SF32> &s8, const Raw8<false> &d8, const Raw8<SF32> &ds8, const u32x4 &w,
                    float (&sum)[8]) {
      float sf[8], df[8], wf[8], of[8], out[8];
      s8.values(sf);
      d8.values(df);
      unpack8(w, wf);
      if (a.dsum) ds8.values(of);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[i] = __builtin_fmaf(df[i], sf[i] * r, sum[i]);
        out[i] = r * __builtin_fmaf(-sf[i], back, df[i] * wf[i]);
        if (a.dsum) out[i] += of[i];
      }
      if (a.dx && ok) store8<SF32>(dxr, c, out);
    };
#pragma unroll
    for (int v = 0; v < VEC; ++v) emit(v * team_size + t, v * team_size + t < k8, s[v], dy[v], ds[v], wv[v], dw[v]);
    if constexpr (LONG)
      for (int c = VEC * team_size + t; c < k8; c += team_size) {
        Raw8<SF32> sl, ol;
        Raw8<false> dl;
        sl.load(sr, c);
        dl.load(dyr, c);
        if (a.dsum) ol.load(dsr, c);
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (mine && !first) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = mine[8 * (int64_t)c + i];
        }
        emit(c, true, sl, dl, ol, ((const u32x4 *)a.w)[c], sum);
        if (mine) store8<true>(mine, c, sum);
      }
  }
  if (!mine) return;
  if constexpr (TEAMS > 1) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) join[((team * VEC + v) * 8 + i) * 64 + t] = dw[v][i];
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        for (int o = 1; o < TEAMS; ++o) dw[v][i] += join[((o * VEC + v) * 8 + i) * 64 + t];
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (v * team_size + t < k8) store8<true>(mine, v * team_size + t, dw[v]);
}

// dw from `parts` rows of fp32 sums: 8 lanes side by side, 4 columns each (a cache
// line), 32 lanes along the parts, joined in order.  512 parts of 4096: 4 us (10 with
// 16 lanes side by side and 64 workgroups).
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float *partial, int parts, int64_t k, void *dw, bool f32) {
  __shared__ f32x4 join[32][8];
  const int side = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 32 + 4 * side;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (c < k) {
#pragma unroll 8
    for (int p = part; p < parts; p += 32) sum += *(const f32x4 *)(partial + p * k + c);
  }
  join[part][side] = sum;
  __syncthreads();
  if (part != 0 || c >= k) return;
#pragma unroll
  for (int o = 1; o < 32; ++o) sum += join[o][side];
  if (f32)
    *(f32x4 *)((float *)dw + c) = sum;
  else
    *(uint2 *)((uint16_t *)dw + c) = uint2{bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
}

namespace {

// Calls go(waves, rows per workgroup, vec, long) with the shape for rows of k
// values: a wave each up to 1024 values, else the fewest waves that hold the row.
template <typename F>
void norm_shape(int64_t k, F &&go) {
  auto call = [&](int waves, auto rows, auto vec, auto is_long) { go(waves, rows, vec, is_long); };
  using std::false_type;
  using std::integral_constant;
  if (k <= 512)
    call(4, integral_constant<int, 4>(), integral_constant<int, 1>(), false_type());
  else if (k <= 1024)
    call(4, integral_constant<int, 4>(), integral_constant<int, 2>(), false_type());
  else if (k <= 2048)
    call((int)((k + 511) / 512), integral_constant<int, 1>(), integral_constant<int, 1>(), false_type());
  else if (k <= 16384)
    call((int)((k + 1023) / 1024), integral_constant<int, 1>(), integral_constant<int, 2>(), false_type());
  else
    call(16, integral_constant<int, 1>(), integral_constant<int, 2>(), std::true_type());
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs &a, bool x_f32, int res, hipStream_t s) {
  norm_shape(a.k, [&](int waves, auto teams, auto vec, auto is_long) {
    constexpr int N = decltype(teams)::value, V = decltype(vec)::value;
    constexpr bool L = decltype(is_long)::value;
    const unsigned grid = (unsigned)std::min<int64_t>((a.rows + N - 1) / N, 256 * 16);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * waves), 0, s, a); };
    if (x_f32)
      res == 0   ? go(rmsnorm_kernel<N, V, L, true, 0>)
      : res == 1 ? go(rmsnorm_kernel<N, V, L, true, 1>)
                 : go(rmsnorm_kernel<N, V, L, true, 2>);
    else
      res == 0   ? go(rmsnorm_kernel<N, V, L, false, 0>)
      : res == 1 ? go(rmsnorm_kernel<N, V, L, false, 1>)
                 : go(rmsnorm_kernel<N, V, L, false, 2>);
  });
  return hipGetLastError();
}

// Rows of `partial`: one per workgroup, at most 512 and at most 64 MB of them.  (The
// grid is the same without dw.  512 workgroups of one-wave rows leave too little in
// flight below 512 values, see the rates above.)
int64_t rmsnorm_back_parts(int64_t rows, int64_t k) {
  const int64_t most = std::max<int64_t>((64ll << 20) / (4 * k), 1), teams = k <= 1024 ? 4 : 1;
  return std::min<int64_t>(std::min<int64_t>((rows + teams - 1) / teams, 512), most);
}

hipError_t launch_rmsnorm_backward(const NormBackArgs &a, bool s_f32, void *dw, bool dw_f32, hipStream_t s) {
  const unsigned parts = (unsigned)rmsnorm_back_parts(a.rows, a.k);
  if (a.rows > 0) {
    norm_shape(a.k, [&](int waves, auto teams, auto vec, auto is_long) {
      constexpr int N = decltype(teams)::value, V = decltype(vec)::value;
      constexpr bool L = decltype(is_long)::value;
      auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(parts), dim3(64 * waves), 0, s, a); };
      s_f32 ? go(rmsnorm_backward_kernel<N, V, L, true>) : go(rmsnorm_backward_kernel<N, V, L, false>);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dw)
    hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)((a.k + 31) / 32)), dim3(256), 0, s, a.partial,
                       a.rows > 0 ? (int)parts : 0, a.k, dw, dw_f32);
  return hipGetLastError();
}

}  // namespace qg
