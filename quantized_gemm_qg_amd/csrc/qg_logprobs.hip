// Log probabilities of given tokens, with the entropy, the token's rank and the
// top alternatives, and the gradient of the logits.  Per row of logits l, with
// M = max l, d = c (l - M) (c > 0), S = sum exp(d), T = sum exp(d) d:
//   logp = d_t - log S,  H = log S - T / S,  rank = #{l > l_t}
//   dl = c (g (1_t - p) - e p (log p + H)),  p = exp(d - log S)
// (l - M before the product with c: masks of the type's lowest value would
// overflow in c l, and a row of them would lose its maximum.)
// A logit of -inf is a masked token: probability 0, never an alternative.  A
// row of nothing else has logp -inf, entropy 0 and gradient 0.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"

namespace qg {

namespace {

__device__ __forceinline__ float logit_at(const void *row, bool f32, int64_t i) {
  return f32 ? ((const float *)row)[i] : bf16_bits_to_f32(((const uint16_t *)row)[i]);
}

// Order of alternatives as one key: larger logits first, equal ones by lower
// id (-0 equals +0); 0 for masked and NaN logits.
__device__ __forceinline__ uint64_t alt_key(float l, uint32_t id) {
  if (!(l > -__builtin_inff())) return 0;
  uint32_t u = __float_as_uint(l + 0.f);
  if (u == 0x80000000u) u = 0;
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (0xFFFFFFFFu - id);
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T *lds, F &&op) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v = op(v, __shfl_xor(v, off));
  if (lane == 0) lds[wave] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < waves; ++w) v = op(v, lds[w]);
  __syncthreads();
  return v;
}

}  // namespace

__global__ __launch_bounds__(256) void logprobs_kernel(LogprobArgs a) {
  __shared__ uint64_t lds[4];
  float *ldf = (float *)lds;
  const float ninf = -__builtin_inff();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t *l = (const uint8_t *)a.logits + row * a.ldl * (a.f32 ? 4 : 2);
    float m = ninf;
    for (int64_t i = threadIdx.x; i < a.vocab; i += blockDim.x) m = fmaxf(m, logit_at(l, a.f32, i));
    m = block_reduce(m, ldf, [](float x, float y) { return fmaxf(x, y); });
    const bool empty = m == ninf;
    const float zm = empty ? 0.f : m;
    const int tok = a.tokens ? a.tokens[row] : -1;
    const bool in = tok >= 0 && tok < a.vocab;
    const float lt = in ? logit_at(l, a.f32, tok) : 0.f;
    float s = 0.f, t = 0.f;
    int above = 0;
    for (int64_t i = threadIdx.x; i < a.vocab; i += blockDim.x) {
      const float x = logit_at(l, a.f32, i);
      const float d = (x - zm) * a.scale, e = __expf(d);
      s += e;
      t += e != 0.f ? e * d : 0.f;
      above += x > lt;
    }
    auto add = [](float x, float y) { return x + y; };
    s = block_reduce(s, ldf, add);
    t = block_reduce(t, ldf, add);
    above = block_reduce(above, (int *)lds, [](int x, int y) { return x + y; });
    const float log_s = empty ? ninf : logf(s);
    if (threadIdx.x == 0) {
      if (a.logp) a.logp[row] = in ? (empty ? ninf : (lt - zm) * a.scale - log_s) : __builtin_nanf("");
      if (a.rank) a.rank[row] = in ? above : -1;
      if (a.entropy) a.entropy[row] = empty ? 0.f : log_s - t / s;
      if (a.stats) {
        a.stats[2 * row] = zm;
        a.stats[2 * row + 1] = log_s;
      }
    }
    uint64_t last = ~0ull;
    for (int j = 0; j < a.top; ++j) {
      uint64_t best = 0;
      for (int64_t i = threadIdx.x; i < a.vocab; i += blockDim.x) {
        const uint64_t k = alt_key(logit_at(l, a.f32, i), (uint32_t)i);
        if (k < last && k > best) best = k;
      }
      best = block_reduce(best, lds, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
      if (threadIdx.x == 0) {
        const int id = best ? (int)(0xFFFFFFFFu - (uint32_t)best) : -1;
        if (a.top_ids) a.top_ids[row * a.top + j] = id;
        if (a.top_logp) a.top_logp[row * a.top + j] = best ? (logit_at(l, a.f32, id) - zm) * a.scale - log_s : ninf;
      }
      last = best;
    }
  }
}

__global__ __launch_bounds__(256) void logprobs_backward_kernel(LogprobArgs a) {
  const float ninf = -__builtin_inff();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t *l = (const uint8_t *)a.logits + row * a.ldl * (a.f32 ? 4 : 2);
    uint8_t *dl = (uint8_t *)a.dlogits + row * a.lddl * (a.f32 ? 4 : 2);
    const float zm = a.stats[2 * row], log_s = a.stats[2 * row + 1];
    const bool empty = log_s == ninf;
    const int tok = a.tokens ? a.tokens[row] : -1;
    const bool in = tok >= 0 && tok < a.vocab;
    const float g = a.dlogp && in ? a.dlogp[row] : 0.f;
    const float e = a.dentropy ? a.dentropy[row] : 0.f;
    const float h = a.dentropy ? a.entropy[row] : 0.f;
    for (int64_t i = threadIdx.x; i < a.vocab; i += blockDim.x) {
      const float lq = (logit_at(l, a.f32, i) - zm) * a.scale - log_s;
      const float p = __expf(lq);
      float v = -g * p;
      if (p != 0.f) v -= e * p * (lq + h);
      if (i == tok) v += g;
      v = empty ? 0.f : v * a.scale;
      if (a.f32)
        ((float *)dl)[i] = v;
      else
        ((uint16_t *)dl)[i] = (uint16_t)bf16_rne(v);
    }
  }
}

uint64_t logprobs_ws_bytes(int64_t, int64_t, int) { return 0; }

hipError_t launch_logprobs(const LogprobArgs &a, void *, hipStream_t s) {
  hipLaunchKernelGGL(logprobs_kernel, dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(logprobs_backward_kernel, dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qg
