// Softmax cross entropy of hidden states x [m][k] against a head's weights W
// [vocab][k], without logits in memory, and its gradients:
//   z = scale x W^T,  lse_r = log sum_v exp z_rv,  loss_r = lse_r - z[r][t_r]
//   d_rv = dloss_r (exp(z_rv - lse_r) - 1{v = t_r}),  dx = scale d W,  dW = scale d^T x
// Forward: the tiled product keeps, per row and tile, the largest logit and the sum
// of exponentials; a small kernel joins them.  Backward: pieces of the vocabulary
// whose d (bf16) stays in the last-level cache, per piece the product again with d
// as its epilogue, then one product for dx (summed over the pieces in fp32) and one
// for the piece's rows of dW.
// d is rounded to bf16 because the matrix cores take bf16.  So that the target's
// entry, the largest of its row, is rounded as little as possible, d holds
// dloss / c with c the largest |dloss|: under a mean over tokens these weights are
// exactly 1 and the entries near -1; c comes back in the products' epilogues.  With
// few tokens (dx 16, dW 32) single entries decide: there d is the sum of two bf16
// parts, as in the gated block's backward pass.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"

namespace qg {

// lse and loss from the statistics of every tile of columns ([tiles][m] of largest
// logit and sum): 16 rows side by side, 64 lanes along the tiles.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float2 *stats, const float *at_target, int tiles, int m,
                                                         int vocab, const int32_t *targets, float scale, float *loss,
                                                         float *lse) {
  __shared__ float2 join[64][16];
  const int side = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int row = blockIdx.x * 16 + side;
  const float base2 = scale * 1.4426950408889634f;
  float most = -INFINITY, sum = 0.f;
  auto add = [&](const float2 &v) {
    const float big = fmaxf(most, v.x), from = big == -INFINITY ? 0.f : big;
    sum = sum * __builtin_amdgcn_exp2f((most - from) * base2) + v.y * __builtin_amdgcn_exp2f((v.x - from) * base2);
    most = big;
  };
  if (row < m) {
    constexpr int GO = 8;  // loads out together
    for (int t0 = part; t0 < tiles; t0 += 64 * GO) {
      float2 v[GO];
#pragma unroll
      for (int g = 0; g < GO; ++g) v[g] = stats[(int64_t)min(t0 + 64 * g, tiles - 1) * m + row];
#pragma unroll
      for (int g = 0; g < GO; ++g)
        if (t0 + 64 * g < tiles) add(v[g]);
    }
  }
  join[part][side] = float2{most, sum};
  __syncthreads();
  if (part != 0 || row >= m) return;
  for (int o = 1; o < 64; ++o) add(join[o][side]);
  const float log_sum = logf(sum);
  // (nothing but NaN logits: `most` is -inf and the sum NaN)
  if (lse) lse[row] = __builtin_fmaf(scale, most, log_sum);
  if (loss) {
    const int t = targets[row];
    // (an ignored row's loss is 0; scale (largest - target's) is exact where the two are near)
    loss[row] = t >= 0 && t < vocab ? __builtin_fmaf(scale, most - at_target[row], log_sum) : 0.f;
  }
}

// Row weights dloss / c (0 for ignored rows) and alpha = scale c, c the largest
// |dloss| of the rows that count (1 where that is 0 or not finite).
__global__ __launch_bounds__(1024) void xent_weights_kernel(const float *dloss, const int32_t *targets, int m, int vocab,
                                                            float scale, float *weight, float *alpha) {
  __shared__ float wave_max[16];
  float most = 0.f;
  for (int r = threadIdx.x; r < m; r += 1024)
    if (targets[r] >= 0 && targets[r] < vocab) most = fmaxf(most, fabsf(dloss[r]));
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) most = fmaxf(most, __shfl_xor(most, off));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) most = fmaxf(most, wave_max[w]);
  const float c = most >= 0x1p-126f && most < INFINITY ? most : 1.f;
  for (int r = threadIdx.x; r < m; r += 1024)
    weight[r] = targets[r] >= 0 && targets[r] < vocab ? dloss[r] / c : 0.f;
  if (threadIdx.x == 0) alpha[0] = scale * c;
}

static int64_t xent_halves(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 0; }
int64_t xent_d_rows(int64_t m) { return m + xent_halves(m); }

// Columns of a piece: d takes up to 128 MB, half of the last-level cache, and at
// least 8192 columns (the products over a piece would be short).
int64_t xent_piece(int64_t m, int64_t vocab) {
  int64_t most = (64ll << 20) / std::max<int64_t>(m, 1);
  most = std::min<int64_t>(std::max<int64_t>(most / 256 * 256, 8192), 1 << 20);
  const int64_t pieces = (vocab + most - 1) / most;
  return std::min<int64_t>(((vocab + pieces - 1) / pieces + 255) / 256 * 256, (vocab + 63) / 64 * 64);
}

// (few tokens, whose d has two parts: one shape)
template <int EPI>
using XentFew = MmCfg<false, kRows, kRows, false, 32, 128, 1, 8, 4, true, EPI>;
template <int EPI>
static hipError_t xent_logits(const MmArgs &a, hipStream_t s, MmInfo *info) {
  return mm_dispatch<MmCfg<false, kRows, kRows, false, 256, 256, 4, 2, 2, false, EPI>,
                     MmCfg<false, kRows, kRows, false, 192, 256, 4, 2, 2, false, EPI>,
                     MmCfg<false, kRows, kRows, false, 128, 128, 4, 2, 2, true, EPI>,
                     MmCfg<false, kRows, kRows, false, 128, 128, 4, 2, 4, true, EPI>,
                     MmCfg<false, kRows, kRows, false, 64, 128, 2, 4, 4, true, EPI>,
                     XentFew<EPI>>(a, kMmPartialBytes, s, info);
}

static MmArgs xent_args(const XentCall &c, int64_t first, int64_t columns) {
  MmArgs a = {};
  a.a = (const uint8_t *)c.x;
  a.lda = c.ldx * 2;
  a.b = (const uint8_t *)c.w + first * c.ldw * 2;
  a.ldb = c.ldw * 2;
  a.m = (int32_t)c.m;
  a.n = (int32_t)columns;
  a.kd = (int32_t)c.k;
  a.group_m = 4;
  a.counters = c.counters;
  a.partials = (uint64_t *)c.partials;
  a.targets = c.targets;
  a.first_token = (int32_t)first;
  a.scale = c.scale;
  return a;
}

// (info: nothing is launched, see mm_dispatch)
hipError_t launch_xent(const XentCall &c, hipStream_t s, MmInfo *info) {
  MmArgs a = xent_args(c, 0, c.vocab);
  a.stats = c.stats;
  a.at_target = c.at_target;
  MmInfo choice;
  hipError_t e = xent_logits<kXentStats>(a, nullptr, &choice);
  if (info) *info = choice;
  if (info || e != hipSuccess) return e;
  e = xent_logits<kXentStats>(a, s, nullptr);
  if (e != hipSuccess) return e;
  const int tiles = (int)((c.vocab + choice.bn - 1) / choice.bn);
  hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)((c.m + 15) / 16)), dim3(1024), 0, s, (const float2 *)c.stats,
                     c.at_target, tiles, (int)c.m, (int)c.vocab, c.targets, c.scale, c.loss, c.lse);
  return hipGetLastError();
}

hipError_t launch_xent_weights(const XentCall &c, const float *dloss, hipStream_t s) {
  hipLaunchKernelGGL(xent_weights_kernel, dim3(1), dim3(1024), 0, s, dloss, c.targets, (int)c.m, (int)c.vocab, c.scale,
                     c.weight, c.alpha);
  return hipGetLastError();
}

// d of one piece
hipError_t launch_xent_d(const XentCall &c, int64_t first, int64_t columns, hipStream_t s, MmInfo *info) {
  MmArgs a = xent_args(c, first, columns);
  a.lse = c.lse;
  a.row_weight = c.weight;
  a.y = c.d;
  a.ldy = c.ldd;
  a.otype = QG_O_BF16;
  a.halves = (int32_t)xent_halves(c.m);
  if (a.halves > 0) return mm_dispatch<XentFew<kXentGrad>>(a, kMmPartialBytes, s, info);
  return xent_logits<kXentGrad>(a, s, info);
}

// dx from one piece: out (bf16 or fp32) = alpha d W (+ add)
hipError_t launch_xent_dx(const XentCall &c, int64_t first, int64_t columns, const float *add, int64_t ldadd, void *out,
                          int out_type, int64_t ldout, hipStream_t s, MmInfo *info) {
  MmArgs a = xent_args(c, first, columns);
  a.a = (const uint8_t *)c.d;
  a.lda = c.ldd * 2;
  a.n = (int32_t)c.k;
  a.kd = (int32_t)columns;
  a.alpha = c.alpha;
  a.add = add;
  a.ldadd = ldadd;
  a.y = out;
  a.otype = out_type;
  a.ldy = ldout;
  using Few = MmCfg<false, kRows, kCols, false, 32, 128, 1, 8, 4, true, kScaled>;
  if (c.m <= 16) {
    a.halves = (int32_t)xent_halves(c.m);
    a.m += a.halves;
    return mm_dispatch<Few>(a, kMmPartialBytes, s, info);
  }
  return mm_dispatch<MmCfg<false, kRows, kCols, false, 256, 256, 4, 2, 2, false, kScaled>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 2, true, kScaled>,
                     MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 4, true, kScaled>,
                     MmCfg<false, kRows, kCols, false, 64, 128, 2, 4, 4, true, kScaled>, Few>(a, kMmPartialBytes, s, info);
}

// rows of dW of one piece
hipError_t launch_xent_dw(const XentCall &c, int64_t first, int64_t columns, void *dw, int dw_type, int64_t lddw,
                          hipStream_t s, MmInfo *info) {
  MmArgs a = xent_args(c, first, columns);
  a.a = (const uint8_t *)c.d;
  a.lda = c.ldd * 2;
  a.b = (const uint8_t *)c.x;
  a.ldb = c.ldx * 2;
  a.m = (int32_t)columns;
  a.n = (int32_t)c.k;
  a.alpha = c.alpha;
  a.y = (uint8_t *)dw + first * lddw * (dw_type == QG_O_F32 ? 4 : 2);
  a.otype = dw_type;
  a.ldy = lddw;
  a.halves = (int32_t)xent_halves(c.m);
  a.kd = (int32_t)c.m + a.halves;
  return mm_dispatch<MmCfg<false, kCols, kCols, false, 256, 256, 4, 2, 2, false, kScaled>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 2, true, kScaled>,
                     MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 4, true, kScaled>>(a, kMmPartialBytes, s, info);
}

}  // namespace qg
