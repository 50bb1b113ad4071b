// Softmax cross entropy of hidden states x [m][k] against a head's weights W
// [vocab][k], without logits in memory, and its gradients:
//   z = scale x W^T,  lse_r = log sum_v exp z_rv,  loss_r = lse_r - z[r][t_r]
//   d_rv = dloss_r (exp(z_rv - lse_r) - 1{v = t_r}),  dx = scale d W,  dW = scale d^T x
// Forward: the tiled product keeps, per row and tile, the largest logit and the sum
// of exponentials; a small kernel joins them.  Backward: pieces of the vocabulary
// whose d (bf16) stays in the last-level cache, per piece the product again with d
// as its epilogue, then one product for dx (summed over the pieces in fp32) and one
// for the piece's rows of dW.  (W does not stay there: up to a few hundred tokens
// have one piece, W is the larger operand and comes from HBM for d and again for dx.)
// d is rounded to bf16 because the matrix cores take bf16.  So that the target's
// entry, the largest of its row, is rounded as little as possible, d holds
// dloss / c with c the largest |dloss|: under a mean over tokens these weights are
// exactly 1 and the entries near -1; c comes back in the products' epilogues.  With
// few tokens (dx 16, dW 32) single entries decide: there d is the sum of two bf16
// parts, as in the gated block's backward pass.
// 4096 tokens of 131072 x 4096: forward 3.15 ms (1.40 PFLOP/s), and per piece of 16384
// tokens d 439 to 458 us (with its exponentials and 134 MB of stores), dx 390 to 417, dW
// 400 to 434.  61 tokens of 100003 x 2048, forward: 95 us, 4.3 TB/s of weights.
#include <hip/hip_runtime.h>

#include "qg_device.h"
#include "qg_internal.h"
#include "qg_mm.h"

namespace qg {

// lse and loss from the statistics of every tile of columns ([tiles][m] of largest
// logit and sum): 16 rows side by side, 64 lanes along the tiles, joined as a tree.
__global__ __launch_bounds__(1024) void xent_join_kernel(const float2 *stats, const float *at_target, int tiles, int m,
                                                         int vocab, const int32_t *targets, float scale, float *loss,
                                                         float *lse) {
  __shared__ float2 join[16][16];
  const int side = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int row = blockIdx.x * 16 + side, at = min(row, m - 1);
  const float base2 = scale * 1.4426950408889634f;
  float most = -INFINITY, sum = 0.f;
  auto add = [&](float big, float s) {
    const float both = fmaxf(most, big), from = both == -INFINITY ? 0.f : both;
    sum = sum * __builtin_amdgcn_exp2f((most - from) * base2) + s * __builtin_amdgcn_exp2f((big - from) * base2);
    most = both;
  };
  auto join_lanes = [&] {
#pragma unroll
    for (int off = 16; off < 64; off <<= 1) add(__shfl_xor(most, off), __shfl_xor(sum, off));
  };
  const int t = targets ? targets[at] : -1;
  const bool counts = t >= 0 && t < vocab;
  const float hit = loss && counts ? at_target[at] : 0.f;
  constexpr int GO = 8;  // loads out together
  for (int t0 = part; t0 < tiles; t0 += 64 * GO) {
    float2 v[GO];
#pragma unroll
    for (int g = 0; g < GO; ++g) v[g] = stats[(int64_t)min(t0 + 64 * g, tiles - 1) * m + at];
#pragma unroll
    for (int g = 0; g < GO; ++g)
      if (t0 + 64 * g < tiles) add(v[g].x, v[g].y);
  }
  join_lanes();
  if ((threadIdx.x & 63) < 16) join[threadIdx.x >> 6][side] = float2{most, sum};
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const int first = threadIdx.x >> 4;
  most = join[first][side].x;
  sum = join[first][side].y;
#pragma unroll
  for (int o = 4; o < 16; o += 4) add(join[first + o][side].x, join[first + o][side].y);
  join_lanes();
  if (threadIdx.x >= 16 || row >= m) return;
  // (nothing but NaN logits: `most` is -inf and the sum NaN)
  const float log_sum = logf(sum);
  if (lse) lse[row] = __builtin_fmaf(scale, most, log_sum);
  // (an ignored row's loss is 0; scale (largest - target's) is exact where the two are near)
  if (loss) loss[row] = counts ? __builtin_fmaf(scale, most - hit, log_sum) : 0.f;
}

// dx (bf16) = alpha times the sum of `parts` fp32 matrices [m][k], in order; k % 8 ==
// 0, 8 values per thread.
__global__ __launch_bounds__(256) void xent_dx_kernel(const float *p, int parts, int64_t stride, int64_t k8, int64_t units,
                                                      const float *alpha, uint16_t *dx, int64_t lddx) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const float by = alpha[0];
  f32x4 sum[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const f32x4 *v = (const f32x4 *)(p + s * stride) + 2 * u;
    sum[0] += v[0];
    sum[1] += v[1];
  }
  const int64_t row = u / k8, c8 = u - row * k8;
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = bf16_rne(by * sum[e / 2][e % 2 * 2]) | bf16_rne(by * sum[e / 2][e % 2 * 2 + 1]) << 16;
  *(u32x4_any *)(dx + row * lddx + 8 * c8) = w;  // (rows of dx start at any element)
}

// The largest |dloss| of the rows that count, for calls of many rows (up to 512, one
// per thread, the gradient's workgroups find it for themselves; with 4096 that cost
// 20 us a round of tiles).
__global__ __launch_bounds__(1024) void xent_most_kernel(const float *dloss, const int32_t *targets, int m, int vocab,
                                                         float *out) {
  __shared__ float wave_most[16];
  float most = 0.f;
  for (int r = threadIdx.x; r < m; r += 1024)
    if ((uint32_t)targets[r] < (uint32_t)vocab) most = fmaxf(most, fabsf(dloss[r]));
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) most = fmaxf(most, __shfl_xor(most, off));
  if ((threadIdx.x & 63) == 0) wave_most[threadIdx.x >> 6] = most;
  __syncthreads();
  for (int w = 0; w < 16; ++w) most = fmaxf(most, wave_most[w]);
  if (threadIdx.x == 0) out[0] = most;
}

// Parts of dx take at most this much (or one part).
constexpr uint64_t kXentPartBytes = 80u << 20;

static int64_t xent_halves(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 0; }
int64_t xent_d_rows(int64_t m) { return m + xent_halves(m); }

// Columns of a piece: d takes up to 128 MB, half of the last-level cache, in which both
// products find it (W's rows are not counted), and at least 8192 columns (the products over a piece would be
// short).
int64_t xent_piece(int64_t m, int64_t vocab) {
  int64_t most = (64ll << 20) / std::max<int64_t>(m, 1);
  most = std::min<int64_t>(std::max<int64_t>(most / 256 * 256, 8192), 1 << 20);
  const int64_t pieces = (vocab + most - 1) / most;
  return std::min<int64_t>(((vocab + pieces - 1) / pieces + 255) / 256 * 256, (vocab + 63) / 64 * 64);
}

// (64 x 128 in three stages, two workgroups per CU: 61 tokens of 100003 x 2048 95 us,
// in four stages 105)
// (few tokens, whose d has two parts: one shape)
template <int EPI>
using XentFew = MmCfg<false, kRows, kRows, false, 32, 128, 1, 8, 4, true, EPI>;
template <int EPI>
using XentLogits = MmShapes<MmCfg<false, kRows, kRows, false, 256, 256, 4, 2, 2, false, EPI>,
                            MmCfg<false, kRows, kRows, false, 192, 256, 4, 2, 2, false, EPI>,
                            MmCfg<false, kRows, kRows, false, 128, 128, 4, 2, 2, true, EPI>,
                            MmCfg<false, kRows, kRows, false, 128, 128, 4, 2, 4, true, EPI>,
                            MmCfg<false, kRows, kRows, false, 64, 128, 2, 4, 3, true, EPI>, XentFew<EPI>>;

static MmMoreArgs xent_args(const XentCall &c, int64_t first, int64_t columns) {
  MmMoreArgs a = {};
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
  MmMoreArgs a = xent_args(c, 0, c.vocab);
  a.stats = c.stats;
  a.at_target = c.at_target;
  MmInfo choice;
  hipError_t e = XentLogits<kXentStats>::dispatch(a, kMmPartialBytes, nullptr, &choice);
  if (info) *info = choice;
  if (info || e != hipSuccess) return e;
  e = XentLogits<kXentStats>::dispatch(a, kMmPartialBytes, s, nullptr);
  if (e != hipSuccess) return e;
  const int tiles = (int)((c.vocab + choice.bn - 1) / choice.bn);
  hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)((c.m + 15) / 16)), dim3(1024), 0, s, (const float2 *)c.stats,
                     c.at_target, tiles, (int)c.m, (int)c.vocab, c.targets, c.scale, c.loss, c.lse);
  return hipGetLastError();
}

// d of one piece
// (alpha: by the workgroup of the first tile; its neighbour holds the largest |dloss|
// of calls that look for it once)
hipError_t launch_xent_d(const XentCall &c, int64_t first, int64_t columns, hipStream_t s, MmInfo *info) {
  MmMoreArgs a = xent_args(c, first, columns);
  a.lse = c.lse;
  a.dloss = c.dloss;
  a.alpha_out = c.alpha;
  if (c.m > 512) {
    a.dloss_most = c.alpha + 1;
    if (first == 0 && !info) {
      hipLaunchKernelGGL(xent_most_kernel, dim3(1), dim3(1024), 0, s, c.dloss, c.targets, (int)c.m, (int)c.vocab, c.alpha + 1);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  a.vocab = (int32_t)c.vocab;
  a.y = c.d;
  a.ldy = c.ldd;
  a.otype = QG_O_BF16;
  a.halves = (int32_t)xent_halves(c.m);
  if (a.halves > 0) return mm_dispatch<XentFew<kXentGrad>>(a, kMmPartialBytes, s, info);
  return XentLogits<kXentGrad>::dispatch(a, kMmPartialBytes, s, info);
}

// d W of one piece into parts of dx.  The contraction is long and the tiles are
// few: parts of it in fp32, which a kernel of all CUs adds up behind the last piece
// (one workgroup per tile would read 4 MB of 16 parts by itself).  400 tokens of
// 50000 x 2048: 256 x 256 in 16 parts 108 us, 128 x 128 in 4 151 (two stages 152); 257
// of 38531 x 1032: 128 x 128 in 8 parts 58, 256 x 256 70, 64 x 128 61.
// info->splits: how many parts the piece has; there: how many hold earlier pieces.
using XentDxFew = MmCfg<false, kRows, kCols, false, 32, 128, 1, 8, 4, true, kParts>;
using XentDx = MmShapes<MmCfg<false, kRows, kCols, false, 256, 256, 4, 2, 2, true, kParts>,
                        MmCfg<false, kRows, kCols, false, 128, 128, 4, 2, 4, true, kParts>,
                        MmCfg<false, kRows, kCols, false, 64, 128, 2, 4, 4, true, kParts>, XentDxFew>;
hipError_t launch_xent_dx(const XentCall &c, int64_t first, int64_t columns, int there, hipStream_t s, MmInfo *info) {
  MmMoreArgs a = xent_args(c, first, columns);
  a.a = (const uint8_t *)c.d;
  a.lda = c.ldd * 2;
  a.n = (int32_t)c.k;
  a.kd = (int32_t)columns;
  a.y = c.parts;
  a.otype = QG_O_F32;
  a.ldy = c.k;
  a.part_stride = c.m * c.k;
  a.parts_there = there;
  if (c.m <= 16) {
    a.halves = (int32_t)xent_halves(c.m);
    a.m += a.halves;
    return mm_dispatch<XentDxFew>(a, kXentPartBytes, s, info);
  }
  return XentDx::dispatch(a, kXentPartBytes, s, info);
}

hipError_t launch_xent_dx_sum(const XentCall &c, int parts, void *dx, int64_t lddx, hipStream_t s) {
  const int64_t units = c.m * c.k / 8;
  hipLaunchKernelGGL(xent_dx_kernel, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, s, (const float *)c.parts, parts,
                     c.m * c.k, c.k / 8, units, c.alpha, (uint16_t *)dx, lddx);
  return hipGetLastError();
}

// rows of dW of one piece
using XentDw = MmShapes<MmCfg<false, kCols, kCols, false, 256, 256, 4, 2, 2, false, kScaled>,
                        MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 2, true, kScaled>,
                        MmCfg<false, kCols, kCols, false, 128, 128, 4, 2, 4, true, kScaled>>;
hipError_t launch_xent_dw(const XentCall &c, int64_t first, int64_t columns, void *dw, int dw_type, int64_t lddw,
                          hipStream_t s, MmInfo *info) {
  MmMoreArgs a = xent_args(c, first, columns);
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
  return XentDw::dispatch(a, kMmPartialBytes, s, info);
}

// Bounds for any call of up to m tokens, which may have other shapes, parts and pieces
// than one of m: a buffer for the largest batch serves the smaller ones.
XentMost xent_most(int64_t m, int64_t k, int64_t vocab) {
  const int64_t whole = (vocab + 63) / 64 * 64;  // a piece at most
  const int64_t rows = m <= 16 ? m + 16 : m <= 32 ? m + 32 : std::max<int64_t>(m, 64);  // xent_d_rows at most
  XentMost b;
  b.partials = XentLogits<kXentStats>::most_bytes(m, vocab, k, kMmPartialBytes);
  b.stat_tiles = (vocab + XentLogits<kXentStats>::narrowest - 1) / XentLogits<kXentStats>::narrowest;
  b.back_partials = std::max(XentLogits<kXentGrad>::most_bytes(m, whole, k, kMmPartialBytes),
                             XentDw::most_bytes(whole, k, rows, kMmPartialBytes));
  // (pieces of up to 64 Mi / m columns, at least 8192, at most 2^20)
  b.d = 2 * (uint64_t)std::min(std::max<int64_t>(64ll << 20, 8192 * m), rows * whole);
  const uint64_t part = 4 * (uint64_t)m * k;
  b.parts = std::max(part, std::min(part * kMmMostSplits, XentDx::most_bytes(rows, k, whole, kXentPartBytes)));
  return b;
}

}  // namespace qg
