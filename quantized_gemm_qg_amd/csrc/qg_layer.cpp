// C ABI of what stands around the products of a layer and behind the last one:
// the root-mean-square norm, the low-rank adapters and the cross entropy of a
// head.  Argument checks, workspaces and dispatch.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "qg_internal.h"

using namespace qg;

// Checks of one matrix of 16-byte accesses: `el` bytes per element.
static qg_status matrix_check(const void *p, int64_t ld, int64_t columns, int el) {
  if (ld < columns) return QG_ERR_SHAPE;
  return aligned(p, 16) && ld * el % 16 == 0 ? QG_OK : QG_ERR_ALIGNMENT;
}
#define QG_TRY(check)                       \
  do {                                      \
    const qg_status st_ = (check);          \
    if (st_ != QG_OK) return st_;           \
  } while (0)

// (The workspaces of the norm's backward pass and of the adapters need no zeros; they
// begin behind the place of the products' arrival counters, so that one buffer may
// serve all of them.)

// Checks that the two directions of the norm share.
static qg_status norm_check(const void *weight, float eps, int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || !std::isfinite(eps) || !(eps > 0.f)) return QG_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 8 != 0) return QG_ERR_SHAPE;
  if (k > (1 << 24)) return QG_ERR_UNSUPPORTED;
  if (rows > 0 && !weight) return QG_ERR_INVALID_ARGUMENT;
  return aligned(weight, 16) ? QG_OK : QG_ERR_ALIGNMENT;
}

extern "C" qg_status qg_rmsnorm(const void *x, int32_t x_type, int64_t ldx, const void *residual, int32_t res_type,
                                int64_t ldr, void *sum, int64_t lds, const void *weight, float eps, int64_t rows,
                                int64_t k, void *y, int64_t ldy, int32_t q_type, void *q, int64_t ldq, void *q_scales,
                                hipStream_t stream) {
  QG_TRY(norm_check(weight, eps, rows, k));
  const bool added = residual || sum;
  if (!out_type(x_type) || (added && !out_type(res_type))) return QG_ERR_INVALID_ARGUMENT;
  if (q_type == QG_A_MXFP4) return QG_ERR_UNSUPPORTED;
  if (q_type != QG_A_BF16 && q_type != QG_A_INT8_TOKEN && q_type != QG_A_FP8_TOKEN && q_type != QG_A_FP8_BLOCK &&
      q_type != QG_A_MXFP8)
    return QG_ERR_INVALID_ARGUMENT;
  if (q_type == QG_A_MXFP8 && k % 32 != 0) return QG_ERR_SHAPE;
  if (rows > 0 && (!x || (!y && !q) || (q != nullptr) != (q_type != QG_A_BF16) || (q && !q_scales)))
    return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(x, ldx, k, el_of(x_type)));
  if (residual) QG_TRY(matrix_check(residual, ldr, k, el_of(res_type)));
  if (sum) QG_TRY(matrix_check(sum, lds, k, el_of(res_type)));
  if (y) QG_TRY(matrix_check(y, ldy, k, 2));
  if (q) {
    if (ldq < k) return QG_ERR_SHAPE;
    if (!aligned(q, 8) || ldq % 8 != 0 || (q_type != QG_A_MXFP8 && !aligned(q_scales, 4))) return QG_ERR_ALIGNMENT;
  }
  if (rows == 0) return QG_OK;
  // (a buffer that is read and written has to be the same matrix both times)
  if (sum && ((sum == x && (x_type != res_type || lds != ldx)) || (sum == residual && lds != ldr)))
    return QG_ERR_INVALID_ARGUMENT;
  const NormArgs a{x, ldx, residual, ldr, sum, lds, weight, eps, rows, k, (uint16_t *)y, ldy, q_type, (uint8_t *)q, ldq, q_scales};
  return hip_status(launch_rmsnorm(a, x_type == QG_O_F32, !added ? 0 : res_type == QG_O_BF16 ? 1 : 2, stream));
}

extern "C" qg_status qg_rmsnorm_backward_workspace_size(int64_t rows, int64_t k, uint64_t *bytes) {
  if (!bytes || rows < 0 || k < 0) return QG_ERR_INVALID_ARGUMENT;
  *bytes = rows == 0 || k == 0 ? 0 : kSplitCounterBytes + align_up((uint64_t)rmsnorm_back_parts(rows, k) * k * 4, 256);
  return QG_OK;
}

extern "C" qg_status qg_rmsnorm_backward(const void *s, int32_t s_type, int64_t lds, const void *weight, float eps,
                                         int64_t rows, int64_t k, const void *dy, int64_t lddy, const void *dsum,
                                         int64_t ldds, void *dx, int64_t lddx, void *dw, int32_t dw_type, void *ws,
                                         uint64_t ws_bytes, hipStream_t stream) {
  QG_TRY(norm_check(weight, eps, rows, k));
  if (!out_type(s_type) || (dw && !out_type(dw_type))) return QG_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!s || !dy)) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(s, lds, k, el_of(s_type)));
  QG_TRY(matrix_check(dy, lddy, k, 2));
  if (dsum) QG_TRY(matrix_check(dsum, ldds, k, el_of(s_type)));
  if (dx) QG_TRY(matrix_check(dx, lddx, k, el_of(s_type)));
  if (!aligned(dw, 16)) return QG_ERR_ALIGNMENT;
  if (dx && dx == dsum && lddx != ldds) return QG_ERR_INVALID_ARGUMENT;
  if (!dw && (!dx || rows == 0)) return QG_OK;
  if (dw) {
    uint64_t need = 0;
    (void)qg_rmsnorm_backward_workspace_size(rows, k, &need);
    QG_TRY(ws_check(need, ws, ws_bytes));
  }
  const NormBackArgs a{s, lds, weight, eps, rows, k, (const uint16_t *)dy, lddy, dsum, ldds, dx, lddx,
                       dw ? (float *)((uint8_t *)ws + kSplitCounterBytes) : nullptr};
  return hip_status(launch_rmsnorm_backward(a, s_type == QG_O_F32, dw, dw_type == QG_O_F32, stream));
}

static qg_status lora_sizes(int64_t m, int64_t k, int64_t n, int32_t adapters, int32_t rank) {
  if (m < 0 || k < 0 || n < 0 || adapters <= 0 || rank <= 0) return QG_ERR_INVALID_ARGUMENT;
  if (k == 0 || n == 0 || k % 8 != 0 || rank % 8 != 0) return QG_ERR_SHAPE;
  if (rank > QG_LORA_MAX_RANK || adapters > kMaxExperts || m > (1 << 21) || k > (1 << 22) || n > (1 << 24))
    return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

// Bytes for `t_rows` fp32 rows of the first product's parts.
static uint64_t lora_bytes(int64_t t_rows, int32_t rank) {
  return kSplitCounterBytes + align_up((uint64_t)t_rows * rank * 4, 256);
}

// (for any call of up to m rows: fewer rows have more parts of k)
extern "C" qg_status qg_lora_workspace_size(int64_t m, int64_t k, int64_t n, int32_t num_adapters, int32_t rank,
                                            uint64_t *bytes) {
  if (!bytes) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(lora_sizes(m, k, n, num_adapters, rank));
  const bool none = m == 0 || lora_plan(m, k, n, num_adapters, rank, false).small;
  *bytes = none ? 0 : lora_bytes(lora_most_rows(m, k), rank);
  return QG_OK;
}

extern "C" qg_status qg_lora(const void *x, int64_t ldx, const void *a, int64_t lda, const void *b, int64_t ldb,
                             const float *scales, int32_t num_adapters, int32_t rank, const int32_t *sorted_rows,
                             const int32_t *offsets, int64_t m, int64_t k, int64_t n, void *y, int32_t y_type,
                             int64_t ldy, void *ws, uint64_t ws_bytes, hipStream_t stream) {
  QG_TRY(lora_sizes(m, k, n, num_adapters, rank));
  if (!out_type(y_type)) return QG_ERR_INVALID_ARGUMENT;
  if (m > 0 && (!x || !a || !b || !sorted_rows || !offsets || !y)) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(x, ldx, k, 2));
  QG_TRY(matrix_check(a, lda, k, 2));
  QG_TRY(matrix_check(b, ldb, rank, 2));
  if (2 * lda > kMaxPitchBytes || 2 * ldb > kMaxPitchBytes) return QG_ERR_UNSUPPORTED;
  if (ldy < n) return QG_ERR_SHAPE;
  if (!aligned(y, el_of(y_type)) || !aligned(scales, 4) || !aligned(sorted_rows, 4) || !aligned(offsets, 4))
    return QG_ERR_ALIGNMENT;
  if (m == 0) return QG_OK;
  const LoraPlan plan = lora_plan(m, k, n, num_adapters, rank, y_type == QG_O_F32);
  if (!plan.small) QG_TRY(ws_check(lora_bytes(plan.splits * m, rank), ws, ws_bytes));
  const bool vectors = aligned(y, 16) && ldy * el_of(y_type) % 16 == 0;
  const LoraArgs args{(const uint16_t *)x, ldx, (const uint16_t *)a, lda, (const uint16_t *)b, ldb, scales, sorted_rows, offsets,
                      num_adapters, rank, (int32_t)m, (int32_t)k, (int32_t)n, y, ldy, vectors,
                      plan.small ? nullptr : (float *)((uint8_t *)ws + kSplitCounterBytes), plan.splits, plan.chunks};
  return hip_status(launch_lora(args, plan, y_type == QG_O_F32, stream));
}

extern "C" qg_status qg_describe_lora(int64_t m, int64_t k, int64_t n, int32_t num_adapters, int32_t rank, int32_t y_type,
                                      char *buf, uint64_t buf_bytes) {
  if (!buf || buf_bytes == 0 || !out_type(y_type)) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(lora_sizes(m, k, n, num_adapters, rank));
  if (m == 0) {
    snprintf(buf, buf_bytes, "nothing");
    return QG_OK;
  }
  const LoraPlan p = lora_plan(m, k, n, num_adapters, rank, y_type == QG_O_F32);
  if (p.small)
    snprintf(buf, buf_bytes, "lora_small NB=%d", p.nb);
  else
    snprintf(buf, buf_bytes, "lora_down NB=%d splits=%d; lora_up RB=%d SD=%d chunks=%d", p.nb, p.splits, p.rb, p.sd, p.chunks);
  return QG_OK;
}

namespace qg {

// Forward workspace: [split-K counters][partial tiles][statistics of the
// tiles][the targets' logits].
struct XentSpace {
  uint64_t partials = 0, stats = 0, at_target = 0;  // bytes
  uint64_t total() const { return kSplitCounterBytes + partials + stats + at_target; }
};
// Backward: [split-K counters][partial tiles][alpha][d of a piece][parts of dx].
struct XentBackSpace {
  int64_t piece = 0;
  int splits = 1, last_splits = 1;  // parts of dx of a whole piece and of the last one
  uint64_t partials = 0, d = 0, parts = 0;
  static constexpr uint64_t alpha = 256;
  uint64_t total() const { return kSplitCounterBytes + partials + alpha + d + parts; }
};

static bool xent_in_range(int64_t m, int64_t k, int64_t vocab) {
  return m <= (1ll << 30) && k <= (1 << 22) && vocab <= (1 << 24) && tiles_fit(m, vocab) && tiles_fit(m, k) &&
         tiles_fit(vocab, k);
}

static XentSpace xent_space(int64_t m, uint64_t partials, int64_t stat_tiles) {
  XentSpace sp;
  sp.partials = align_up(partials, 256);
  sp.stats = align_up((uint64_t)stat_tiles * m * 8, 256);
  sp.at_target = align_up((uint64_t)m * 4, 256);
  return sp;
}

static XentSpace xent_space(const XentCall &c) {
  MmInfo i;
  (void)launch_xent(c, nullptr, &i);
  return xent_space(c.m, i.bytes, (c.vocab + i.bn - 1) / i.bn);
}

static XentBackSpace xent_back_space(const XentCall &c) {
  XentBackSpace sp;
  sp.piece = xent_piece(c.m, c.vocab);
  // the last piece may be shorter, and its products split otherwise
  const int64_t last = c.vocab - (c.vocab - 1) / sp.piece * sp.piece;
  auto count = [&](int64_t columns) {
    MmInfo i;
    (void)launch_xent_d(c, 0, columns, nullptr, &i);
    sp.partials = std::max(sp.partials, i.bytes);
    (void)launch_xent_dw(c, 0, columns, nullptr, 0, 0, nullptr, &i);
    sp.partials = std::max(sp.partials, i.bytes);
    (void)launch_xent_dx(c, 0, columns, 0, nullptr, &i);
    return i.splits;
  };
  sp.last_splits = count(last);
  sp.splits = sp.piece < c.vocab ? count(sp.piece) : sp.last_splits;
  sp.partials = align_up(sp.partials, 256);
  sp.parts = align_up((uint64_t)std::max(sp.splits, sp.last_splits) * c.m * c.k * 4, 256);
  sp.d = align_up((uint64_t)xent_d_rows(c.m) * sp.piece * 2, 256);
  return sp;
}

// Checks that the two directions of the cross entropy share.
static qg_status xent_check(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k, int64_t vocab,
                            const int32_t *targets, float scale) {
  if (m < 0 || k < 0 || vocab < 0 || !std::isfinite(scale) || !(scale > 0.f)) return QG_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 8 != 0 || vocab == 0) return QG_ERR_SHAPE;
  if (!xent_in_range(m, k, vocab) || 2 * ldx > kMaxPitchBytes || 2 * ldw > kMaxPitchBytes) return QG_ERR_UNSUPPORTED;
  if (m > 0 && (!x || !w)) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(x, ldx, k, 2));
  QG_TRY(matrix_check(w, ldw, k, 2));
  return aligned(targets, 4) ? QG_OK : QG_ERR_ALIGNMENT;
}

static XentCall xent_call(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k, int64_t vocab,
                          const int32_t *targets, float scale) {
  XentCall c = {};
  c.x = x;
  c.ldx = ldx;
  c.w = w;
  c.ldw = ldw;
  c.m = m;
  c.k = k;
  c.vocab = vocab;
  c.targets = targets;
  c.scale = scale;
  return c;
}

// Bytes of either workspace, for any call of up to m tokens; 0 for sizes that the calls
// refuse or that need none.
static qg_status xent_bytes(int64_t m, int64_t k, int64_t vocab, bool backward, uint64_t *bytes) {
  if (!bytes || m < 0 || k < 0 || vocab < 0) return QG_ERR_INVALID_ARGUMENT;
  *bytes = 0;
  if (m == 0 || k == 0 || vocab == 0 || !xent_in_range(m, k, vocab)) return QG_OK;
  const XentMost most = xent_most(m, k, vocab);
  if (!backward) {
    *bytes = xent_space(m, most.partials, most.stat_tiles).total();
    return QG_OK;
  }
  XentBackSpace sp;
  sp.partials = align_up(most.back_partials, 256);
  sp.d = align_up(most.d, 256);
  sp.parts = align_up(most.parts, 256);
  *bytes = sp.total();
  return QG_OK;
}

}  // namespace qg

extern "C" qg_status qg_linear_xent_workspace_size(int64_t m, int64_t k, int64_t vocab, uint64_t *bytes) {
  return xent_bytes(m, k, vocab, false, bytes);
}

extern "C" qg_status qg_linear_xent(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k,
                                    int64_t vocab, const int32_t *targets, float scale, float *loss, float *lse,
                                    void *ws, uint64_t ws_bytes, hipStream_t stream) {
  QG_TRY(xent_check(x, ldx, w, ldw, m, k, vocab, targets, scale));
  if (!aligned(loss, 4) || !aligned(lse, 4)) return QG_ERR_ALIGNMENT;
  if (m == 0) return QG_OK;
  if ((!loss && !lse) || (loss && !targets)) return QG_ERR_INVALID_ARGUMENT;
  XentCall c = xent_call(x, ldx, w, ldw, m, k, vocab, targets, scale);
  const XentSpace sp = xent_space(c);
  QG_TRY(ws_check(sp.total(), ws, ws_bytes));
  c.loss = loss;
  c.lse = lse;
  uint8_t *p = (uint8_t *)ws;
  c.counters = (uint32_t *)p;
  c.partials = p += kSplitCounterBytes;
  c.stats = (float *)(p += sp.partials);
  c.at_target = (float *)(p + sp.stats);
  return hip_status(launch_xent(c, stream));
}

extern "C" qg_status qg_linear_xent_backward_workspace_size(int64_t m, int64_t k, int64_t vocab, uint64_t *bytes) {
  return xent_bytes(m, k, vocab, true, bytes);
}

extern "C" qg_status qg_linear_xent_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k,
                                             int64_t vocab, const int32_t *targets, float scale, const float *lse,
                                             const float *dloss, void *dx, int64_t lddx, void *dw, int32_t dw_type,
                                             int64_t lddw, void *ws, uint64_t ws_bytes, hipStream_t stream) {
  QG_TRY(xent_check(x, ldx, w, ldw, m, k, vocab, targets, scale));
  if (dw && !out_type(dw_type)) return QG_ERR_INVALID_ARGUMENT;
  if ((dx && lddx < k) || (dw && lddw < k)) return QG_ERR_SHAPE;
  if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dx, 16) || !aligned(dw, 16)) return QG_ERR_ALIGNMENT;
  if (m == 0)  // a sum over no tokens
    return dw ? hip_status(launch_ffn_zero(dw, lddw * el_of(dw_type), k * el_of(dw_type), vocab, stream)) : QG_OK;
  if (!targets || !lse || !dloss) return QG_ERR_INVALID_ARGUMENT;
  if (!dx && !dw) return QG_OK;
  XentCall c = xent_call(x, ldx, w, ldw, m, k, vocab, targets, scale);
  const XentBackSpace sp = xent_back_space(c);
  QG_TRY(ws_check(sp.total(), ws, ws_bytes));
  c.lse = const_cast<float *>(lse);
  c.dloss = dloss;
  uint8_t *p = (uint8_t *)ws;
  c.counters = (uint32_t *)p;
  c.partials = p += kSplitCounterBytes;
  c.alpha = (float *)(p += sp.partials);
  c.d = p += sp.alpha;
  c.ldd = sp.piece;
  c.parts = (float *)(p + sp.d);
  hipError_t e = hipSuccess;
  for (int64_t first = 0; e == hipSuccess && first < vocab; first += sp.piece) {
    const int64_t columns = std::min(sp.piece, vocab - first);
    e = launch_xent_d(c, first, columns, stream);
    if (e == hipSuccess && dx) e = launch_xent_dx(c, first, columns, first > 0 ? sp.splits : 0, stream);
    if (e == hipSuccess && dw) e = launch_xent_dw(c, first, columns, dw, dw_type, lddw, stream);
  }
  if (e == hipSuccess && dx) e = launch_xent_dx_sum(c, std::max(sp.splits, sp.last_splits), dx, lddx, stream);
  return hip_status(e);
}

extern "C" qg_status qg_describe_linear_xent(int64_t m, int64_t k, int64_t vocab, char *buf, uint64_t buf_bytes) {
  if (!buf || buf_bytes == 0 || m < 0 || k < 0 || vocab < 0) return QG_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 8 != 0 || vocab == 0) return QG_ERR_SHAPE;
  if (!xent_in_range(m, k, vocab)) return QG_ERR_UNSUPPORTED;
  char out[512] = "nothing";
  int at = 0;
  MmInfo i;
  auto add = [&](const char *name, hipError_t) {  // (the choice is in i)
    at += snprintf(out + at, sizeof out - at, "%s BM=%d BN=%d stages=%d splits=%d", name, i.bm, i.bn, i.stages, i.splits);
  };
  if (m > 0) {
    const XentCall c = xent_call(nullptr, k, nullptr, k, m, k, vocab, nullptr, 1.f);
    add("logits", launch_xent(c, nullptr, &i));
    const int64_t piece = xent_piece(m, vocab), pieces = (vocab + piece - 1) / piece, last = vocab - (pieces - 1) * piece;
    // pieces of full length, and a last one of another
    const int64_t full = last == piece ? pieces : pieces - 1;
    for (int64_t columns : {piece, last}) {
      const int64_t count = columns == piece ? full : 1;
      if (count == 0) continue;
      at += snprintf(out + at, sizeof out - at, "; %lld x %lld:", (long long)count, (long long)columns);
      add(" d", launch_xent_d(c, 0, columns, nullptr, &i));
      add(", dx", launch_xent_dx(c, 0, columns, 0, nullptr, &i));
      add(", dw", launch_xent_dw(c, 0, columns, nullptr, 0, 0, nullptr, &i));
      if (last == piece) break;
    }
  }
  snprintf(buf, buf_bytes, "%s", out);
  return QG_OK;
}
