// C ABI of the int8 products, the gated feed-forward block and the token log
// probabilities: argument checks, workspaces and dispatch.
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "qg_internal.h"

namespace qg {

static bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
static int el_of(int otype) { return otype == QG_O_F32 ? 4 : 2; }
static bool out_type(int t) { return t == QG_O_BF16 || t == QG_O_F32; }

// Checks a workspace of `need` bytes (0: none).
static qg_status ws_check(uint64_t need, const void *ws, uint64_t ws_bytes) {
  if (need == 0) return QG_OK;
  if (!ws) return QG_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return QG_ERR_BUFFER_TOO_SMALL;
  return aligned(ws, 256) ? QG_OK : QG_ERR_ALIGNMENT;
}

// The tiled products address a tile's rows with 32-bit offsets from a 64-bit
// base: 256 rows of this pitch stay below 2 GiB.  (The gradient of the
// pre-activations has rows of up to 64 MiB, of which 64 are within reach: shapes
// of more rows are left out where theirs are not.)
constexpr int64_t kMaxPitchBytes = 1 << 23;
// Tiles are numbered in 32 bits (the smallest tile is 32 x 64 outputs).
static bool tiles_fit(int64_t m, int64_t n) { return ((m + 31) / 32) * ((n + 63) / 64) < (1ll << 31) - 8; }

// Int8 workspace: [split-K counters][partial tiles][codes of the quantized
// rows][their scales]; nothing where none of them is needed.
struct I8Space {
  uint64_t partials = 0, codes = 0, scales = 0;  // bytes
  uint64_t total() const {
    const uint64_t b = partials + codes + scales;
    return b ? kSplitCounterBytes + b : 0;
  }
};
static I8Call i8_call(const qg_weight &w, bool gated, int64_t m, uint32_t flags) {
  I8Call c = {};
  c.n = (int32_t)(gated ? w.desc.n / 2 : w.desc.n);
  c.k = (int32_t)w.desc.k;
  c.k_blocks = w.k_blocks;
  c.gated = gated;
  c.m = m;
  c.small_scratch = (flags & kI8SmallScratch) != 0;
  c.quantize = (flags & QG_GEMM_QUANTIZE_X) && i8_quantizes_in_kernel(m, w.desc.k);
  return c;
}
static I8Space i8_space(const I8Call &c, uint32_t flags) {
  I8Space sp;
  sp.partials = align_up(i8_info(c).bytes, 256);
  if ((flags & QG_GEMM_QUANTIZE_X) && !c.quantize) {
    sp.codes = align_up((uint64_t)c.m * c.k, 256);
    sp.scales = align_up((uint64_t)c.m * 4, 256);
  }
  return sp;
}
uint64_t i8_ws_bytes(const qg_weight &w, bool gated, int64_t m, uint32_t flags) {
  return m <= 0 || m > (1ll << 30) ? 0 : i8_space(i8_call(w, gated, m, flags), flags).total();
}

void i8_describe(const qg_weight &w, int64_t m, uint32_t flags, char *buf, uint64_t buf_bytes) {
  const I8Call c = i8_call(w, false, std::min<int64_t>(std::max<int64_t>(m, 1), 1 << 30), flags);
  const MmInfo i = i8_info(c);
  if (i.bn == 0)
    snprintf(buf, buf_bytes, "i8_rows M<=%d%s", i.bm, c.quantize ? " quantizing" : "");
  else
    snprintf(buf, buf_bytes, i.splits > 1 ? "i8_tiled BM=%d BN=%d splits=%d" : "i8_tiled BM=%d BN=%d", i.bm, i.bn,
             i.splits);
}

qg_status i8_product(const qg_weight *w, const Layout &L, bool gated, const void *x, const void *x_scales, int64_t m,
                     int64_t ldx, void *y, int32_t otype, int64_t ldy, int32_t act, void *ws, uint64_t ws_bytes,
                     uint32_t flags, hipStream_t stream) {
  const qg_layer_desc &d = w->desc;
  const bool quantize = (flags & QG_GEMM_QUANTIZE_X) != 0;
  const int64_t n = gated ? d.n / 2 : d.n;
  if (m < 0 || !out_type(otype) || (flags & ~(kI8Flags | kI8SmallScratch)) != 0) return QG_ERR_INVALID_ARGUMENT;
  if (m > (1ll << 30) || !tiles_fit(m, n)) return QG_ERR_UNSUPPORTED;
  if (m == 0) return QG_OK;
  if (!x || !y || (!quantize && !x_scales)) return QG_ERR_INVALID_ARGUMENT;
  if (ldx < d.k || ldy < n) return QG_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || ldx * (quantize ? 2 : 1) % 16 != 0 || ldy * el_of(otype) % 4 != 0)
    return QG_ERR_ALIGNMENT;
  if (!quantize && !aligned(x_scales, 4)) return QG_ERR_ALIGNMENT;
  if (ldx > kMaxPitchBytes) return QG_ERR_UNSUPPORTED;
  I8Call c = i8_call(*w, gated, m, flags);
  const I8Space sp = i8_space(c, flags);
  const qg_status wst = ws_check(sp.total(), ws, ws_bytes);
  if (wst != QG_OK) return wst;
  c.codes = (const uint8_t *)w->data;
  c.scales = (const float *)(c.codes + L.scales_offset);
  c.act = act;
  c.x = x;
  c.ldx = ldx;
  c.x_scales = (const float *)x_scales;
  c.y = y;
  c.otype = otype;
  c.ldy = ldy;
  if (sp.partials) {
    c.counters = (uint32_t *)ws;
    c.partials = (uint8_t *)ws + kSplitCounterBytes;
  }
  if (quantize && !c.quantize) {
    uint8_t *q = (uint8_t *)ws + kSplitCounterBytes + sp.partials;
    float *qs = (float *)(q + sp.codes);
    const hipError_t e = launch_quantize_int8(x, m, d.k, ldx, q, d.k, qs, stream);
    if (e != hipSuccess) return hip_status(e);
    c.x = q;
    c.ldx = d.k;
    c.x_scales = qs;
  }
  return hip_status(launch_i8(c, stream));
}

// Row pitch (elements) of the gradient of the pre-activations: a multiple of
// 64 elements, so that rows start on 128-byte lines.
static int64_t dgu_pitch(int64_t inter) { return (int64_t)align_up(2 * (uint64_t)inter, 64); }

// Checks that the forward and the backward pass of the block share.
static qg_status ffn_check(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k, int64_t inter,
                           int32_t act) {
  if (m < 0 || k < 0 || inter < 0 || (act != QG_ACT_SILU && act != QG_ACT_GELU_TANH)) return QG_ERR_INVALID_ARGUMENT;
  if (k % 8 != 0 || k == 0 || inter == 0 || ldx < k || ldw < k) return QG_ERR_SHAPE;
  if (m > (1ll << 30) || inter > (1 << 24) || k > (1 << 22) || !tiles_fit(m, inter) || !tiles_fit(m, k) ||
      !tiles_fit(2 * inter, k) || 2 * ldx > kMaxPitchBytes || 2 * ldw > kMaxPitchBytes ||
      2 * dgu_pitch(inter) > 8 * kMaxPitchBytes)
    return QG_ERR_UNSUPPORTED;
  if (m > 0 && (!x || !w)) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(w, 16) || ldw % 8 != 0) return QG_ERR_ALIGNMENT;
  return QG_OK;
}

static qg_status gu_check(const void *gu, int32_t gu_type, int64_t ldgu, int64_t inter) {
  if (!gu) return QG_OK;
  if (!out_type(gu_type)) return QG_ERR_INVALID_ARGUMENT;
  if (ldgu < 2 * inter) return QG_ERR_SHAPE;
  return aligned(gu, 16) ? QG_OK : QG_ERR_ALIGNMENT;
}

// Workspaces: [split-K counters][partial tiles][gradient of the
// pre-activations][the pre-activations, where they are computed again].
struct FfnSpace {
  uint64_t partials = 0, dgu = 0, gu = 0;  // bytes
  uint64_t total() const {
    const uint64_t b = partials + dgu + gu;
    return b ? kSplitCounterBytes + b : 0;
  }
};
// (the choice of a shape depends on the pitch of the gradient, not on the caller's)
static FfnSpace ffn_space(int64_t m, int64_t k, int64_t inter, bool backward, bool recompute) {
  FfnSpace sp;
  if (m <= 0 || k <= 0 || inter <= 0 || m > (1ll << 30) || k > (1 << 22) || inter > (1 << 24)) return sp;
  FfnCall c = {};
  c.m = m;
  c.k = k;
  c.inter = inter;
  MmInfo i;
  if (!backward || recompute) {
    (void)launch_ffn_forward(c, nullptr, &i);
    sp.partials = i.bytes;
  }
  if (backward) {
    (void)launch_ffn_dx(c, nullptr, dgu_pitch(inter), nullptr, 0, nullptr, &i);
    sp.partials = std::max(sp.partials, i.bytes);
    (void)launch_ffn_dw(c, nullptr, dgu_pitch(inter), nullptr, 0, 0, nullptr, &i);
    sp.partials = std::max(sp.partials, i.bytes);
    sp.dgu = align_up((uint64_t)ffn_dgu_rows(m) * dgu_pitch(inter) * 2, 256);
    if (recompute) sp.gu = align_up((uint64_t)m * 2 * inter * 4, 256);
  }
  sp.partials = align_up(sp.partials, 256);
  return sp;
}
static void ffn_split_space(FfnCall *c, const FfnSpace &sp, void *ws) {
  if (!sp.partials) return;
  c->counters = (uint32_t *)ws;
  c->partials = (uint8_t *)ws + kSplitCounterBytes;
}
}  // namespace qg

using namespace qg;

extern "C" qg_status qg_quantize_int8(const void *x, int64_t rows, int64_t k, int64_t ldx, void *q, int64_t ldq,
                                      float *q_scales, hipStream_t stream) {
  if (rows < 0 || k < 0) return QG_ERR_INVALID_ARGUMENT;
  if (k % 8 != 0 || ldx < k || ldq < k) return QG_ERR_SHAPE;
  if (rows == 0 || k == 0) return QG_OK;
  if (!x || !q || !q_scales) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(q, 8) || ldq % 8 != 0 || !aligned(q_scales, 4))
    return QG_ERR_ALIGNMENT;
  return hip_status(launch_quantize_int8(x, rows, k, ldx, q, ldq, q_scales, stream));
}

extern "C" qg_status qg_gated_gemm_workspace_size(const qg_weight *w, int64_t m, uint32_t flags, uint64_t *bytes) {
  Layout L;
  const qg_status st = check_weight(w, &L);
  if (st != QG_OK) return st;
  if (!bytes || m < 0 || (flags & ~kI8Flags) != 0) return QG_ERR_INVALID_ARGUMENT;
  if (!L.i8) return QG_ERR_UNSUPPORTED;
  if (w->desc.n % 2 != 0) return QG_ERR_SHAPE;
  *bytes = i8_ws_bytes(*w, true, m, flags);
  return QG_OK;
}

extern "C" qg_status qg_gated_gemm(const qg_weight *w, const void *x, const void *x_scales, int64_t m, int64_t ldx,
                                   void *h, int32_t otype, int64_t ldh, int32_t act, void *ws, uint64_t ws_bytes,
                                   uint32_t flags, hipStream_t stream) {
  Layout L;
  const qg_status st = check_weight(w, &L);
  if (st != QG_OK) return st;
  if ((act != QG_ACT_SILU && act != QG_ACT_GELU_TANH) || (flags & ~kI8Flags) != 0) return QG_ERR_INVALID_ARGUMENT;
  if (!L.i8) return QG_ERR_UNSUPPORTED;
  if (w->desc.n % 2 != 0) return QG_ERR_SHAPE;
  return i8_product(w, L, true, x, x_scales, m, ldx, h, otype, ldh, act, ws, ws_bytes, flags, stream);
}

extern "C" qg_status qg_ffn_gated_workspace_size(int64_t m, int64_t k, int64_t inter, uint64_t *bytes) {
  if (!bytes || m < 0 || k < 0 || inter < 0) return QG_ERR_INVALID_ARGUMENT;
  *bytes = ffn_space(m, k, inter, false, false).total();
  return QG_OK;
}

extern "C" qg_status qg_ffn_gated(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k,
                                  int64_t inter, int32_t act, void *h, int64_t ldh, void *gu, int32_t gu_type,
                                  int64_t ldgu, void *ws, uint64_t ws_bytes, hipStream_t stream) {
  qg_status st = ffn_check(x, ldx, w, ldw, m, k, inter, act);
  if (st != QG_OK) return st;
  if (ldh < inter) return QG_ERR_SHAPE;
  if ((st = gu_check(gu, gu_type, ldgu, inter)) != QG_OK) return st;
  if (m == 0) return QG_OK;
  if (!h) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(h, 16)) return QG_ERR_ALIGNMENT;
  const FfnSpace sp = ffn_space(m, k, inter, false, false);
  if ((st = ws_check(sp.total(), ws, ws_bytes)) != QG_OK) return st;
  FfnCall c{x, ldx, w, ldw, m, k, inter, act, h, ldh, gu, ldgu, gu_type, nullptr, nullptr};
  ffn_split_space(&c, sp, ws);
  return hip_status(launch_ffn_forward(c, stream));
}

extern "C" qg_status qg_ffn_gated_backward_workspace_size(int64_t m, int64_t k, int64_t inter, int32_t recompute,
                                                          uint64_t *bytes) {
  if (!bytes || m < 0 || k < 0 || inter < 0) return QG_ERR_INVALID_ARGUMENT;
  *bytes = ffn_space(m, k, inter, true, recompute != 0).total();
  return QG_OK;
}

extern "C" qg_status qg_ffn_gated_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *dh,
                                           int64_t lddh, int64_t m, int64_t k, int64_t inter, int32_t act, void *dx,
                                           int64_t lddx, void *dw, int32_t dw_type, int64_t lddw, const void *gu,
                                           int32_t gu_type, int64_t ldgu, void *ws, uint64_t ws_bytes,
                                           hipStream_t stream) {
  qg_status st = ffn_check(x, ldx, w, ldw, m, k, inter, act);
  if (st != QG_OK) return st;
  if (dw && !out_type(dw_type)) return QG_ERR_INVALID_ARGUMENT;
  if (lddh < inter || (dx && lddx < k) || (dw && lddw < k)) return QG_ERR_SHAPE;
  if ((st = gu_check(gu, gu_type, ldgu, inter)) != QG_OK) return st;
  if (!aligned(dh, 2) || !aligned(dx, 16) || !aligned(dw, 16)) return QG_ERR_ALIGNMENT;
  if (m == 0)  // a sum over no tokens
    return dw ? hip_status(launch_ffn_zero(dw, lddw * el_of(dw_type), k * el_of(dw_type), 2 * inter, stream)) : QG_OK;
  if (!dh) return QG_ERR_INVALID_ARGUMENT;
  if (!dx && !dw) return QG_OK;
  const FfnSpace sp = ffn_space(m, k, inter, true, gu == nullptr);
  if ((st = ws_check(sp.total(), ws, ws_bytes)) != QG_OK) return st;
  uint8_t *dgu = (uint8_t *)ws + kSplitCounterBytes + sp.partials;
  FfnCall c{x, ldx, w, ldw, m, k, inter, act, nullptr, 0, const_cast<void *>(gu), ldgu, gu_type, nullptr, nullptr};
  ffn_split_space(&c, sp, ws);
  hipError_t e = hipSuccess;
  if (!gu) {  // the pre-activations again, in fp32
    c.gu = dgu + sp.dgu;
    c.ldgu = 2 * inter;
    c.gu_type = QG_O_F32;
    e = launch_ffn_forward(c, stream);
  }
  const int64_t ldd = dgu_pitch(inter);
  if (e == hipSuccess) e = launch_ffn_dgu(c, dh, lddh, dgu, ldd, stream);
  if (e == hipSuccess && dx) e = launch_ffn_dx(c, dgu, ldd, dx, lddx, stream);
  if (e == hipSuccess && dw) e = launch_ffn_dw(c, dgu, ldd, dw, dw_type, lddw, stream);
  return hip_status(e);
}

// Checks shared by the two directions of the token log probabilities.
static qg_status logprob_check(const void *logits, int32_t ltype, int64_t rows, int64_t vocab, int64_t ldl,
                               const void *tokens, float scale) {
  if (!out_type(ltype) || rows < 0 || vocab < 0 || !std::isfinite(scale) || !(scale > 0.f))
    return QG_ERR_INVALID_ARGUMENT;
  if (vocab == 0 || ldl < vocab) return QG_ERR_SHAPE;
  if (vocab > (1 << 24) || rows > (1ll << 30)) return QG_ERR_UNSUPPORTED;
  if (rows > 0 && !logits) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, el_of(ltype)) || !aligned(tokens, 4)) return QG_ERR_ALIGNMENT;
  return QG_OK;
}

extern "C" qg_status qg_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t top, uint64_t *bytes) {
  if (!bytes || rows < 0 || vocab < 0 || top < 0) return QG_ERR_INVALID_ARGUMENT;
  if (top > QG_MAX_ALTERNATIVES) return QG_ERR_UNSUPPORTED;
  *bytes = logprobs_ws_bytes(rows, vocab, top);
  return QG_OK;
}

extern "C" qg_status qg_token_logprobs(const void *logits, int32_t ltype, int64_t rows, int64_t vocab, int64_t ldl,
                                       const int32_t *tokens, float scale, int32_t top, float *logp, float *entropy,
                                       float *stats, int32_t *rank, int32_t *top_ids, float *top_logp, void *ws,
                                       uint64_t ws_bytes, hipStream_t stream) {
  const qg_status st = logprob_check(logits, ltype, rows, vocab, ldl, tokens, scale);
  if (st != QG_OK) return st;
  if (top < 0) return QG_ERR_INVALID_ARGUMENT;
  if (top > QG_MAX_ALTERNATIVES) return QG_ERR_UNSUPPORTED;
  if (rows == 0) return QG_OK;
  if ((!tokens && (logp || rank)) || (top > 0 && !top_ids && !top_logp)) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(stats, 4) || !aligned(rank, 4) || !aligned(top_ids, 4) ||
      !aligned(top_logp, 4))
    return QG_ERR_ALIGNMENT;
  const qg_status wst = ws_check(logprobs_ws_bytes(rows, vocab, top), ws, ws_bytes);
  if (wst != QG_OK) return wst;
  LogprobArgs a = {};
  a.logits = logits;
  a.f32 = ltype == QG_O_F32;
  a.rows = rows;
  a.vocab = vocab;
  a.ldl = ldl;
  a.tokens = tokens;
  a.scale = scale;
  a.top = top;
  a.logp = logp;
  a.entropy = entropy;
  a.stats = stats;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  return hip_status(launch_logprobs(a, ws, stream));
}

extern "C" qg_status qg_token_logprobs_backward(const void *logits, int32_t ltype, int64_t rows, int64_t vocab,
                                                int64_t ldl, const int32_t *tokens, float scale, const float *stats,
                                                const float *entropy, const float *dlogp, const float *dentropy,
                                                void *dlogits, int64_t lddl, hipStream_t stream) {
  const qg_status st = logprob_check(logits, ltype, rows, vocab, ldl, tokens, scale);
  if (st != QG_OK) return st;
  if (lddl < vocab) return QG_ERR_SHAPE;
  if (rows == 0) return QG_OK;
  if (!stats || !dlogits || (dlogp && !tokens) || (dentropy && !entropy)) return QG_ERR_INVALID_ARGUMENT;
  if (!aligned(dlogits, el_of(ltype)) || !aligned(stats, 4) || !aligned(entropy, 4) || !aligned(dlogp, 4) ||
      !aligned(dentropy, 4))
    return QG_ERR_ALIGNMENT;
  LogprobArgs a = {};
  a.logits = logits;
  a.f32 = ltype == QG_O_F32;
  a.rows = rows;
  a.vocab = vocab;
  a.ldl = ldl;
  a.tokens = tokens;
  a.scale = scale;
  a.stats = const_cast<float *>(stats);
  a.entropy = const_cast<float *>(entropy);
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dlogits = dlogits;
  a.lddl = lddl;
  return hip_status(launch_logprobs_backward(a, stream));
}
