"""Host tests of the int8 layers' layout and of the refusals of the int8
products, the gated feed-forward block and the token log probabilities (no GPU:
every check comes before the first device call)."""
import ctypes

import numpy as np
import pytest

import quantized_gemm_qg_amd as qg

DEV = 1 << 20   # a well-aligned address that is never read


def layer(n=256, k=512, **kw):
    return qg.layer_desc(kw.pop("wtype", qg.W_INT8), n, k, kw.pop("group_size", k), atype=qg.A_INT8_TOKEN, **kw)


def bound(d):
    return qg.weight_bind(d, DEV, qg.packed_size(d))


def refuses(status, fn, *a, **kw):
    with pytest.raises(qg.QGError) as e:
        fn(*a, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=500), qg.QG_ERR_SHAPE), (dict(group_size=128), qg.QG_ERR_UNSUPPORTED), (dict(stype=qg.S_BF16), qg.QG_ERR_UNSUPPORTED),
    (dict(k=1 << 17), qg.QG_ERR_UNSUPPORTED), (dict(num_experts=2), qg.QG_ERR_UNSUPPORTED), (dict(n=0), qg.QG_ERR_SHAPE),
    (dict(wtype=qg.W_UINT8), qg.QG_ERR_UNSUPPORTED), (dict(wtype=qg.W_INT4), qg.QG_ERR_UNSUPPORTED),
    (dict(wtype=qg.W_FP8), qg.QG_ERR_UNSUPPORTED), (dict(wtype=qg.W_MXFP4, group_size=32, stype=qg.S_E8M0), qg.QG_ERR_UNSUPPORTED),
])
def test_layer_refusals(kw, status):
    refuses(status, qg.packed_size, layer(**kw))


@pytest.mark.parametrize("n,k", [(1, 32), (17, 160), (33, 512), (300, 96), (1030, 4096)])
def test_packed_layout(n, k):
    r = np.random.default_rng(n)
    codes, scales = r.integers(-128, 128, (n, k), dtype=np.int8), r.random(n, dtype=np.float32)
    d = layer(n, k)
    out = np.full(qg.packed_size(d), 0xAA, np.uint8)
    qg.repack_host(d, codes, scales, None, out)
    w = qg.weight_bind(d, DEV, out.nbytes)
    assert w.n_tiles == -(-n // 16) and w.k_blocks == -(-k // 128)
    blocks = out[:w.n_tiles * w.k_blocks * 2048].reshape(w.n_tiles, w.k_blocks, 2, 4, 16, 16).view(np.int8)
    padded = np.zeros((w.n_tiles * 16, w.k_blocks * 128), np.int8)
    padded[:n, :k] = codes
    # [tile, column, block, half, quarter, byte] -> [tile, block, half, quarter, column, byte]
    want = padded.reshape(w.n_tiles, 16, w.k_blocks, 2, 4, 16).transpose(0, 2, 3, 4, 1, 5)
    assert (blocks == want).all()
    s = out[w.scales_offset:w.scales_offset + w.n_tiles * 64].view(np.float32)
    assert (s[:n] == scales).all() and (s[n:] == 0).all()


def test_described_choice():
    """The description names the kernel that a call takes; a call whose tiles are
    split over k, and only such a call, needs a workspace."""
    w = bound(layer(4096, 14336))
    rows = {m: qg.describe_dispatch(w, m) for m in (1, 16, 17, 23, 128, 4096)}
    assert rows[1] == rows[16] == "i8_rows M<=16" and rows[17] == rows[23] == "i8_rows M<=32"
    assert rows[128].startswith("i8_tiled") and rows[4096].startswith("i8_tiled")
    assert qg.describe_dispatch(w, 1, qg.GEMM_QUANTIZE_X) == "i8_rows M<=16 quantizing"
    assert qg.describe_dispatch(w, 23, qg.GEMM_QUANTIZE_X) == rows[23]
    for m in (1, 23, 128, 333, 1000, 4096):
        assert ("splits" in qg.describe_dispatch(w, m)) == (qg.gemm_workspace_size_ex(w, m, 0) > 0), m


def test_int8_product_refusals():
    w = bound(layer())

    def gemm(x=DEV, xs=DEV, m=4, ldx=512, y=DEV, otype=qg.O_BF16, ldy=256, ws=DEV, wsb=1 << 30, flags=0, w=w):
        qg.gemm_ex(w, x, xs, m, ldx, y, otype, ldy, ws, wsb, flags, stream=0)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(x=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(y=None)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(xs=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(m=-1)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(otype=2)), (qg.QG_ERR_INVALID_ARGUMENT, dict(flags=4)),
                       (qg.QG_ERR_SHAPE, dict(ldx=511)), (qg.QG_ERR_SHAPE, dict(ldy=255)),
                       (qg.QG_ERR_ALIGNMENT, dict(x=DEV + 8)), (qg.QG_ERR_ALIGNMENT, dict(ldx=520)),
                       (qg.QG_ERR_ALIGNMENT, dict(xs=DEV + 2)), (qg.QG_ERR_ALIGNMENT, dict(y=DEV + 4)),
                       (qg.QG_ERR_ALIGNMENT, dict(ldy=257)),
                       (qg.QG_ERR_ALIGNMENT, dict(flags=qg.GEMM_QUANTIZE_X, ldx=516)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(flags=qg.GEMM_QUANTIZE_X, ws=None, m=400)),
                       (qg.QG_ERR_BUFFER_TOO_SMALL, dict(flags=qg.GEMM_QUANTIZE_X, wsb=1 << 16, m=400)),
                       (qg.QG_ERR_ALIGNMENT, dict(flags=qg.GEMM_QUANTIZE_X, ws=DEV + 16, m=400)),
                       (qg.QG_ERR_UNSUPPORTED, dict(ldx=1 << 24)), (qg.QG_ERR_UNSUPPORTED, dict(m=(1 << 30) + 1))):
        refuses(status, gemm, **kw)
    gemm(m=0, x=None, xs=None, y=None, ws=None, wsb=0)
    # the flag belongs to these layers, the rest of the library does not take them
    other = bound(qg.layer_desc(qg.W_INT4, 256, 512, 128))
    refuses(qg.QG_ERR_INVALID_ARGUMENT, gemm, w=other, flags=qg.GEMM_QUANTIZE_X)
    refuses(qg.QG_ERR_UNSUPPORTED, qg.gemm_autotune_workspace_size, w, 4)
    refuses(qg.QG_ERR_UNSUPPORTED, qg.moe_workspace_size, w, 4, 2)
    refuses(qg.QG_ERR_UNSUPPORTED, qg.moe_gemm, w, DEV, DEV, 0, DEV, DEV, 4, 2, DEV, 0, 1, DEV, 1 << 30, stream=0)
    assert "i8" in qg.describe_dispatch(w, 1) and "i8" in qg.describe_dispatch(w, 4096)


def test_quantize_int8_refusals():
    def q(x=DEV, rows=4, k=512, ldx=512, q=DEV, ldq=512, s=DEV):
        qg.quantize_int8(x, rows, k, ldx, q, ldq, s, stream=0)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(x=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(rows=-1)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(s=None)), (qg.QG_ERR_SHAPE, dict(k=516, ldx=520, ldq=520)),
                       (qg.QG_ERR_SHAPE, dict(ldq=504)), (qg.QG_ERR_ALIGNMENT, dict(ldx=516)),
                       (qg.QG_ERR_ALIGNMENT, dict(q=DEV + 4)), (qg.QG_ERR_ALIGNMENT, dict(s=DEV + 1))):
        refuses(status, q, **kw)
    q(rows=0, x=None)
    q(k=0)


def test_gated_gemm_refusals():
    w = bound(layer())

    def gated(w=w, x=DEV, xs=DEV, m=4, ldx=512, h=DEV, otype=qg.O_BF16, ldh=128, act=qg.ACT_SILU, ws=DEV, wsb=1 << 30, flags=0):
        qg.gated_gemm(w, x, xs, m, ldx, h, otype, ldh, act, ws, wsb, flags, stream=0)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(act=2)), (qg.QG_ERR_INVALID_ARGUMENT, dict(h=None)),
                       (qg.QG_ERR_SHAPE, dict(ldh=127)), (qg.QG_ERR_ALIGNMENT, dict(ldh=129)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(flags=8)), (qg.QG_ERR_SHAPE, dict(w=bound(layer(n=255)))),
                       (qg.QG_ERR_UNSUPPORTED, dict(w=bound(qg.layer_desc(qg.W_INT4, 256, 512, 128))))):
        refuses(status, gated, **kw)
    gated(m=0, x=None, h=None)
    refuses(qg.QG_ERR_SHAPE, qg.gated_gemm_workspace_size, bound(layer(n=255)), 4)


def test_ffn_refusals():
    def fwd(x=DEV, ldx=64, w=DEV, ldw=64, m=4, k=64, inter=48, act=0, h=DEV, ldh=48, ws=DEV, wsb=1 << 30, **kw):
        qg.ffn_gated(x, ldx, w, ldw, m, k, inter, act, h, ldh, ws, wsb, stream=0, **kw)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(x=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(w=None)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(h=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(act=7)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(m=-1)), (qg.QG_ERR_SHAPE, dict(k=60)), (qg.QG_ERR_SHAPE, dict(k=0)),
                       (qg.QG_ERR_SHAPE, dict(inter=0)), (qg.QG_ERR_SHAPE, dict(ldx=56)), (qg.QG_ERR_SHAPE, dict(ldw=56)),
                       (qg.QG_ERR_SHAPE, dict(ldh=47)), (qg.QG_ERR_ALIGNMENT, dict(ldx=68)), (qg.QG_ERR_ALIGNMENT, dict(w=DEV + 8)),
                       (qg.QG_ERR_ALIGNMENT, dict(h=DEV + 8)), (qg.QG_ERR_SHAPE, dict(gu=DEV, ldgu=95)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(gu=DEV, ldgu=96, gu_type=5)), (qg.QG_ERR_ALIGNMENT, dict(gu=DEV + 4, ldgu=96)),
                       (qg.QG_ERR_UNSUPPORTED, dict(ldx=1 << 23))):
        refuses(status, fwd, **kw)
    fwd(m=0, x=None, w=None, h=None)

    def bwd(dh=DEV, lddh=48, m=4, dx=DEV, lddx=64, dw=DEV, dw_type=0, lddw=64, ws=DEV, wsb=1 << 30, **kw):
        qg.ffn_gated_backward(DEV, 64, DEV, 64, dh, lddh, m, 64, 48, 0, dx, lddx, dw, dw_type, lddw, ws, wsb, stream=0, **kw)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(dh=None)), (qg.QG_ERR_SHAPE, dict(lddh=47)), (qg.QG_ERR_SHAPE, dict(lddx=63)),
                       (qg.QG_ERR_SHAPE, dict(lddw=63)), (qg.QG_ERR_INVALID_ARGUMENT, dict(dw_type=3)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(ws=None)), (qg.QG_ERR_BUFFER_TOO_SMALL, dict(wsb=100)),
                       (qg.QG_ERR_ALIGNMENT, dict(ws=DEV + 64)), (qg.QG_ERR_ALIGNMENT, dict(dx=DEV + 2)),
                       (qg.QG_ERR_SHAPE, dict(gu=DEV, ldgu=10))):
        refuses(status, bwd, **kw)
    small = qg.ffn_gated_backward_workspace_size(4, 64, 48)
    assert qg.ffn_gated_backward_workspace_size(4, 64, 48, recompute=True) > small
    refuses(qg.QG_ERR_BUFFER_TOO_SMALL, bwd, wsb=small)   # without gu the call needs more
    bwd(dx=None, dw=None)
    bwd(m=0, dw=None, dh=None)


def test_logprobs_refusals():
    def fwd(l=DEV, ltype=1, rows=4, vocab=100, ldl=100, tok=DEV, scale=1.0, top=5, logp=DEV, ent=DEV, rank=DEV, ids=DEV, tl=DEV,
            ws=DEV, wsb=1 << 30):
        qg.token_logprobs(l, ltype, rows, vocab, ldl, tok, scale, top, logp, ent, None, rank, ids, tl, ws, wsb, stream=0)

    for status, kw in ((qg.QG_ERR_INVALID_ARGUMENT, dict(l=None)), (qg.QG_ERR_INVALID_ARGUMENT, dict(ltype=2)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(rows=-1)), (qg.QG_ERR_SHAPE, dict(ldl=99)), (qg.QG_ERR_SHAPE, dict(vocab=0)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(scale=0.0)), (qg.QG_ERR_INVALID_ARGUMENT, dict(scale=float("nan"))),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(scale=float("inf"))), (qg.QG_ERR_INVALID_ARGUMENT, dict(tok=None)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(top=-1)), (qg.QG_ERR_UNSUPPORTED, dict(top=qg.MAX_ALTERNATIVES + 1)),
                       (qg.QG_ERR_INVALID_ARGUMENT, dict(ids=None, tl=None)), (qg.QG_ERR_ALIGNMENT, dict(l=DEV + 2)),
                       (qg.QG_ERR_ALIGNMENT, dict(tok=DEV + 2)), (qg.QG_ERR_ALIGNMENT, dict(rank=DEV + 2)),
                       (qg.QG_ERR_UNSUPPORTED, dict(vocab=(1 << 24) + 1, ldl=1 << 25))):
        refuses(status, fwd, **kw)
    fwd(rows=0, l=None, tok=None)

    def bwd(l=DEV, rows=4, tok=DEV, stats=DEV, ent=DEV, dlogp=DEV, dent=DEV, dl=DEV, lddl=100):
        qg.token_logprobs_backward(l, 1, rows, 100, 100, tok, 1.0, stats, ent, dlogp, dent, dl, lddl, stream=0)

    for kw in (dict(l=None), dict(stats=None), dict(dl=None), dict(tok=None), dict(ent=None)):
        refuses(qg.QG_ERR_INVALID_ARGUMENT, bwd, **kw)
    refuses(qg.QG_ERR_SHAPE, bwd, lddl=99)
    bwd(rows=0, l=None, dl=None)


def test_sizes_refuse_null_and_negative():
    assert qg._lib.qg_ffn_gated_workspace_size(1, 8, 1, None) == qg.QG_ERR_INVALID_ARGUMENT
    out = ctypes.c_uint64()
    assert qg._lib.qg_ffn_gated_backward_workspace_size(-1, 8, 1, 0, ctypes.byref(out)) == qg.QG_ERR_INVALID_ARGUMENT
    assert qg._lib.qg_token_logprobs_workspace_size(1, 100, 33, ctypes.byref(out)) == qg.QG_ERR_UNSUPPORTED


def test_described_choice_at_9_to_32_rows():
    """Both sides of the measured crossings of the few-rows and the tiled kernel."""
    def kernel(m, n, k):
        return qg.describe_dispatch(bound(layer(n, k)), m).split()[0]

    for m, n, k in ((16, 1000, 11264), (24, 1536, 8192), (24, 4096, 14336), (32, 4096, 8192), (20, 5120, 4096), (17, 7168, 4096),
                    (16, 14336, 8192), (8, 14336, 28672)):
        assert kernel(m, n, k) == "i8_rows", (m, n, k)
    for m, n, k in ((16, 1000, 14336), (28, 1536, 8192), (28, 4096, 14336), (32, 5120, 4096), (17, 5120, 11264), (24, 7168, 14336),
                    (16, 5120, 14336), (17, 8192, 4096), (33, 4096, 64)):
        assert kernel(m, n, k) == "i8_tiled", (m, n, k)
