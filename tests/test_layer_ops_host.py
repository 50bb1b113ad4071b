"""Refusals of the root-mean-square norm, the low-rank adapters and the cross
entropy of a head (no GPU: every check comes before the first device call)."""
import ctypes
import re

import pytest

import lora_sizes
import quantized_gemm_qg_amd as qg

DEV = 1 << 20   # a well-aligned address that is never read
INVALID, SHAPE, ALIGNMENT = qg.QG_ERR_INVALID_ARGUMENT, qg.QG_ERR_SHAPE, qg.QG_ERR_ALIGNMENT
UNSUPPORTED, SMALL = qg.QG_ERR_UNSUPPORTED, qg.QG_ERR_BUFFER_TOO_SMALL


def refuses(status, fn, **kw):
    with pytest.raises(qg.QGError) as e:
        fn(**kw)
    assert e.value.status == status, (kw, e.value)


def norm(x=DEV, x_type=qg.O_BF16, ldx=64, weight=DEV, eps=1e-5, rows=4, k=64, y=DEV, ldy=64, **kw):
    qg.rmsnorm(x, x_type, ldx, weight, eps, rows, k, y=y, ldy=ldy, stream=0, **kw)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(x=None)), (INVALID, dict(weight=None)), (INVALID, dict(y=None)), (INVALID, dict(x_type=2)), (INVALID, dict(rows=-1)),
    (INVALID, dict(k=-8)), (INVALID, dict(eps=0.0)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(eps=float("inf"))), (SHAPE, dict(k=60)), (SHAPE, dict(k=0)), (SHAPE, dict(ldx=56)), (SHAPE, dict(ldy=56)),
    (UNSUPPORTED, dict(k=(1 << 24) + 8, ldx=1 << 25, ldy=1 << 25)), (ALIGNMENT, dict(x=DEV + 8)), (ALIGNMENT, dict(weight=DEV + 8)),
    (ALIGNMENT, dict(y=DEV + 2)), (ALIGNMENT, dict(ldx=68)), (ALIGNMENT, dict(ldy=66)), (ALIGNMENT, dict(x_type=qg.O_F32, ldx=66)),
    (SHAPE, dict(residual=DEV, ldr=56)), (ALIGNMENT, dict(residual=DEV + 4, ldr=64)), (INVALID, dict(residual=DEV, ldr=64, res_type=3)),
    (INVALID, dict(sum=DEV, lds=72)), (INVALID, dict(sum=DEV, lds=64, res_type=qg.O_F32)),   # x's memory, another matrix
    (INVALID, dict(residual=2 * DEV, ldr=64, sum=2 * DEV, lds=72)),
    (SHAPE, dict(sum=DEV, lds=8)), (ALIGNMENT, dict(sum=DEV, lds=68)), (ALIGNMENT, dict(sum=DEV + 8, lds=64)),
    (INVALID, dict(q=DEV, ldq=64, q_scales=DEV)),                                # codes without their type
    (INVALID, dict(q_type=qg.A_INT8_TOKEN)),                                     # a type without codes
    (INVALID, dict(q_type=qg.A_INT8_TOKEN, q=DEV, ldq=64)), (INVALID, dict(q_type=5, q=DEV, ldq=64, q_scales=DEV)),
    (UNSUPPORTED, dict(q_type=qg.A_MXFP4, q=DEV, ldq=64, q_scales=DEV)),
    (SHAPE, dict(q_type=qg.A_MXFP8, q=DEV, ldq=80, q_scales=DEV, k=72, ldx=72, ldy=72)),
    (SHAPE, dict(q_type=qg.A_FP8_TOKEN, q=DEV, ldq=56, q_scales=DEV)),
    (ALIGNMENT, dict(q_type=qg.A_FP8_TOKEN, q=DEV + 4, ldq=64, q_scales=DEV)),
    (ALIGNMENT, dict(q_type=qg.A_FP8_BLOCK, q=DEV, ldq=68, q_scales=DEV)),
    (ALIGNMENT, dict(q_type=qg.A_FP8_BLOCK, q=DEV, ldq=64, q_scales=DEV + 2)),
])
def test_norm_refusals(status, kw):
    refuses(status, norm, **kw)


def test_norm_of_no_rows():
    norm(rows=0, x=None, weight=None, y=None)


def norm_back(s=DEV, s_type=qg.O_BF16, lds=64, weight=DEV, eps=1e-5, rows=4, k=64, dy=DEV, lddy=64, dx=DEV, lddx=64, dw=DEV,
              dw_type=qg.O_F32, ws=DEV, wsb=1 << 20, **kw):
    qg.rmsnorm_backward(s, s_type, lds, weight, eps, rows, k, dy, lddy, dx, lddx, dw, dw_type, ws, wsb, stream=0, **kw)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(s=None)), (INVALID, dict(dy=None)), (INVALID, dict(weight=None)), (INVALID, dict(s_type=2)), (INVALID, dict(dw_type=2)),
    (INVALID, dict(rows=-1)), (INVALID, dict(eps=0.0)), (SHAPE, dict(k=12)), (SHAPE, dict(lds=56)), (SHAPE, dict(lddy=56)),
    (SHAPE, dict(lddx=56)), (SHAPE, dict(dsum=DEV, ldds=8)), (INVALID, dict(dsum=DEV, ldds=72)), (ALIGNMENT, dict(dsum=DEV + 8, ldds=64)), (ALIGNMENT, dict(dx=DEV + 8)),
    (ALIGNMENT, dict(dw=DEV + 4)), (ALIGNMENT, dict(lddy=68)), (INVALID, dict(ws=None)), (SMALL, dict(wsb=100)),
    (ALIGNMENT, dict(ws=DEV + 64)), (UNSUPPORTED, dict(k=1 << 25, lds=1 << 25, lddy=1 << 25, lddx=1 << 25)),
])
def test_norm_backward_refusals(status, kw):
    refuses(status, norm_back, **kw)


def test_norm_backward_without_outputs():
    norm_back(dx=None, dw=None, ws=None, wsb=0)
    norm_back(rows=0, s=None, dy=None, weight=None, dw=None, ws=None, wsb=0)
    assert qg.rmsnorm_backward_workspace_size(0, 64) == 0
    # bounded, however many rows and however long they are
    assert qg.rmsnorm_backward_workspace_size(1 << 20, 1 << 24) <= (64 << 20) + (64 << 10)
    assert qg._lib.qg_rmsnorm_backward_workspace_size(1, 64, None) == INVALID
    assert qg._lib.qg_rmsnorm_backward_workspace_size(1, -64, ctypes.byref(ctypes.c_uint64())) == INVALID


def xent(x=DEV, ldx=64, w=DEV, ldw=64, m=4, k=64, vocab=100, targets=DEV, scale=1.0, loss=DEV, lse=DEV, ws=DEV, wsb=1 << 40):
    qg.linear_xent(x, ldx, w, ldw, m, k, vocab, targets, scale, loss, lse, ws, wsb, stream=0)


def xent_back(x=DEV, ldx=64, w=DEV, ldw=64, m=4, k=64, vocab=100, targets=DEV, scale=1.0, lse=DEV, dloss=DEV, dx=DEV, lddx=64, dw=DEV,
              dw_type=qg.O_F32, lddw=64, ws=DEV, wsb=1 << 40):
    qg.linear_xent_backward(x, ldx, w, ldw, m, k, vocab, targets, scale, lse, dloss, dx, lddx, dw, dw_type, lddw, ws, wsb, stream=0)


@pytest.mark.parametrize("fn", [xent, xent_back])
@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(m=-1)), (INVALID, dict(k=-8)), (INVALID, dict(vocab=-1)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(targets=None)), (SHAPE, dict(k=60)), (SHAPE, dict(k=0)), (SHAPE, dict(vocab=0)), (SHAPE, dict(ldx=56)),
    (SHAPE, dict(ldw=56)), (ALIGNMENT, dict(x=DEV + 8)), (ALIGNMENT, dict(w=DEV + 2)), (ALIGNMENT, dict(ldx=68)),
    (ALIGNMENT, dict(ldw=68)), (ALIGNMENT, dict(targets=DEV + 2)), (ALIGNMENT, dict(lse=DEV + 2)), (INVALID, dict(ws=None)),
    (SMALL, dict(wsb=1 << 16)), (ALIGNMENT, dict(ws=DEV + 64)), (UNSUPPORTED, dict(ldx=1 << 23)), (UNSUPPORTED, dict(ldw=1 << 23)),
    (UNSUPPORTED, dict(vocab=(1 << 24) + 1)), (UNSUPPORTED, dict(m=(1 << 30) + 1)),
])
def test_xent_refusals(fn, status, kw):
    refuses(status, fn, **kw)


@pytest.mark.parametrize("status,kw", [(INVALID, dict(loss=None, lse=None)), (ALIGNMENT, dict(loss=DEV + 1))])
def test_xent_forward_refusals(status, kw):
    refuses(status, xent, **kw)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(lse=None)), (INVALID, dict(dloss=None)), (INVALID, dict(dw_type=2)), (SHAPE, dict(lddx=56)), (SHAPE, dict(lddw=63)),
    (ALIGNMENT, dict(dx=DEV + 2)), (ALIGNMENT, dict(dw=DEV + 4)), (ALIGNMENT, dict(dloss=DEV + 2)),
])
def test_xent_backward_refusals(status, kw):
    refuses(status, xent_back, **kw)


def test_xent_without_work():
    xent(m=0, x=None, w=None, targets=None, loss=None, lse=None, ws=None, wsb=0)
    xent_back(m=0, dw=None, x=None, w=None, targets=None, lse=None, dloss=None, ws=None, wsb=0)
    xent_back(dx=None, dw=None, ws=None, wsb=0)
    for size in (qg.linear_xent_workspace_size, qg.linear_xent_backward_workspace_size):
        assert size(0, 64, 100) == size(4, 0, 100) == size(4, 64, 0) == 0
    for fn in (qg._lib.qg_linear_xent_workspace_size, qg._lib.qg_linear_xent_backward_workspace_size):
        assert fn(4, 64, 100, None) == INVALID and fn(-1, 64, 100, ctypes.byref(ctypes.c_uint64())) == INVALID


def test_xent_memory_does_not_grow_with_the_vocabulary():
    """The logits' gradient of a piece, whatever the vocabulary; many tokens: at
    least 8192 columns of it."""
    m, k = 4096, 4096
    fixed = 48 << 20   # partial tiles at most
    assert qg.linear_xent_backward_workspace_size(m, k, 1 << 24) <= (128 << 20) + 4 * m * k + fixed + (1 << 20)
    assert qg.linear_xent_backward_workspace_size(1 << 20, 64, 1 << 20) <= (1 << 20) * (8192 * 2 + 4 * 64 + 4) + fixed + (1 << 20)


def lora(x=DEV, ldx=64, a=DEV, lda=64, b=DEV, ldb=16, scales=DEV, adapters=3, rank=16, rows=DEV, offsets=DEV, m=4, k=64, n=100, y=DEV,
         y_type=qg.O_BF16, ldy=100, ws=DEV, wsb=1 << 30):
    qg.lora(x, ldx, a, lda, b, ldb, scales, adapters, rank, rows, offsets, m, k, n, y, y_type, ldy, ws, wsb, stream=0)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(x=None)), (INVALID, dict(a=None)), (INVALID, dict(b=None)), (INVALID, dict(rows=None)), (INVALID, dict(offsets=None)),
    (INVALID, dict(y=None)), (INVALID, dict(y_type=2)), (INVALID, dict(m=-1)), (INVALID, dict(k=-8)), (INVALID, dict(n=-1)),
    (INVALID, dict(adapters=0)), (INVALID, dict(rank=0)), (SHAPE, dict(k=60)), (SHAPE, dict(k=0)), (SHAPE, dict(n=0)),
    (SHAPE, dict(rank=12, ldb=16)), (SHAPE, dict(ldx=56)), (SHAPE, dict(lda=56)), (SHAPE, dict(ldb=8)), (SHAPE, dict(ldy=99)),
    (UNSUPPORTED, dict(rank=264, ldb=264)), (UNSUPPORTED, dict(adapters=1025)), (UNSUPPORTED, dict(m=(1 << 21) + 1)),
    (UNSUPPORTED, dict(n=(1 << 24) + 1, ldy=1 << 25)), (ALIGNMENT, dict(x=DEV + 8)), (ALIGNMENT, dict(a=DEV + 8)),
    (ALIGNMENT, dict(b=DEV + 8)), (ALIGNMENT, dict(ldx=68)), (ALIGNMENT, dict(lda=68)), (ALIGNMENT, dict(ldb=20)),
    (ALIGNMENT, dict(y=DEV + 1)), (ALIGNMENT, dict(y=DEV + 2, y_type=qg.O_F32)), (ALIGNMENT, dict(scales=DEV + 2)),
    (ALIGNMENT, dict(rows=DEV + 2)), (ALIGNMENT, dict(offsets=DEV + 1)), (INVALID, dict(rank=128, ldb=128, ws=None)), (SMALL, dict(rank=128, ldb=128, wsb=16)),
    (ALIGNMENT, dict(rank=128, ldb=128, ws=DEV + 64)),
])
def test_lora_refusals(status, kw):
    refuses(status, lora, **kw)


def test_lora_sizes():
    lora(m=0, x=None, a=None, b=None, rows=None, offsets=None, y=None, ws=None, wsb=0)
    out = ctypes.c_uint64()
    size = lambda m, k, n, adapters, rank: qg._lib.qg_lora_workspace_size(m, k, n, adapters, rank, ctypes.byref(out))  # noqa: E731
    assert qg._lib.qg_lora_workspace_size(1, 64, 8, 1, 8, None) == INVALID
    assert size(-1, 64, 8, 1, 8) == INVALID and size(1, 64, 8, 0, 8) == INVALID and size(1, 60, 8, 1, 8) == SHAPE
    assert size(1, 64, 8, 1, 264) == UNSUPPORTED
    # none where one launch does both products, and what fp32 parts of the low-rank rows take where two do
    assert qg.lora_workspace_size(1, 4096, 4096, 8, 16) == qg.lora_workspace_size(16, 4096, 4096, 8, 32) == 0
    assert qg.lora_workspace_size(4096, 4096, 14336, 6, 64) == (64 << 10) + 4096 * 64 * 4


def test_a_workspace_of_the_adapters_serves_fewer_rows():
    """A program allocates once, for its largest batch."""
    for k, n, adapters, rank in ((4096, 14336, 1, 16), (4096, 14336, 6, 64), (520, 300, 3, 128), (8192, 90, 40, 256), (264, 700, 1000, 8)):
        for most in (20, 300, 1023, 2048, 2300):
            size = qg.lora_workspace_size(most, k, n, adapters, rank)
            for m in range(1, most):
                need = qg.lora_workspace_size(m, k, n, adapters, rank)
                assert need <= size, (m, most, k, n, adapters, rank)
                if need:   # (the size is looked at before the alignment, which ends the call here)
                    refuses(ALIGNMENT, lora, m=m, k=k, ldx=k, lda=k, n=n, ldy=n, adapters=adapters, rank=rank, ldb=rank, ws=DEV + 64,
                            wsb=size)


@pytest.mark.parametrize("size,call", [(qg.linear_xent_workspace_size, xent), (qg.linear_xent_backward_workspace_size, xent_back)])
@pytest.mark.parametrize("k,vocab,upto", [(4096, 3000, 1100), (1024, 128000, 700), (64, 50, 300), (520, 1100001, 70), (1032, 38531, 600)])
def test_a_workspace_of_the_cross_entropy_serves_fewer_tokens(size, call, k, vocab, upto):
    sizes = [size(m, k, vocab) for m in range(upto + 1)]
    assert sizes == sorted(sizes)
    sizes += [size(m, k, vocab) for m in (5000, 8191, 8192, 8193, 20000, 70000, 1 << 20)]
    assert sizes == sorted(sizes)
    more = dict(lddx=k, lddw=k) if call is xent_back else {}
    for largest in (20, 33, 64, upto):
        for m in range(1, largest + 1):   # (the size is looked at before the alignment, which ends the call here)
            refuses(ALIGNMENT, call, m=m, k=k, ldx=k, ldw=k, vocab=vocab, ws=DEV + 64, wsb=sizes[largest], **more)


def test_a_workspace_of_the_norm_serves_fewer_rows():
    for k in (64, 1024, 1032, 4096, 1 << 20):
        sizes = [qg.rmsnorm_backward_workspace_size(rows, k) for rows in [*range(700), 2047, 2048, 2049, 1 << 20]]
        assert sizes == sorted(sizes)


def test_the_adapters_sizes_reach_every_kernel():
    """The GPU tests run EVERY_KERNEL; a change of the rules must not turn them away from a kernel."""
    for y_type in (qg.O_BF16, qg.O_F32):
        small, down, parts, up, side, zeros, twice, tails = (set() for _ in range(8))
        for m, k, n, rank, adapters in lora_sizes.EVERY_KERNEL:
            t = lora_sizes.taken(m, k, n, rank, adapters, y_type)
            if "splits" not in t:
                small.add(t["NB"])
                continue
            s, stages = t["splits"], -(-k // 64)
            down.add((t["NB"], 1 if s == 1 else 2 if s < 5 else 5))
            parts |= {name for name, yes in (("all", s == 16), ("empty", (s - 1) * -(-stages // s) >= stages), ("group", s > 4 and s % 4))
                      if yes}
            up.add((t["RB"], t["SD"], min(t["chunks"], 2)))
            if rank <= 16:
                side.add((rank, t["RB"]))
            elif rank // 8 % (4 * t["SD"]):
                zeros.add((t["RB"], t["SD"]))
            if rank > 128:
                twice.add(t["RB"])   # two groups of the rank
            tails.add((n % 8 != 0, t["RB"]))
        assert small == {1, 2, 4}
        assert down == {(nb, s) for nb in (1, 2, 4, 8, 16) for s in (1, 2, 5)} and parts == {"all", "empty", "group"}
        assert up == {(rb, sd, chunks) for rb in (1, 2, 4) for sd in (1, 2, 4) for chunks in (1, 2)}
        assert side == {(rank, rb) for rank in (8, 16) for rb in (1, 2, 4)}
        assert zeros == {(rb, sd) for rb in (1, 2, 4) for sd in (1, 2, 4)}
        assert twice == {1, 2, 4} and tails == {(odd, rb) for odd in (False, True) for rb in (1, 2, 4)}


def test_describe_lora():
    assert qg.describe_lora(0, 64, 100, 3, 16, qg.O_BF16) == "nothing"
    assert qg.describe_lora(1, 4096, 4096, 8, 16, qg.O_BF16) == "lora_small NB=1"
    out = ctypes.create_string_buffer(64)
    call = lambda *a: qg._lib.qg_describe_lora(*a)  # noqa: E731
    assert call(1, 64, 100, 3, 16, 2, out, 64) == INVALID and call(1, 64, 100, 3, 16, qg.O_F32, None, 64) == INVALID
    assert call(1, 64, 100, 3, 16, qg.O_F32, out, 0) == INVALID and call(-1, 64, 100, 3, 16, qg.O_F32, out, 64) == INVALID
    assert call(1, 60, 100, 3, 16, qg.O_F32, out, 64) == SHAPE and call(1, 64, 100, 3, 264, qg.O_F32, out, 64) == UNSUPPORTED


def test_the_cross_entropys_sizes_reach_every_tile_shape():
    """Every compiled shape of the four products, whole and, where it may, in parts of the contraction: a change of
    the cost model must not turn the GPU tests away from one."""
    import test_gpu_xent as gpu
    reached = set()
    for size in gpu.SIZES + gpu.TILES + gpu.MORE_TILES:
        for name, bm, bn, stages, splits in re.findall(r"(logits|d|dx|dw) BM=(\d+) BN=(\d+) stages=(\d+) splits=(\d+)",
                                                       qg.describe_linear_xent(*size)):
            reached.add((name, int(bm), int(bn), int(stages), int(splits) > 1))
    whole = {("dw", 256, 256, 2)} | {(name, bm, 256, 2) for name in ("logits", "d") for bm in (192, 256)}
    both = {("dx", 256, 256, 2), ("dx", 128, 128, 4), ("dx", 64, 128, 4), ("dx", 32, 128, 4), ("dw", 128, 128, 2), ("dw", 128, 128, 4)}
    both |= {(name, *t) for name in ("logits", "d") for t in ((128, 128, 2), (128, 128, 4), (64, 128, 3), (32, 128, 4))}
    assert reached == {(*t, False) for t in whole | both} | {(*t, True) for t in both}


def test_describe_linear_xent():
    assert qg.describe_linear_xent(0, 64, 100) == "nothing"
    assert qg.describe_linear_xent(20, 16, 1100001).count(" x ") == 2   # two pieces, the last one shorter
    assert "; 8 x 16384: d " in qg.describe_linear_xent(4096, 4096, 131072)
    out = ctypes.create_string_buffer(64)
    call = lambda *a: qg._lib.qg_describe_linear_xent(*a)  # noqa: E731
    assert call(1, 64, 100, None, 64) == INVALID and call(1, 64, 100, out, 0) == INVALID and call(-1, 64, 100, out, 64) == INVALID
    assert call(1, 60, 100, out, 64) == SHAPE and call(1, 64, 0, out, 64) == SHAPE and call(1, 64, (1 << 24) + 1, out, 64) == UNSUPPORTED
