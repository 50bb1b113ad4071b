"""Refusals of the root-mean-square norm, the low-rank adapters and the cross
entropy of a head (no GPU: every check comes before the first device call)."""
import ctypes

import pytest

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
    (SHAPE, dict(lddx=56)), (SHAPE, dict(dsum=DEV, ldds=8)), (ALIGNMENT, dict(dsum=DEV + 8, ldds=64)), (ALIGNMENT, dict(dx=DEV + 8)),
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
    assert qg.rmsnorm_backward_workspace_size(1 << 20, 1 << 24) <= 64 << 20
    assert qg._lib.qg_rmsnorm_backward_workspace_size(1, 64, None) == INVALID
    assert qg._lib.qg_rmsnorm_backward_workspace_size(1, -64, ctypes.byref(ctypes.c_uint64())) == INVALID
