"""GPU tests of the root-mean-square norm, its 8-bit outputs and its backward pass
against the formulas in 64 bits and, for the gradients, against differences.

Tolerances: fp32 sums of k terms are within k roundings (2^-24) of the sum of the
terms' magnitudes, whatever their order; each output is rounded once (half a
step: bf16 2^-8, e4m3 2^-4 of the value, int8 half a unit)."""
import numpy as np
import pytest
import torch

import norm_reference as ref
import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu
from norm_reference import D, U32

pytestmark = pytest.mark.gpu
NAN = float("nan")
QS = [qg.A_INT8_TOKEN, qg.A_FP8_TOKEN, qg.A_FP8_BLOCK, qg.A_MXFP8]
BF, F32 = qg.O_BF16, qg.O_F32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def padded(t, extra, fill=NAN):
    """The rows with a longer pitch and a row more, `fill` behind them."""
    d = torch.full((t.shape[0] + 1, t.shape[1] + extra), fill, dtype=t.dtype, device="cuda")
    d[:t.shape[0], :t.shape[1]] = t.cuda()
    return d


def rows_of(gen, rows, k, t, spread=1.0):
    return (torch.randn(rows, k, generator=gen) * spread).to(ref.types(t))


class Forward:
    def __init__(self, rows, k, x_type=BF, res_type=None, residual=True, seed=0, eps=1e-5, edit=None):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.k, self.x_type, self.res_type, self.eps = rows, k, x_type, res_type, eps
        self.x = rows_of(gen, rows, k, x_type)
        self.res = rows_of(gen, rows, k, res_type, 2.0) if res_type is not None and residual else None
        self.w = (1 + 0.3 * torch.randn(k, generator=gen)).to(torch.bfloat16)
        if edit:
            edit(self)
        self.s = ref.added(self.x, self.res, res_type)

    def run(self, y=True, q_type=qg.A_BF16, keep_sum=True, in_place=None):
        rows, k = self.rows, self.k
        xd, wd = padded(self.x, 8), padded(self.w[None], 8)[0]
        rd = None if self.res is None else padded(self.res, 16)
        sd = torch.full((rows + 1, k + 24), 7.0, dtype=ref.types(self.res_type), device="cuda") if self.res_type is not None and keep_sum else None
        if in_place:
            sd = {"x": xd, "residual": rd}[in_place]
        yd = torch.full((rows + 1, k + 8), 7.0, dtype=torch.bfloat16, device="cuda") if y else None
        qd = qs = None
        if q_type != qg.A_BF16:
            qd = torch.full((rows + 1, k + 8), 77, dtype=torch.uint8, device="cuda")
            per = {qg.A_MXFP8: k // 32, qg.A_FP8_BLOCK: -(-k // 128)}.get(q_type, 1)
            qs = torch.full((rows * per + 5,), 7, dtype=torch.uint8 if q_type == qg.A_MXFP8 else torch.float32, device="cuda")
        qg.rmsnorm(xd, self.x_type, k + 8, wd, self.eps, rows, k, residual=rd, res_type=self.res_type or 0, ldr=k + 16, sum=sd,
                   lds=sd.stride(0) if sd is not None else 0, y=yd, ldy=k + 8, q_type=q_type, q=qd, ldq=k + 8, q_scales=qs)
        torch.cuda.synchronize()
        # nothing behind the rows is written
        if sd is not None and not in_place:
            assert (sd[rows:] == 7).all() and (sd[:, k:] == 7).all()
        if y:
            assert (yd[rows:] == 7).all() and (yd[:, k:] == 7).all()
        if qd is not None:
            assert (qd[rows:] == 77).all() and (qd[:, k:] == 77).all() and (qs[rows * per:] == 7).all()
        cut = lambda t: None if t is None else t[:rows, :k].cpu()  # noqa: E731
        return cut(sd), cut(yd), cut(qd), None if qs is None else qs[:rows * per].view(rows, per).cpu()

    def check(self, out, q_type):
        sd, yd, qd, qs = out
        if sd is not None:
            assert torch.equal(sd.to(D), self.s)
        y, e = ref.norm(self.s, self.w.to(D), self.eps)
        if yd is not None:
            u = ref.half_step(torch.bfloat16)
            bound = y.abs() * (e + u * (1 + e)) + 2.0 ** -134   # (bf16 subnormals)
            assert ((yd.to(D) - y).abs() <= bound).all(), ((yd.to(D) - y).abs() - bound).max()
        if qd is None:
            return
        ideal, scale = ref.codes(y, q_type)
        if q_type == qg.A_MXFP8:
            got_scale = torch.ldexp(torch.ones_like(scale), qs.to(torch.int32) - 127)
            # a largest value that e carries over a power of two has the neighbouring scale
            most = ideal.view(self.rows, -1, 32).abs().amax(2)
            near = (most >= 512 * (1 - 3 * e)) | (most <= 256 * (1 + 3 * e))
            assert ((got_scale == scale) | near).all()
            ideal = ideal * (scale / got_scale).repeat_interleave(32, 1)
        else:
            assert ((qs.to(D) - scale).abs() <= scale * (e + 3 * U32)).all()
        if q_type == qg.A_INT8_TOKEN:
            off, step = (qd.view(torch.int8).to(D) - ideal).abs(), torch.full_like(ideal, 0.5)
        else:
            value = ideal.clamp(-448, 448)
            off = (qd.view(torch.float8_e4m3fn).to(D) - value).abs()
            # half a step of e4m3: 2^-4 relative, 2^-10 below the least normal 2^-6
            step = torch.maximum(value.abs() * 2.0 ** -4, torch.full_like(value, 2.0 ** -10))
        bound = step + ideal.abs() * (2 * e + 6 * U32)
        assert (off <= bound).all(), (off - bound).max()


SIZES = [(1, 8), (1, 512), (3, 520), (5, 1024), (2, 1032), (7, 2048), (3, 2056), (1, 4096), (67, 4096), (3, 4104), (2, 8192),
         (2, 8200), (3, 16384), (2, 16392), (3, 33000), (9, 136), (1030, 64)]


@pytest.mark.parametrize("rows,k", SIZES)
@pytest.mark.parametrize("x_type,res_type", [(BF, None), (F32, None), (BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_forward(rows, k, x_type, res_type):
    print(f"rmsnorm rows={rows} k={k} x={x_type} res={res_type}", flush=True)
    c = Forward(rows, k, x_type, res_type, seed=rows + k)
    for q_type in [qg.A_BF16] + QS:
        if q_type == qg.A_MXFP8 and k % 32:
            continue
        out = c.run(True, q_type)
        c.check(out, q_type)
        if q_type != qg.A_BF16:   # the codes alone: the same
            alone = c.run(False, q_type, keep_sum=False)
            assert torch.equal(alone[2], out[2]) and torch.equal(alone[3], out[3])


@pytest.mark.parametrize("rows,k", [(5, 1000), (4, 4096), (2, 20000)])
@pytest.mark.parametrize("t", [BF, F32])
def test_sum_in_place(rows, k, t):
    c = Forward(rows, k, t, t, seed=k)
    for q_type in (qg.A_BF16, qg.A_INT8_TOKEN):
        want = c.run(True, q_type)
        for where in ("x", "residual"):
            got = c.run(True, q_type, in_place=where)
            assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("x_type,res_type", [(BF, BF), (F32, BF), (BF, F32)])
def test_sum_without_a_residual(x_type, res_type):
    """A copy of x in the residual's type, and its norm."""
    c = Forward(6, 4096, x_type, res_type, residual=False, seed=3)
    c.check(c.run(True, qg.A_FP8_TOKEN), qg.A_FP8_TOKEN)


@pytest.mark.parametrize("k", [64, 4096, 16992])
def test_zero_rows_tiny_and_large_values(k):
    def edit(c):
        c.x[0] = 0
        c.x[1] *= 1e-30       # s^2 underflows: eps decides
        c.x[2] *= 1e15
        c.x[3] = 0
        c.x[3, k - 1] = 3.0   # one value
        c.x[4] = 0
        c.x[4, 0] = -1e-40    # codes' scales at their least

    c = Forward(6, k, F32, None, seed=5, edit=edit)
    for q_type in [qg.A_BF16] + QS:
        out = c.run(True, q_type)
        assert (out[1][0] == 0).all()
        if q_type != qg.A_BF16:
            assert (out[2][0] & 0x7F == 0).all() and (out[3][0] == (127 if q_type == qg.A_MXFP8 else 1)).all()
        if q_type in (qg.A_BF16, qg.A_INT8_TOKEN, qg.A_FP8_TOKEN, qg.A_FP8_BLOCK):
            c.check(out, q_type)


def test_a_row_of_nan_stays_its_own():
    c = Forward(9, 4096, BF, BF, seed=8, edit=lambda c: c.x.__setitem__((4, 17), NAN))
    good = Forward(9, 4096, BF, BF, seed=8)
    a, b = c.run(True, qg.A_FP8_TOKEN), good.run(True, qg.A_FP8_TOKEN)
    others = [i for i in range(9) if i != 4]
    assert all(torch.equal(p[others], q[others]) for p, q in zip(a, b))
    assert a[1][4].isnan().all()


def backward(s, s_type, w, eps, dy, dsum, want_dx=True, dw_type=F32, in_place=False, want_dw=True):
    rows, k = s.shape
    sd, dyd, wd = padded(s, 8), padded(dy, 16), w.cuda()
    dsd = None if dsum is None else padded(dsum, 8)
    dx = (dsd if in_place else torch.full((rows + 1, k + 8), 7.0, dtype=ref.types(s_type), device="cuda")) if want_dx else None
    dw = torch.full((k + 8,), 7.0, dtype=ref.types(dw_type), device="cuda") if want_dw else None
    n = qg.rmsnorm_backward_workspace_size(rows, k)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")   # (any contents)
    for _ in range(1 if in_place else 2):
        qg.rmsnorm_backward(sd, s_type, k + 8, wd, eps, rows, k, dyd, k + 16, dx, k + 8, dw, dw_type, ws if want_dw else None, n,
                            dsum=dsd, ldds=k + 8)
    torch.cuda.synchronize()
    assert (ws[:1 << 16] == 255).all()   # where a product's workspace has its counters
    if want_dx and not in_place:
        assert (dx[rows:] == 7).all() and (dx[:, k:] == 7).all()
    if want_dw:
        assert (dw[k:] == 7).all()
        dw = dw[:k].cpu()
    return dx[:rows, :k].cpu() if want_dx else None, dw


@pytest.mark.parametrize("rows,k", SIZES + [(700, 1024), (600, 2048), (1300, 520), (530, 20000)])
@pytest.mark.parametrize("s_type,summed", [(BF, True), (F32, True), (BF, False)])
def test_backward(rows, k, s_type, summed):
    print(f"rmsnorm backward rows={rows} k={k} s={s_type} dsum={summed}", flush=True)
    gen = torch.Generator().manual_seed(rows * 7 + k)
    s, dy = rows_of(gen, rows, k, s_type, 2.0), rows_of(gen, rows, k, BF)
    dsum = rows_of(gen, rows, k, s_type) if summed else None
    w = (1 + 0.3 * torch.randn(k, generator=gen)).to(torch.bfloat16)
    sD, wD, dyD = s.to(D), w.to(D), dy.to(D)
    dx, dw = ref.gradients(sD, wD, 1e-5, dyD, dsum.to(D) if summed else None)
    got_dx, got_dw = backward(s, s_type, w, 1e-5, dy, dsum)
    # r is off by e, the mean of g s by k roundings of the mean of its magnitudes
    e = (k / 2 + 8) * U32
    r = 1 / torch.sqrt((sD * sD).mean(1, keepdim=True) + 1e-5)
    g = (dyD * wD).abs()
    second = sD.abs() * r ** 3
    bound = (r * g + second * (g * sD.abs()).mean(1, keepdim=True)) * (4 * e + (k + 8) * U32)
    u = ref.half_step(ref.types(s_type))
    bound = bound + (u + 4 * U32) * (dx.abs() + bound) + 2 * U32 * (dx.abs() + (dsum.to(D).abs() if summed else 0)) + 1e-40
    assert ((got_dx.to(D) - dx).abs() <= bound).all(), ((got_dx.to(D) - dx).abs() - bound).max()
    dw_bound = (dyD * sD * r).abs().sum(0) * (e + (rows + 4) * U32) + 1e-40
    assert ((got_dw.to(D) - dw).abs() <= dw_bound).all(), ((got_dw.to(D) - dw).abs() - dw_bound).max()
    # each gradient alone, and dw rounded to bf16: the same values
    only, none = backward(s, s_type, w, 1e-5, dy, dsum, want_dw=False)
    assert none is None and torch.equal(only, got_dx)
    none, dw16 = backward(s, s_type, w, 1e-5, dy, dsum, want_dx=False, dw_type=BF)
    assert none is None and torch.equal(dw16, got_dw.to(torch.bfloat16))
    if summed:
        there, dw2 = backward(s, s_type, w, 1e-5, dy, dsum, in_place=True)
        assert torch.equal(there, got_dx) and torch.equal(dw2, got_dw)


def test_gradients_against_differences():
    """Along each gradient's own direction the loss sum(dy y) + sum(dsum s) has to
    change by the gradient's norm."""
    gen = torch.Generator().manual_seed(4)
    rows, k, eps = 7, 264, 1e-3
    s, dy, dsum = (rows_of(gen, rows, k, F32) for _ in range(3))
    dy = dy.to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(k, generator=gen)).to(torch.bfloat16)
    dx, dw = backward(s, F32, w, eps, dy, dsum)

    def loss(s, w):
        return (dy.to(D) * ref.norm(s, w, eps)[0]).sum() + (dsum.to(D) * s).sum()

    for name, at, grad, f in (("dx", s.to(D), dx.to(D), lambda t: loss(t, w.to(D))), ("dw", w.to(D), dw.to(D), lambda t: loss(s.to(D), t))):
        masks = [torch.ones_like(grad)]
        if grad.dim() == 2:
            for axis in (0, 1):
                for i in (0, grad.shape[axis] - 1):
                    m = torch.zeros_like(grad)
                    m.select(axis, i).fill_(1)
                    masks.append(m)
        for mask in masks:
            v = grad * mask
            n = v.norm()
            v, step = v / n, 1e-5
            slope = (f(at + step * v) - f(at - step * v)) / (2 * step)
            assert n > 0 and abs(slope - n) <= 1e-5 * n + 1e-6, name


def test_no_rows_and_the_gradient_of_none():
    c = torch.zeros(8, device="cuda")
    qg.rmsnorm(None, BF, 64, None, 1e-5, 0, 64, y=None)
    dw = torch.full((72,), 7.0, device="cuda")
    qg.rmsnorm_backward(None, BF, 64, None, 1e-5, 0, 64, None, 64, None, 64, dw, F32)
    assert (dw[:64] == 0).all() and (dw[64:] == 7).all() and (c == 0).all()


def test_another_stream_and_a_captured_graph():
    rows, k = 33, 4096
    c = Forward(rows, k, BF, BF, seed=2)
    x, res, w = c.x.cuda(), c.res.cuda(), c.w.cuda()
    dy = torch.randn(rows, k, device="cuda").to(torch.bfloat16)
    out = {n: torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda") for n in ("sum", "y", "dx")}
    q, qs, dw = torch.zeros(rows, k, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(k, device="cuda")
    n = qg.rmsnorm_backward_workspace_size(rows, k)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def step():
        qg.rmsnorm(x, BF, k, w, 1e-5, rows, k, residual=res, res_type=BF, ldr=k, sum=out["sum"], lds=k, y=out["y"], ldy=k,
                   q_type=qg.A_INT8_TOKEN, q=q, ldq=k, q_scales=qs)
        qg.rmsnorm_backward(out["sum"], BF, k, w, 1e-5, rows, k, dy, k, out["dx"], k, dw, F32, ws, n)

    step()
    torch.cuda.synchronize()
    every = list(out.values()) + [q, qs, dw]
    want = [t.clone() for t in every]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for t in every:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(every, want))
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        for t in every:
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(every, want)), i


# more rows than a launch has workgroups (4096 of one or of four rows): every workgroup
# or wave takes several in turn, and not all of them the last time
TURNS = [(12300, 1032), (16391, 512), (16401, 1000)]


@pytest.mark.parametrize("rows,k", TURNS)
@pytest.mark.parametrize("x_type,res_type", [(BF, BF), (F32, None)])
def test_forward_of_rows_in_turn(rows, k, x_type, res_type):
    test_forward(rows, k, x_type, res_type)


@pytest.mark.parametrize("rows,k", TURNS + [(9000, 2080), (36870, 64), (4101, 16416)])
@pytest.mark.parametrize("x_type,res_type", [(BF, BF), (F32, F32)])
def test_rows_in_turn_are_as_rows_apart(rows, k, x_type, res_type):
    """The same bits from one call and from calls of a thousand rows, each of which a workgroup of its own takes."""
    print(f"rmsnorm in turn rows={rows} k={k} x={x_type} res={res_type}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, k, generator=gen, device="cuda").to(ref.types(x_type))
    res = torch.randn(rows, k, generator=gen, device="cuda").to(ref.types(res_type))
    w = (1 + 0.3 * torch.randn(k, generator=gen, device="cuda")).to(torch.bfloat16)
    for q_type in QS:
        if q_type == qg.A_MXFP8 and k % 32:
            continue
        per = {qg.A_MXFP8: k // 32, qg.A_FP8_BLOCK: -(-k // 128)}.get(q_type, 1)
        outs = []
        for step in (rows, 1000):
            s, y, q = torch.zeros_like(res), torch.zeros_like(x, dtype=torch.bfloat16), torch.zeros_like(x, dtype=torch.uint8)
            qs = torch.zeros(rows, per, dtype=torch.uint8 if q_type == qg.A_MXFP8 else torch.float32, device="cuda")
            for r in range(0, rows, step):
                n = min(step, rows - r)
                qg.rmsnorm(x[r:], x_type, k, w, 1e-5, n, k, residual=res[r:], res_type=res_type, ldr=k, sum=s[r:], lds=k, y=y[r:], ldy=k,
                           q_type=q_type, q=q[r:], ldq=k, q_scales=qs[r:])
            outs.append((s, y, q, qs))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs)), q_type
        assert outs[0][1].float().abs().amax(1).min() > 0


@pytest.mark.parametrize("rows,k", [(6200, 520), (6203, 1024), (8197, 72), (1300, 1032)])
@pytest.mark.parametrize("s_type", [BF, F32])
def test_backward_of_rows_in_turn(rows, k, s_type):
    """512 workgroups of one or of four rows."""
    test_backward(rows, k, s_type, True)


@pytest.mark.parametrize("q_type", [qg.A_INT8_TOKEN, qg.A_FP8_TOKEN, qg.A_FP8_BLOCK])
def test_codes_by_the_reciprocal_and_by_division(q_type):
    """The codes are the nearest to y times the scale's reciprocal, bit for bit; the quantizers divide.  Rows of
    small whole numbers, whose sums are exact, so that y is known to the last bit.

    y and the row's largest |y| are off by 2^-24 of themselves, so is the scale; the quotient adds one rounding
    more, the reciprocal two: codes differ only where the quotient of the exact numbers is within 5 2^-24 of itself
    from a tie of two codes, and then by one.  (Evenly spread quotients: 2 * 127 * 5 * 2^-24 = 8e-5 of them for
    int8, 2 * 16 * 5 * 2^-24 = 1e-5 for e4m3; products of small numbers as here meet ties more often.)"""
    rows, k, eps = 64, 4096, 1e-5
    gen = torch.Generator().manual_seed(11)
    x = torch.randint(-32, 33, (rows, k), generator=gen).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(k, generator=gen)).to(torch.bfloat16)
    q = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    per = k // 128 if q_type == qg.A_FP8_BLOCK else 1
    qs = torch.zeros(rows, per, device="cuda")
    qg.rmsnorm(x.cuda(), BF, k, w.cuda(), eps, rows, k, q_type=q_type, q=q, ldq=k, q_scales=qs, y=None)
    torch.cuda.synchronize()
    # (numpy, whose square root and quotients are correctly rounded, as the kernel's are)
    one = np.float32(1)
    s, wf = x.float().numpy(), w.float().numpy()
    r = one / np.sqrt((s * s).sum(1, keepdims=True) / np.float32(k) + np.float32(eps))
    y = ((s * wf) * r).reshape(rows, per, k // per)
    most = np.abs((s * wf).reshape(rows, per, -1)).max(2, keepdims=True) * r[:, None]
    scale = most / np.float32(127 if q_type == qg.A_INT8_TOKEN else 448)
    assert np.array_equal(qs.cpu().numpy(), scale[:, :, 0])

    def codes(t):
        if q_type == qg.A_INT8_TOKEN:
            return torch.from_numpy(t).round().to(torch.int8).view(torch.uint8).view(rows, k)
        return torch.from_numpy(t).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, k)

    assert torch.equal(q.cpu(), codes(y * (one / scale)))
    step = (q.cpu().view(torch.int8).int() - codes(y / scale).view(torch.int8).int()).abs()
    assert step.max() <= 1
    sw = (x.double() * w.double()).view(rows, per, -1)
    exact = ((127 if q_type == qg.A_INT8_TOKEN else 448) * sw / sw.abs().amax(2, keepdim=True)).view(rows, k)
    unit = torch.ones_like(exact) if q_type == qg.A_INT8_TOKEN else torch.exp2(torch.floor(torch.log2(exact.abs())).clamp_min(-6) - 3)
    near = ((exact / unit - torch.floor(exact / unit) - 0.5).abs() * unit) <= 5 * 2.0 ** -24 * exact.abs()
    print(f"codes that differ: {int((step > 0).sum())} of {step.numel()}, near a tie: {int(near.sum())}", flush=True)
    assert not ((step > 0) & ~near).any()
