"""GPU tests of the head's cross entropy and its gradients against the formulas in
64 bits and, for the gradients, against differences.

Tolerances: an fp32 sum of K products is within K 2^-23 of the sum of the
products' magnitudes; the exponentials' sums are trees of less than 200 + V / 2048
additions; d is rounded once to bf16 (2^-8; in two parts 2^-16), outputs once."""
import pytest
import torch

import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
D = torch.float64
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def padded(t, extra):
    """The rows with a longer pitch and a row more, NaN behind them."""
    d = torch.full((t.shape[0] + 1, t.shape[1] + extra), NAN, dtype=t.dtype, device="cuda")
    d[:t.shape[0], :t.shape[1]] = t
    return d


class Case:
    """Inputs on the GPU and the formulas' results there in 64 bits."""

    def __init__(self, m, k, vocab, seed=0, scale=1.0, ignore=0.2, edit=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.m, self.k, self.vocab, self.scale = m, k, vocab, scale
        w = rand(vocab, k) * (1.5 / k ** 0.5)
        target = torch.randint(vocab, (m,), generator=gen, device="cuda")
        # the first and the last token, as edges of tiles
        target[0] = vocab - 1
        if m > 3:
            target[1], target[2] = 0, min(vocab - 1, 128)
        x = rand(m, k) + 2.0 * w[target] * torch.rand(m, 1, generator=gen, device="cuda")
        self.x, self.w = x.to(torch.bfloat16), w.to(torch.bfloat16)
        self.targets = target.to(torch.int32)
        if m > 1:
            drop = torch.rand(m, generator=gen, device="cuda") < ignore
            drop[0] = False
            bad = torch.tensor([-100, -1, vocab, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
            self.targets = torch.where(drop, bad[torch.arange(m, device="cuda") % 4], self.targets)
        self.dloss = torch.rand(m, generator=gen, device="cuda") + 0.5
        if edit:
            edit(self)
        self.xd, self.wd = padded(self.x, 8), padded(self.w, 16)
        self.fwd_bytes = qg.linear_xent_workspace_size(m, k, vocab)
        self.bwd_bytes = qg.linear_xent_backward_workspace_size(m, k, vocab)
        self.ws = torch.zeros(max(self.fwd_bytes, self.bwd_bytes), dtype=torch.uint8, device="cuda")

    def solve(self):
        x, w = self.x.to(D), self.w.to(D)
        self.z = self.scale * torch.mm(x, w.t().contiguous())
        self.e_z = self.scale * self.k * 2 * U32 * torch.mm(x.abs(), w.abs().t().contiguous())
        self.lse = torch.logsumexp(self.z, 1)
        self.e_lse = self.e_z.amax(1) + (200 + self.vocab / 2048 + 40) * U32 + 2 * U32 * self.lse.abs()
        t = self.targets.long()
        self.counts = (t >= 0) & (t < self.vocab)
        self.rows = self.counts.nonzero()[:, 0]
        self.loss = torch.zeros_like(self.lse)
        self.loss[self.rows] = self.lse[self.rows] - self.z[self.rows, t[self.rows]]
        # (scale (largest - target's): a rounding of the difference's own size)
        gap = self.z.amax(1) - self.z.gather(1, t.clamp(0, self.vocab - 1)[:, None])[:, 0]
        self.e_loss = self.e_lse + self.e_z.amax(1) + 4 * U32 * gap.abs()

    def forward(self, loss=True, lse=True):
        out = [torch.full((self.m + 3,), 7.0, device="cuda") if wanted else None for wanted in (loss, lse)]
        for _ in range(2):
            qg.linear_xent(self.xd, self.k + 8, self.wd, self.k + 16, self.m, self.k, self.vocab, self.targets if loss else None,
                           self.scale, *out, self.ws, self.fwd_bytes)
        torch.cuda.synchronize()
        assert all(t is None or (t[self.m:] == 7).all() for t in out)
        return [None if t is None else t[:self.m] for t in out]

    def backward(self, lse, want_dx=True, dw_type=qg.O_F32, want_dw=True, twice=True):
        m, k, vocab = self.m, self.k, self.vocab
        dx = torch.full((m + 1, k + 8), 7.0, dtype=torch.bfloat16, device="cuda") if want_dx else None
        t = torch.float32 if dw_type == qg.O_F32 else torch.bfloat16
        dw = torch.full((vocab + 1, k + 4), 7.0, dtype=t, device="cuda") if want_dw else None
        for _ in range(2 if twice else 1):
            qg.linear_xent_backward(self.xd, k + 8, self.wd, k + 16, m, k, vocab, self.targets, self.scale, lse, self.dloss, dx, k + 8,
                                    dw, dw_type, k + 4, self.ws, self.bwd_bytes)
        torch.cuda.synchronize()
        assert (self.ws[:65536] == 0).all()   # arrival counters
        if want_dx:
            assert (dx[m:] == 7).all() and (dx[:, k:] == 7).all()
            dx = dx[:m, :k]
        if want_dw:
            assert (dw[vocab:] == 7).all() and (dw[:, k:] == 7).all()
            dw = dw[:vocab, :k]
        return dx, dw

    def gradients(self, u_dx, u_dw):
        """dx, dw and bounds on their errors before the outputs' rounding; u: of d's."""
        m, k, t = self.m, self.k, self.targets.long()
        x, w = self.x.to(D), self.w.to(D)
        weight = torch.where(self.counts, self.dloss.to(D), torch.zeros(m, dtype=D, device="cuda"))[:, None]
        p = torch.exp(self.z - self.lse[:, None])
        e = p * (self.e_z + self.e_lse[:, None] + 4 * U32 * (self.z.abs() + self.lse[:, None].abs()) + 8 * U32)
        hit = torch.zeros_like(p)
        hit[self.rows, t[self.rows]] = 1
        d = weight * (p - hit) * self.scale
        e = weight.abs() * self.scale * (e + 3 * U32 * (p + hit))
        dx, dw = torch.mm(d, w), torch.mm(d.t().contiguous(), x)
        grown = d.abs() + e
        ex, ew = e + u_dx * grown, e + u_dw * grown
        pieces = 2 + self.vocab // 4096
        b_dx = torch.mm(ex + (self.vocab * 2 + pieces) * U32 * grown, w.abs())
        b_dw = torch.mm((ew + (m * 2 + 4) * U32 * grown).t().contiguous(), x.abs())
        return dx, dw, b_dx, b_dw


def within(got, want, bound):
    off = (got.to(D) - want).abs() - bound
    assert (off <= 0).all(), f"{off.max().item():.3g} over the bound"


SIZES = [(1, 8, 1), (1, 264, 1000), (1, 4096, 515), (2, 72, 33), (5, 512, 130), (16, 128, 517), (17, 136, 45), (32, 1032, 300),
         (33, 520, 129), (40, 72, 1000), (61, 2048, 3003), (65, 72, 257), (100, 264, 128), (129, 1032, 700), (192, 136, 3001),
         (257, 264, 2001), (300, 520, 14000), (384, 1032, 9001), (600, 40, 90), (1100, 128, 310), (1345, 264, 12000)]


@pytest.mark.parametrize("m,k,vocab", SIZES)
def test_forward_and_backward(m, k, vocab):
    print(f"xent m={m} k={k} vocab={vocab}", flush=True)
    c = Case(m, k, vocab, seed=m + k, scale=1.0 if m % 2 else 0.7)
    c.solve()
    loss, lse = c.forward()
    within(lse, c.lse, c.e_lse)
    within(loss, c.loss, c.e_loss)
    assert (loss[~c.counts] == 0).all()
    alone, none = c.forward(lse=False)
    none2, lse2 = c.forward(loss=False)
    assert none is None and none2 is None and torch.equal(alone, loss) and torch.equal(lse2, lse)
    few = 2.0 ** -16
    dx, dw, b_dx, b_dw = c.gradients(few if m <= 16 else U16, few if m <= 32 else U16)
    got_dx, got_dw = c.backward(lse)
    within(got_dx, dx, b_dx * (1 + U16) + U16 * dx.abs() + 1e-37)
    within(got_dw, dw, b_dw + 2 * U32 * dw.abs() + 1e-37)
    assert (got_dx[~c.counts] == 0).all()
    if m * vocab > 1000:   # the roundings of d are independent: far nearer in the 2-norm
        assert (got_dw.to(D) - dw).norm() <= (few if m <= 32 else U16) * dw.norm()
        assert (got_dx.to(D) - dx).norm() <= 2 * U16 * dx.norm()
    only, none = c.backward(lse, want_dw=False)
    none2, dw16 = c.backward(lse, want_dx=False, dw_type=qg.O_BF16)
    assert none is None and none2 is None and torch.equal(only, got_dx)
    assert torch.equal(dw16, got_dw.to(torch.bfloat16))


# every tile shape of the three products, whole and in parts of the contraction
TILES = [(33, 16, 34), (34, 16, 32871), (1379, 16, 1204), (686, 16, 35037), (909, 1216, 30), (2747, 1800, 30), (2713, 808, 678),
         (2803, 2832, 264), (579, 3280, 7231), (2315, 3408, 954), (2953, 1408, 3564)]


@pytest.mark.parametrize("m,k,vocab", TILES)
def test_every_tile_shape(m, k, vocab):
    test_forward_and_backward(m, k, vocab)


@pytest.mark.parametrize("m,k,vocab", [(1, 8, 1100000), (20, 16, 1100001), (9000, 64, 20003), (40, 24, 2200000)])
def test_several_pieces(m, k, vocab):
    print(f"xent pieces m={m} k={k} vocab={vocab}", flush=True)
    c = Case(m, k, vocab, seed=vocab % 97)
    c.solve()
    _, lse = c.forward()
    within(lse, c.lse, c.e_lse)
    few = 2.0 ** -16
    dx, dw, b_dx, b_dw = c.gradients(few if m <= 16 else U16, few if m <= 32 else U16)
    del c.z, c.e_z
    got_dx, got_dw = c.backward(lse)
    within(got_dx, dx, b_dx * (1 + U16) + U16 * dx.abs() + 1e-37)
    within(got_dw, dw, b_dw + 2 * U32 * dw.abs() + 1e-37)


@pytest.mark.parametrize("m", [3, 40, 200])
def test_weights_of_zero_and_of_many_sizes(m):
    """Gradients of the losses from 1e-30 to 1e3, zeros among them: relative to the
    largest one nothing underflows that an fp32 product would hold."""
    def edit(c):
        c.dloss = torch.logspace(-30, 3, m, device="cuda")
        c.dloss[m // 2] = 0
        c.targets = c.targets.clamp(0, c.vocab - 1)

    c = Case(m, 136, 501, seed=m, edit=edit, ignore=0)
    c.solve()
    _, lse = c.forward()
    few = 2.0 ** -16
    dx, dw, b_dx, b_dw = c.gradients(few if m <= 16 else U16, few if m <= 32 else U16)
    got_dx, got_dw = c.backward(lse)
    within(got_dx, dx, b_dx * (1 + U16) + U16 * dx.abs() + 1e-36)
    within(got_dw, dw, b_dw + 2 * U32 * dw.abs() + 1e-36)
    assert (got_dx[m // 2] == 0).all()
    c.dloss.zero_()
    got_dx, got_dw = c.backward(lse)
    assert (got_dx == 0).all() and (got_dw == 0).all()


def test_all_rows_ignored():
    c = Case(50, 72, 300, edit=lambda c: c.targets.fill_(-100))
    loss, lse = c.forward()
    assert (loss == 0).all() and lse.isfinite().all()
    dx, dw = c.backward(lse)
    assert (dx == 0).all() and (dw == 0).all()


def test_certain_tokens():
    """Losses near 0: the target's logit far above the others."""
    def edit(c):
        c.x = (40.0 * c.w[c.targets.long()].float()).to(torch.bfloat16)

    c = Case(70, 264, 1000, ignore=0, edit=edit)
    c.solve()
    loss, lse = c.forward()
    within(loss, c.loss, c.e_loss)
    # where the target is the largest logit the loss is a logarithm near 1 alone
    assert ((loss.to(D) - c.loss).abs()[c.loss < 1e-3] <= 2e-3 * c.e_z.amax() + 300 * U32).all()
    dx, dw, b_dx, b_dw = c.gradients(U16, U16)
    got_dx, got_dw = c.backward(lse)
    within(got_dx, dx, b_dx * (1 + U16) + U16 * dx.abs() + 1e-37)
    within(got_dw, dw, b_dw + 2 * U32 * dw.abs() + 1e-37)


def test_a_row_of_nan_stays_its_own():
    good = Case(150, 136, 700, seed=3)
    bad = Case(150, 136, 700, seed=3, edit=lambda c: c.x.__setitem__((77, 5), NAN))
    a, b = good.forward(), bad.forward()
    others = [i for i in range(150) if i != 77]
    for p, q in zip(a, b):
        assert torch.equal(p[others], q[others])
    assert b[1][77].isnan()
    p, q = good.backward(a[1], want_dw=False)[0], bad.backward(b[1], want_dw=False)[0]
    assert torch.equal(p[others], q[others])


def test_gradients_against_differences():
    """Along each gradient's own direction the weighted loss has to change by the
    gradient's norm."""
    c = Case(23, 136, 301, seed=6)
    _, lse = c.forward()
    dx, dw = c.backward(lse)
    weight = torch.where((c.targets >= 0) & (c.targets < c.vocab), c.dloss, torch.zeros_like(c.dloss)).to(D)
    t = c.targets.long().clamp(0, c.vocab - 1)

    def value(x, w):
        z = torch.mm(x, w.t().contiguous())
        return (weight * (torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0])).sum()

    x, w, step = c.x.to(D), c.w.to(D), 1e-5
    for name, at, grad, f in (("dx", x, dx.to(D), lambda v: value(v, w)), ("dw", w, dw.to(D), lambda v: value(x, v))):
        masks = [torch.ones_like(grad)]
        for axis in (0, 1):
            for i in (0, grad.shape[axis] // 2, grad.shape[axis] - 1):
                mask = torch.zeros_like(grad)
                mask.select(axis, i).fill_(1)
                masks.append(mask)
        for mask in masks:
            v = grad * mask
            n = v.norm()
            if n == 0:
                continue   # (an ignored row)
            v = v / n
            slope = (f(at + step * v) - f(at - step * v)) / (2 * step)
            # (dx is rounded to bf16, and so is d)
            assert abs(slope - n) <= 2 * U16 * n + 1e-6, name


def test_no_tokens():
    dw = torch.full((11, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.linear_xent(None, 64, None, 64, 0, 64, 10, None, 1.0, None, None, None, 0)
    qg.linear_xent_backward(None, 64, None, 64, 0, 64, 10, None, 1.0, None, None, None, 64, dw, qg.O_BF16, 72, None, 0)
    assert (dw[:10, :64] == 0).all() and (dw[10:] == 7).all() and (dw[:, 64:] == 7).all()


@pytest.mark.parametrize("m,k,vocab", [(9, 264, 1000), (200, 520, 3001)])
def test_two_graphs_share_a_workspace(m, k, vocab):
    """Two captured steps on one stream, replayed in turn with eager work and waits between."""
    side = torch.cuda.Stream()
    cases = [Case(m, k, vocab, seed=1), Case(m + 3, k, vocab - 5, seed=2)]
    nbytes = max(max(c.fwd_bytes, c.bwd_bytes) for c in cases)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    outs, want, graphs = [], [], []

    def step(c, o):
        qg.linear_xent(c.xd, c.k + 8, c.wd, c.k + 16, c.m, c.k, c.vocab, c.targets, 1.0, o[0], o[1], ws, nbytes)
        qg.linear_xent_backward(c.xd, c.k + 8, c.wd, c.k + 16, c.m, c.k, c.vocab, c.targets, 1.0, o[1], c.dloss, o[2], c.k, o[3],
                                qg.O_F32, c.k, ws, nbytes)

    for c in cases:
        outs.append([torch.zeros(c.m, device="cuda"), torch.zeros(c.m, device="cuda"),
                     torch.zeros(c.m, c.k, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.vocab, c.k, device="cuda")])
        step(c, outs[-1])
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[-1]])
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            step(c, o)
        graphs.append(g)
    for i in range(3):
        for g, o, w in zip(graphs, outs, want):
            for t in o:
                t.fill_(5)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(o, w)), i
    step(cases[0], outs[0])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], want[0]))


def test_a_workspace_for_more_tokens():
    """One buffer, allocated for the largest batch, for smaller ones, which split otherwise."""
    largest, k, vocab = 300, 520, 3001
    n_f, n_b = qg.linear_xent_workspace_size(largest, k, vocab), qg.linear_xent_backward_workspace_size(largest, k, vocab)
    ws = torch.zeros(max(n_f, n_b) + 256, dtype=torch.uint8, device="cuda")
    ws[max(n_f, n_b):] = 7
    for m in (1, 20, 60, 129, 256, 299):
        c = Case(m, k, vocab, seed=m)
        c.solve()
        c.ws, c.fwd_bytes, c.bwd_bytes = ws, n_f, n_b
        loss, lse = c.forward()
        within(lse, c.lse, c.e_lse)
        within(loss, c.loss, c.e_loss)
        few = 2.0 ** -16
        dx, dw, b_dx, b_dw = c.gradients(few if m <= 16 else U16, few if m <= 32 else U16)
        got_dx, got_dw = c.backward(lse)
        within(got_dx, dx, b_dx * (1 + U16) + U16 * dx.abs() + 1e-37)
        within(got_dw, dw, b_dw + 2 * U32 * dw.abs() + 1e-37)
        assert (ws[max(n_f, n_b):] == 7).all()


MORE_TILES = [(3589, 1280, 1574)]   # dw in parts of two stages


@pytest.mark.parametrize("m,k,vocab", MORE_TILES)
def test_more_tile_shapes(m, k, vocab):
    test_forward_and_backward(m, k, vocab)


@pytest.mark.parametrize("m,vocab", [(5, 300), (150, 700), (700, 3001)])
def test_infinite_logits(m, vocab):
    """-inf: a token of probability 0.  +inf, or nothing but -inf: NaN losses, in those rows alone."""
    big, k = 2.0 ** 100, 72

    def edit(c):
        c.w[:, :2] = (torch.randn(vocab, 2, device="cuda") / big).to(torch.bfloat16)
        c.w[5, 0], c.w[9, 1], c.w[:, 2] = -big, big, -big
        c.x[:, :3] = 0
        c.x[:5] = 0
        c.x[0, 0] = c.x[1, 0] = c.x[2, 1] = c.x[3, 2] = big   # one of -inf, the same, one of +inf, all of -inf
        c.x[4, 3] = 1
        c.targets[:5] = torch.tensor([7, 5, 7, 7, 7], dtype=torch.int32)

    c = Case(m, k, vocab, seed=m, edit=edit)
    c.solve()
    loss, lse = c.forward()
    ordinary = torch.arange(m, device="cuda") > 3
    ordinary[0] = True
    z = c.z.clone()
    z[:2, 5] = -float("inf")
    e_z = c.e_z.clone()
    e_z[:2, 5] = 0
    for row in (0, 1):
        want = torch.logsumexp(z[row], 0)
        e = e_z[row].max() + (200 + vocab / 2048 + 40) * U32 + 2 * U32 * want.abs()
        assert abs(lse[row].item() - want) <= e
    assert abs(loss[0].item() - (torch.logsumexp(z[0], 0) - z[0, 7])) <= 2 * e_z[0].max() + 300 * U32 + 8 * U32 * z[0].abs()[z[0] > -1e30].max()
    assert loss[1] == float("inf")
    assert loss[2].isnan() and lse[2].isnan() and loss[3].isnan() and lse[3] == -float("inf")
    rest = ordinary.clone()
    rest[0] = False
    within(lse[rest], c.lse[rest], c.e_lse[rest])
    within(loss[rest], c.loss[rest], c.e_loss[rest])
    # gradients without the rows of NaN: d is that of the other tokens
    c.targets[2], c.targets[3] = -1, -1
    dx, dw = c.backward(lse)
    p = torch.exp(z[:2] - torch.logsumexp(z[:2], 1, keepdim=True))
    p[0, 7] -= 1
    p[1, 5] -= 1
    d = c.dloss[:2, None].to(D) * p
    want = torch.mm(d, c.w.to(D))[:, 4:]
    bound = (2 * U16) * torch.mm(d.abs() + 1e-6, c.w.to(D).abs())[:, 4:]
    within(dx[:2, 4:], want, bound + U16 * want.abs())
    assert (dx[2:4] == 0).all() and dx[rest.nonzero()[:, 0], 4:].isfinite().all() and dw[:, 4:].isfinite().all()
    # the target of the second row, whose logit is -inf, has the whole of its gradient (the first column: rows 0 and 1 alone)
    assert abs(dw[5, 0].item() / big + c.dloss[1].item()) <= 2 * U16 * c.dloss[1].item()
