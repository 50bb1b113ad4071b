"""GPU tests of the bf16 gated feed-forward block, forward and backward,
against the formulas in 64 bits and, for the gradients, against differences.

Tolerances: fp32 sums of K products are within K 2^-23 of the sum of the
products' magnitudes (one rounding per product and one per addition), outputs
and the gradient of the pre-activations are rounded once to bf16 (2^-8)."""
import math

import pytest
import torch

import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu
from gradient_check import check_block_gradients

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
D = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def act64(g, act):
    """act(g), act'(g)"""
    if act == qg.ACT_SILU:
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


class Case:
    def __init__(self, m, k, inter, act, seed=0, pad=8):
        gen = torch.Generator().manual_seed(seed)
        bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
        self.m, self.k, self.inter, self.act = m, k, inter, act
        self.x, self.dh = bf(m, k), bf(m, inter)
        self.w = (torch.randn(2 * inter, k, generator=gen) * (1.5 / math.sqrt(k))).to(torch.bfloat16)
        self.ldx = self.ldw = k + pad
        self.lddh = inter + 3
        self.xd = self._pad(self.x, self.ldx)
        self.wd = self._pad(self.w, self.ldw)
        self.dhd = self._pad(self.dh, self.lddh)
        x, w = self.x.to(D), self.w.to(D)
        gu = x @ w.T
        self.e_gu = k * 2 * U32 * (x.abs() @ w.abs().T)   # bound on the error of the fp32 sums
        self.g, self.u = gu[:, :inter], gu[:, inter:]
        self.a, self.da = act64(self.g, act)
        self.h = self.a * self.u
        dh = self.dh.to(D)
        self.dgu = torch.cat((dh * self.u * self.da, dh * self.a), 1)
        self.dx, self.dw = self.dgu @ w, self.dgu.T @ x

    @staticmethod
    def _pad(t, ld):
        """Rows with a longer pitch, NaN behind them."""
        d = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
        d[:, :t.shape[1]] = t.cuda()
        return d

    def e_h(self):
        eg, eu = self.e_gu[:, :self.inter], self.e_gu[:, self.inter:]
        # |act'| <= 1.13, |act''| <= 0.8, |act(g)| <= |g|; the activation itself in fp32
        act = 2.0 ** -20 * (1 + self.g.abs())
        return 1.13 * eg * (self.u.abs() + eu) + self.a.abs() * eu + act * self.u.abs()

    def e_dgu(self):
        eg, eu = self.e_gu[:, :self.inter], self.e_gu[:, self.inter:]
        dh, act = self.dh.to(D).abs(), 2.0 ** -20 * (1 + self.g.abs())
        e_dg = dh * (0.8 * eg * (self.u.abs() + eu) + 1.13 * eu + act * self.u.abs())
        e_du = dh * (1.13 * eg + act)
        return torch.cat((e_dg, e_du), 1) + U16 * self.dgu.abs()

    def forward(self, gu_type=None):
        m, i = self.m, self.inter
        ldh = i + 5
        h = torch.full((m + 1, ldh), 7.0, dtype=torch.bfloat16, device="cuda")
        gu, ldgu = None, 0
        if gu_type is not None:
            ldgu = 2 * i + 3
            gu = torch.full((m + 1, ldgu), 7.0, dtype=torch.float32 if gu_type == qg.O_F32 else torch.bfloat16, device="cuda")
        wsb = qg.ffn_gated_workspace_size(m, self.k, i)
        self.fws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        for _ in range(2):
            qg.ffn_gated(self.xd, self.ldx, self.wd, self.ldw, m, self.k, i, self.act, h, ldh, self.fws, wsb, gu=gu,
                         gu_type=gu_type or 0, ldgu=ldgu)
        assert (h[m:] == 7).all() and (h[:m, i:] == 7).all()
        if gu is not None:
            assert (gu[m:] == 7).all() and (gu[:m, 2 * i:] == 7).all()
        return h[:m, :i].cpu().to(D), gu, ldgu

    def backward(self, gu=None, gu_type=0, ldgu=0, want_dx=True, dw_type=qg.O_F32, want_dw=True):
        m, k, i = self.m, self.k, self.inter
        dx = torch.full((m + 1, k + 8), 7.0, dtype=torch.bfloat16, device="cuda") if want_dx else None
        dwt = torch.float32 if dw_type == qg.O_F32 else torch.bfloat16
        dw = torch.full((2 * i + 1, k + 4), 7.0, dtype=dwt, device="cuda") if want_dw else None
        wsb = qg.ffn_gated_backward_workspace_size(m, k, i, recompute=gu is None)
        ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        for _ in range(2):
            qg.ffn_gated_backward(self.xd, self.ldx, self.wd, self.ldw, self.dhd, self.lddh, m, k, i, self.act, dx, k + 8, dw,
                                  dw_type, k + 4, ws, wsb, gu=gu, gu_type=gu_type, ldgu=ldgu)
        if want_dx:
            assert (dx[m:] == 7).all() and (dx[:m, k:] == 7).all()
            dx = dx[:m, :k].cpu().to(D)
        if want_dw:
            assert (dw[2 * i:] == 7).all() and (dw[:2 * i, k:] == 7).all()
            dw = dw[:2 * i, :k].cpu().to(D)
        return dx, dw


def within(got, ref, bound):
    off = (got - ref).abs() - bound
    assert (off <= 0).all(), f"{off.max().item():.3g} over the bound"


FORWARD = [(1, 8, 1), (1, 4096, 300), (1, 1032, 2048), (2, 264, 17), (5, 512, 130), (16, 2048, 96), (17, 72, 33), (40, 1000, 64),
           (64, 256, 200), (100, 136, 257), (128, 64, 128), (257, 1032, 281), (600, 40, 90), (1100, 128, 70)]


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
@pytest.mark.parametrize("m,k,inter", FORWARD)
def test_forward(m, k, inter, act):
    print(f"ffn forward m={m} k={k} inter={inter} act={act}", flush=True)
    c = Case(m, k, inter, act, seed=m + k)
    h, _, _ = c.forward()
    within(h, c.h, c.e_h() * (1 + U16) + U16 * c.h.abs() + 1e-37)
    for t, u in ((qg.O_F32, 0.0), (qg.O_BF16, U16)):
        h2, gu, _ = c.forward(t)
        assert torch.equal(h, h2)
        ref = torch.cat((c.g, c.u), 1)
        within(gu[:m, :2 * inter].cpu().to(D), ref, c.e_gu * (1 + u) + u * ref.abs() + 1e-37)


BACKWARD = [(1, 8, 1), (1, 512, 100), (3, 264, 17), (16, 128, 64), (31, 1000, 130), (65, 72, 33), (128, 256, 192), (257, 1032, 281),
            (600, 40, 90), (1100, 128, 70)]


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
@pytest.mark.parametrize("m,k,inter", BACKWARD)
def test_backward(m, k, inter, act):
    print(f"ffn backward m={m} k={k} inter={inter} act={act}", flush=True)
    c = Case(m, k, inter, act, seed=m * 3 + k)
    e = c.e_dgu()
    x, w = c.x.to(D).abs(), c.w.to(D).abs()
    grown = c.dgu.abs() + e
    b_dx = e @ w + 2 * inter * 2 * U32 * (grown @ w)
    b_dw = e.T @ x + m * 2 * U32 * (grown.T @ x)
    _, gu, ldgu = c.forward(qg.O_F32)
    for saved in (dict(gu=gu, gu_type=qg.O_F32, ldgu=ldgu), {}):
        dx, dw = c.backward(**saved)
        within(dx, c.dx, b_dx * (1 + U16) + U16 * c.dx.abs() + 1e-37)
        within(dw, c.dw, b_dw + 1e-37)
        # the roundings of the pre-activations' gradient are independent: far nearer in the 2-norm
        if c.dgu.numel() > 1000:
            assert (dw - c.dw).norm() <= U16 * c.dw.norm()
            assert (dx - c.dx).norm() <= 2 * U16 * c.dx.norm()
    only_dx, none = c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu, want_dw=False)
    none2, dw16 = c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu, want_dx=False, dw_type=qg.O_BF16)
    assert none is None and none2 is None
    again, dw = c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu)
    assert torch.equal(only_dx, again)
    assert torch.equal(dw16, dw.to(torch.bfloat16).to(D))


# every tile shape of the three products, whole and in parts of k
TILES = [(36, 32, 8848), (85, 32, 9950), (394, 32, 13727), (399, 32, 4700), (429, 608, 4836), (77, 4160, 1916), (620, 2496, 803),
         (1345, 2016, 71), (1345, 2976, 100), (403, 8320, 64), (173, 5632, 65)]


@pytest.mark.parametrize("m,k,inter", TILES)
def test_every_tile_shape(m, k, inter):
    test_forward(m, k, inter, qg.ACT_SILU)
    test_backward(m, k, inter, qg.ACT_GELU_TANH)


@pytest.mark.parametrize("m,k,inter", [(1, 312, 200), (1, 4096, 70), (2, 72, 33), (15, 264, 517), (16, 128, 1000), (17, 312, 200),
                                       (31, 136, 45), (32, 1032, 300)])
def test_few_tokens_keep_the_gradient_of_the_pre_activations_in_two_parts(m, k, inter):
    """One bf16 rounding would put 1.7e-3 on dW and dx; two parts leave 2^-17 of
    each element, far below what rounding dx to bf16 costs."""
    c = Case(m, k, inter, qg.ACT_SILU, seed=m + inter)
    _, gu, ldgu = c.forward(qg.O_F32)
    dx, dw = c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu)
    assert (dw - c.dw).norm() <= 2.0 ** -15 * c.dw.norm()
    if m <= 16:
        rounded = c.dx.to(torch.bfloat16).to(D)
        assert (dx - c.dx).norm() <= 1.1 * (rounded - c.dx).norm() + 2.0 ** -15 * c.dx.norm()


def test_backward_from_pre_activations_saved_in_bf16():
    c = Case(130, 256, 96, qg.ACT_SILU, seed=5)
    _, gu, ldgu = c.forward(qg.O_BF16)
    dx, dw = c.backward(gu=gu, gu_type=qg.O_BF16, ldgu=ldgu)
    # g and u each off by 2^-8 of themselves, then the gradient's own rounding
    assert (dx - c.dx).norm() <= 5 * U16 * c.dx.norm()
    assert (dw - c.dw).norm() <= 5 * U16 * c.dw.norm()


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
def test_gradient_against_differences(act):
    c = Case(70, 136, 45, act, seed=11)
    dx, dw = c.backward()
    gen = torch.Generator().manual_seed(1)

    def loss(x, w):
        gu = x @ w.T
        return (c.dh.to(D) * act64(gu[:, :c.inter], act)[0] * gu[:, c.inter:]).sum()

    x, w = c.x.to(D), c.w.to(D)
    for _ in range(4):
        vx, vw = torch.randn(x.shape, generator=gen, dtype=D), torch.randn(w.shape, generator=gen, dtype=D)
        eps = 1e-5
        slope = (loss(x + eps * vx, w + eps * vw) - loss(x - eps * vx, w - eps * vw)) / (2 * eps)
        got = (dx * vx).sum() + (dw * vw).sum()
        # both gradients are within 2^-7 of their norm, the direction is random
        assert abs(got - slope) <= 2 * U16 * (dx.norm() * vx.norm() + dw.norm() * vw.norm())


def test_inf_and_nan_stay_in_their_rows_and_columns():
    c = Case(40, 72, 33, qg.ACT_SILU, seed=2)   # k ends inside a stage of the ring
    c.xd[7, 71] = float("nan")
    c.xd[9, 0] = float("inf")
    h, _, _ = c.forward()
    bad = ~torch.isfinite(h)
    assert bad[7].all() and bad[9].any()
    bad[7] = bad[9] = False
    assert not bad.any()
    clean = [r for r in range(40) if r not in (7, 9)]
    within(h[clean], c.h[clean], (c.e_h() * (1 + U16) + U16 * c.h.abs())[clean] + 1e-37)


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
def test_activation_and_derivative_over_their_whole_range(act):
    """One token with x = (1, 1, 0 ..): g is the weights' first column and u = 1,
    so dW's first column is act'(g) and its second act(g).  Tails and
    overflowing squares included."""
    vals = [0.0, 1e-30, 1e-3, 0.3, 0.75, 1.0, 2.0, 5.0, 12.0, 30.0, 200.0, 1e5, 1e13, 1e20, 3e38]
    g = torch.tensor(vals + [-v for v in vals]).to(torch.bfloat16)
    n, k = g.numel(), 32
    c = Case(1, k, n, act)
    c.xd[:] = 0
    c.xd[0, :2] = 1
    c.wd[:] = 0
    c.wd[:n, 0] = g.cuda()
    c.wd[n:, 1] = 1
    c.dhd[:] = 1
    h, gu, ldgu = c.forward(qg.O_F32)
    v, dv = act64(g.to(D), act)
    # the gate p in fp32 (its exponent off by 2^-22 of itself, 150 at most where p
    # is a normal number), then one rounding to bf16
    tol = U16 + 2.0 ** -14
    within(h[0], v, tol * v.abs() + 1e-36)
    _, dw = c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu)
    # act' = p + g p (1 - p) z': near its zero the two cancel
    within(dw[:n, 0], dv, tol * dv.abs() + 2.0 ** -20 + 1e-36)
    within(dw[n:, 1], v, tol * v.abs() + 1e-36)


def test_no_tokens():
    c = Case(1, 64, 16, qg.ACT_SILU)
    dw = torch.full((33, 64), 7.0, device="cuda")
    qg.ffn_gated(c.xd, c.ldx, c.wd, c.ldw, 0, 64, 16, qg.ACT_SILU, None, 16)
    qg.ffn_gated_backward(c.xd, c.ldx, c.wd, c.ldw, None, 16, 0, 64, 16, qg.ACT_SILU, None, 64, dw, qg.O_F32, 64, None, 0)
    assert (dw[:32] == 0).all() and (dw[32] == 7).all()


def test_graph_replays():
    for m in (1, 40):
        c = Case(m, 256, 64, qg.ACT_SILU, seed=m)
        h = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
        gu = torch.zeros(m, 128, device="cuda")
        dx = torch.zeros(m, 256, dtype=torch.bfloat16, device="cuda")
        dw = torch.zeros(128, 256, device="cuda")
        wsb = max(qg.ffn_gated_workspace_size(m, 256, 64), qg.ffn_gated_backward_workspace_size(m, 256, 64))
        ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")

        def run():
            qg.ffn_gated(c.xd, c.ldx, c.wd, c.ldw, m, 256, 64, c.act, h, 64, ws, wsb, gu=gu, gu_type=qg.O_F32, ldgu=128)
            qg.ffn_gated_backward(c.xd, c.ldx, c.wd, c.ldw, c.dhd, c.lddh, m, 256, 64, c.act, dx, 256, dw, qg.O_F32, 256, ws, wsb,
                                  gu=gu, gu_type=qg.O_F32, ldgu=128)

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for rep in range(3):
            c.dhd[:, :64] = torch.randn(m, 64, device="cuda").to(torch.bfloat16)
            run()
            eager = [t.clone() for t in (h, dx, dw)]
            for t in (h, gu, dx, dw):
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, (h, dx, dw)))


def test_dx_of_a_feed_forward_size_whose_rows_lie_megabytes_apart():
    """8.5 million inner columns: 128 rows of [dg du] are further apart than 32
    bits of bytes.  Only 64 columns and their weights are not zero, so the
    products' bound is that of 128 terms."""
    m, k, inter = 129, 264, 8500000
    gen = torch.Generator().manual_seed(3)
    at = torch.randint(inter, (64,), generator=gen).unique()
    at[0], at[-1] = 0, inter - 1
    n = at.numel()
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    g, u, dh, wg, wu = bf(m, n), bf(m, n), bf(m, n), bf(n, k), bf(n, k)
    gu = torch.zeros(m, 2 * inter, dtype=torch.bfloat16, device="cuda")
    dhd = torch.zeros(m, inter, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2 * inter, k, dtype=torch.bfloat16, device="cuda")
    cols = at.cuda()
    gu[:, cols], gu[:, inter + cols], dhd[:, cols] = g.cuda(), u.cuda(), dh.cuda()
    w[cols], w[inter + cols] = wg.cuda(), wu.cuda()
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((m, k), 7.0, dtype=torch.bfloat16, device="cuda")
    wsb = qg.ffn_gated_backward_workspace_size(m, k, inter)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    ws[:65536] = 0
    print(f"ffn dx m={m} k={k} inter={inter}, workspace {wsb} bytes", flush=True)
    qg.ffn_gated_backward(x, k, w, k, dhd, inter, m, k, inter, qg.ACT_SILU, dx, k, None, 0, 0, ws, wsb, gu=gu,
                          gu_type=qg.O_BF16, ldgu=2 * inter)
    got = dx.cpu().to(D)
    del gu, dhd, w, ws
    torch.cuda.empty_cache()
    g, u, dh = g.to(D), u.to(D), dh.to(D)
    a, da = act64(g, qg.ACT_SILU)
    dgu, both = torch.cat((dh * u * da, dh * a), 1), torch.cat((wg, wu)).to(D)
    act = 2.0 ** -20 * (1 + g.abs())
    e = torch.cat((dh.abs() * act * u.abs(), dh.abs() * act), 1) + U16 * dgu.abs()
    bound = e @ both.abs() + 2 * n * 2 * U32 * ((dgu.abs() + e) @ both.abs())
    ref = dgu @ both
    within(got, ref, bound * (1 + U16) + U16 * ref.abs() + 1e-37)


@pytest.mark.parametrize("m", [1, 20, 40])
@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
def test_backward_of_aligned_rows_gives_the_bits_of_unaligned_ones(m, act):
    """The elementwise pass takes four elements a thread where rows of dh (and
    of bf16 pre-activations) allow it, else one: the same results, of which the
    other tests compare the latter with 64 bits."""
    c = Case(m, 264, 100, act, seed=m)
    _, gu, ldgu = c.forward(qg.O_F32)
    i = c.inter
    narrow = torch.full((m, 2 * i + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide = torch.full((m, 2 * i + 4), float("nan"), dtype=torch.bfloat16, device="cuda")
    narrow[:, :2 * i] = wide[:, :2 * i] = gu[:m, :2 * i]
    one = [c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu), c.backward(gu=narrow, gu_type=qg.O_BF16, ldgu=2 * i + 3)]
    assert c.lddh % 4 != 0
    c.lddh = i + 4
    c.dhd = c._pad(c.dh, c.lddh)
    four = [c.backward(gu=gu, gu_type=qg.O_F32, ldgu=ldgu), c.backward(gu=wide, gu_type=qg.O_BF16, ldgu=2 * i + 4)]
    for (dx1, dw1), (dx4, dw4) in zip(one, four):
        assert torch.equal(dx1, dx4) and torch.equal(dw1, dw4)


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
@pytest.mark.parametrize("m", [9, 70])
def test_each_gradient_against_differences_along_itself(m, act):
    """The roundings of [dg du] and of the output take each at most 2^-8 of a
    part's norm."""
    c = Case(m, 136, 45, act, seed=11)
    dx, dw = c.backward()
    check_block_gradients(c.x.to(D), c.w.to(D), c.dh.to(D), act == qg.ACT_SILU, dx, dw, 2 * U16)
