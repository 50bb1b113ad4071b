"""GPU tests of the low-rank adapters against the formula in 64 bits.

Tolerances: fp32 sums of K products are within K 2^-23 of the sum of the products'
magnitudes; the low-rank row goes on in two bf16 parts (2^-16 of it is left) or
three (2^-23); y is rounded once."""
import pytest
import torch

import lora_sizes
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
    """Longer pitch of the last dimension, NaN behind the values."""
    d = torch.full((*t.shape[:-1], t.shape[-1] + extra), NAN, dtype=t.dtype, device="cuda")
    d[..., :t.shape[-1]] = t.cuda()
    return d


class Case:
    def __init__(self, m, k, n, rank, adapters, y_type=qg.O_BF16, seed=0, prompts=False, none=0.15, scales=True, pad=8, shift=0,
                 ids=None, edit=None):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.m, self.k, self.n, self.rank, self.adapters, self.y_type = m, k, n, rank, adapters, y_type
        self.x = rand(m, k).to(torch.bfloat16)
        self.a = (rand(adapters, rank, k) / k ** 0.5).to(torch.bfloat16)
        self.b = rand(adapters, n, rank).to(torch.bfloat16)
        self.scales = (0.2 + torch.rand(adapters, generator=gen)) if scales else None
        if ids is None:
            if prompts:
                cuts = torch.randint(m + 1, (adapters + 2,), generator=gen).sort().values
                owner = torch.randint(-1, adapters, (adapters + 3,), generator=gen)
                ids = owner[torch.searchsorted(cuts, torch.arange(m), right=True)]
            else:
                ids = torch.randint(adapters, (m,), generator=gen)
                ids[torch.rand(m, generator=gen) < none] = -1
        self.ids = ids.to(torch.int32)
        t = torch.float32 if y_type == qg.O_F32 else torch.bfloat16
        self.y = rand(m, n).to(t)
        if edit:
            edit(self)
        # the outputs' memory: `shift` elements in, so that rows are not on 16 bytes
        self.ldy = n + pad
        self.flat = torch.full((m * self.ldy + shift + 64,), 7.0, dtype=t, device="cuda")
        self.shift = shift
        self.yd = self.flat[shift:shift + m * self.ldy].view(m, self.ldy)
        self.yd[:, :n] = self.y.cuda()
        self.before = self.flat.clone()
        self.xd, self.ad, self.bd = padded(self.x, 8), padded(self.a, 16), padded(self.b, 8)
        self.sd = None if self.scales is None else self.scales.cuda()
        self.sorted = torch.full((max(m, 1),), -7, dtype=torch.int32, device="cuda")
        self.offsets = torch.zeros(adapters + 1, dtype=torch.int32, device="cuda")
        sort_ws = torch.zeros(-(-4 * (adapters + 1) // 256) * 256, dtype=torch.uint8, device="cuda")
        qg.moe_sort(self.ids.cuda(), m, 1, adapters, self.sorted, self.offsets, sort_ws, sort_ws.numel())
        self.ws_bytes = qg.lora_workspace_size(m, k, n, adapters, rank)
        self.ws = torch.full((max(self.ws_bytes, 1),), 255, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        qg.lora(self.xd, self.k + 8, self.ad, self.k + 16, self.bd, self.rank + 8, self.sd, self.adapters, self.rank, self.sorted,
                self.offsets, self.m, self.k, self.n, self.yd, self.y_type, self.ldy, self.ws, self.ws_bytes, stream=stream)

    def run(self):
        self.call()
        torch.cuda.synchronize()
        assert (self.flat[:self.shift] == 7).all() and (self.flat[self.shift + self.m * self.ldy:] == 7).all()
        assert (self.yd[:, self.n:] == 7).all()
        assert (self.ws[:1 << 16] == 255).all()   # where a product's workspace has its counters
        return self.yd[:, :self.n].cpu()

    def check(self, got):
        u, part = (U32, 2.0 ** -23) if self.y_type == qg.O_F32 else (U16, 2.0 ** -16)
        for i in range(-1, self.adapters):
            at = (self.ids == i).nonzero()[:, 0]
            if not len(at):
                continue
            if i < 0:
                assert torch.equal(got[at], self.y[at])   # no adapter: no change
                continue
            x, a, b = self.x[at].to(D), self.a[i].to(D), self.b[i].to(D)
            s = 1.0 if self.scales is None else self.scales[i].item()
            t, mag = s * x @ a.T, s * x.abs() @ a.abs().T
            e_t = mag * (2 * self.k + 2) * U32 + part * t.abs()
            want = self.y[at].to(D) + t @ b.T
            bound = (e_t + (t.abs() + e_t) * (6 * self.rank + 8) * U32) @ b.abs().T
            bound = bound + (u + U32) * (want.abs() + bound) + 1e-37
            off = (got[at].to(D) - want).abs() - bound
            assert (off <= 0).all(), f"adapter {i}: {off.max().item():.3g} over the bound"


SIZES = [  # m, k, n, rank, adapters
    (1, 8, 1, 8, 1), (1, 4096, 300, 16, 8), (2, 264, 17, 24, 3), (7, 1032, 1000, 8, 4), (16, 512, 256, 32, 1), (17, 72, 65, 40, 2),
    (33, 2056, 515, 16, 40), (64, 1024, 640, 64, 48), (40, 136, 100, 128, 5), (50, 520, 77, 200, 6), (65, 264, 130, 256, 2),
    (100, 264, 257, 16, 1), (129, 1032, 300, 8, 3), (333, 520, 509, 24, 5), (300, 136, 260, 48, 2), (257, 72, 64, 72, 4),
    (500, 264, 192, 136, 3), (1100, 40, 70, 16, 7), (200, 72, 40, 16, 1000), (1030, 264, 90, 256, 16)]


@pytest.mark.parametrize("m,k,n,rank,adapters", SIZES)
@pytest.mark.parametrize("y_type", [qg.O_BF16, qg.O_F32])
def test_lora(m, k, n, rank, adapters, y_type):
    for prompts, pad, shift in ((False, 8 - n % 8, 0), (True, 3, 0), (False, 8, 1)):
        print(f"lora m={m} k={k} n={n} rank={rank} adapters={adapters} y={y_type} prompts={prompts} pad={pad} shift={shift}", flush=True)
        c = Case(m, k, n, rank, adapters, y_type, seed=m + n, prompts=prompts, pad=pad, shift=shift, scales=not prompts)
        c.check(c.run())


@pytest.mark.parametrize("m", [1, 20, 300])
def test_no_row_has_an_adapter(m):
    c = Case(m, 136, 100, 16, 3, ids=torch.full((m,), -1))
    got = c.run()
    assert torch.equal(got, c.y)


def test_one_adapter_of_many_has_all_rows():
    c = Case(150, 264, 300, 16, 900, ids=torch.full((150,), 899))
    c.check(c.run())
    c = Case(150, 264, 300, 16, 2, ids=torch.zeros(150))
    c.check(c.run())


def test_rows_do_not_touch_each_other():
    """NaN and infinities in a row of x, in an adapter that is not the row's, behind the rank."""
    for m, adapters in ((40, 6), (300, 3)):
        good = Case(m, 264, 260, 24, adapters, seed=5)
        victim = (good.ids == 1).nonzero()[0, 0].item()

        def edit(c):
            c.x[victim] = NAN
            c.a[0] = float("inf")
            c.b[0] = NAN

        bad = Case(m, 264, 260, 24, adapters, seed=5, edit=edit)
        a, b = good.run(), bad.run()
        same = (good.ids != 0)
        same[victim] = False
        assert torch.equal(a[same], b[same]) and b[victim].isnan().all()


def test_entries_that_name_no_row_are_skipped():
    for m, adapters in ((30, 4), (200, 2)):
        c = Case(m, 264, 100, 16, adapters, none=0.0)
        lost = [3, m // 2, m - 1]
        rows = c.sorted[lost].cpu().long()
        c.sorted[torch.tensor(lost, device="cuda")] = torch.tensor([-1, m, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        got = c.run()
        assert torch.equal(got[rows], c.y[rows])
        c.ids[rows] = -1
        c.check(got)


def test_columns_of_a_fused_projection():
    """Two adapters' calls on column ranges of one output."""
    m, k, n = 50, 264, 320
    c = Case(m, k, n, 16, 4, seed=9)
    half = Case(m, k, 128, 16, 4, seed=9, ids=c.ids)
    qg.lora(half.xd, k + 8, half.ad, k + 16, half.bd, 24, half.sd, 4, 16, c.sorted, c.offsets, m, k, 128, c.yd[:, 64:].data_ptr(),
            qg.O_BF16, c.ldy, c.ws, c.ws_bytes)
    torch.cuda.synchronize()
    got = c.yd[:, :n].cpu()
    assert torch.equal(got[:, :64], c.y[:, :64]) and torch.equal(got[:, 192:], c.y[:, 192:])
    half.y = c.y[:, 64:192]
    half.check(got[:, 64:192])


def test_no_rows():
    qg.lora(None, 64, None, 64, None, 16, None, 2, 16, None, None, 0, 64, 100, None, qg.O_BF16, 100, None, 0)
    assert qg.lora_workspace_size(0, 64, 100, 2, 16) == 0


def test_another_stream_and_a_captured_graph():
    """The sort and two projections of a batch, replayed with other adapters each time."""
    c = Case(70, 264, 300, 16, 5, seed=4)
    ids = c.ids.cuda()
    sort_ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        qg.moe_sort(ids, c.m, 1, c.adapters, c.sorted, c.offsets, sort_ws, 256)
        c.call()

    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    c.check(c.yd[:, :c.n].cpu())
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        other = (c.ids + i).remainder(c.adapters + 1) - 1
        c.flat.copy_(c.before)
        ids.copy_(other)
        c.ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept, c.ids = c.ids, other
        c.check(c.yd[:, :c.n].cpu())
        c.ids = kept


def test_a_workspace_for_more_rows():
    """One buffer, allocated for the largest batch, for batches that split k into more parts."""
    largest, k, n, rank = 2048, 4096, 264, 16
    size = qg.lora_workspace_size(largest, k, n, 1, rank)
    for m in (700, 1023, 2047):
        c = Case(m, k, n, rank, 1, seed=m)
        c.ws_bytes = size
        c.ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
        c.check(c.run())
        assert (c.ws[size:] == 255).all()


@pytest.mark.parametrize("m,k,n,rank,adapters", lora_sizes.EVERY_KERNEL)
@pytest.mark.parametrize("y_type", [qg.O_BF16, qg.O_F32])
def test_every_kernel(m, k, n, rank, adapters, y_type):
    prompts, shift = adapters > 8 and m > 500, n % 3 % 2   # (rows of every adapter side by side anyway; y on and off 16 bytes)
    print(f"lora m={m} k={k} n={n} rank={rank} adapters={adapters} y={y_type} prompts={prompts} shift={shift}: "
          f"{qg.describe_lora(m, k, n, adapters, rank, y_type)}", flush=True)
    c = Case(m, k, n, rank, adapters, y_type, seed=m + n, prompts=prompts, pad=8 - n % 8, shift=shift, none=0.0 if m < 10 else 0.15)
    c.call()
    torch.cuda.synchronize()
    assert (c.flat[:shift] == 7).all() and (c.flat[shift + m * c.ldy:] == 7).all() and (c.yd[:, n:] == 7).all()
    # as Case.check, on the GPU
    u, part = (U32, 2.0 ** -23) if y_type == qg.O_F32 else (U16, 2.0 ** -16)
    got, before = c.yd[:, :n], c.before[shift:shift + m * c.ldy].view(m, c.ldy)[:, :n]
    x, a, b, ids = c.x.cuda(), c.a.cuda(), c.b.cuda(), c.ids.cuda()
    assert torch.equal(got[ids < 0], before[ids < 0])
    for i in c.ids.unique().tolist():
        if i < 0:
            continue
        at = (ids == i).nonzero()[:, 0]
        xi, ai, bt = x[at].to(D), a[i].to(D).t().contiguous(), b[i].to(D).t().contiguous()
        s = c.scales[i].item()
        t, mag = s * torch.mm(xi, ai), s * torch.mm(xi.abs(), ai.abs())
        e_t = mag * (2 * k + 2) * U32 + part * t.abs()
        want = before[at].to(D) + torch.mm(t, bt)
        bound = torch.mm(e_t + (t.abs() + e_t) * (6 * rank + 8) * U32, bt.abs())
        bound = bound + (u + U32) * (want.abs() + bound) + 1e-37
        off = (got[at].to(D) - want).abs() - bound
        assert (off <= 0).all(), f"adapter {i}: {off.max().item():.3g} over the bound"
    assert c.ids.max() >= 0
