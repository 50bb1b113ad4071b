"""GPU tests of the norm, the adapters and the head's cross entropy on matrices of more
than 4 GiB: what lies behind 32-bit offsets."""
import pytest
import torch

import quantized_gemm_qg_amd as qg
import test_gpu_xent
from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu
D, U32, U16 = torch.float64, 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def test_cross_entropy_of_a_large_head():
    """Weights and their gradient of 4.4 and 8.8 GB."""
    test_gpu_xent.test_forward_and_backward(40, 8192, 270000)


def test_norm_of_many_rows():
    """Both directions: the same bits as from calls of a part of the rows each."""
    rows, k, part = 530000, 4096, 60000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, res, dy = ((torch.randn(rows, k, generator=gen, device="cuda", dtype=BF)) for _ in range(3))
    w = (1 + 0.3 * torch.randn(k, generator=gen, device="cuda")).to(BF)
    outs = []
    for step in (rows, part):
        s, y, dx, q = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x, dtype=torch.uint8)
        qs = torch.zeros(rows, k // 32, dtype=torch.uint8, device="cuda")
        for r in range(0, rows, step):
            n = min(step, rows - r)
            qg.rmsnorm(x[r:], qg.O_BF16, k, w, 1e-5, n, k, residual=res[r:], ldr=k, sum=s[r:], lds=k, y=y[r:], ldy=k, q_type=qg.A_MXFP8,
                       q=q[r:], ldq=k, q_scales=qs[r:])
            qg.rmsnorm_backward(s[r:], qg.O_BF16, k, w, 1e-5, n, k, dy[r:], k, dx[r:], k, None, qg.O_F32, dsum=res[r:], ldds=k)
        outs.append((s, y, dx, q, qs))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert all(t[-1].any() for t in outs[0])


def adapters_call(m, k, n, rank, adapters, ids, x, a, b, y):
    order, offsets = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty(adapters + 1, dtype=torch.int32, device="cuda")
    sort_ws = torch.zeros(8192, dtype=torch.uint8, device="cuda")
    qg.moe_sort(ids, m, 1, adapters, order, offsets, sort_ws, sort_ws.numel())
    nbytes = qg.lora_workspace_size(m, k, n, adapters, rank)
    ws = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    qg.lora(x, k, a, k, b, rank, None, adapters, rank, order, offsets, m, k, n, y, qg.O_BF16, y.stride(0), ws, nbytes)
    torch.cuda.synchronize()


def adapters_check(rows, ids, x, a, b, before, y):
    """As in the adapters' own tests: fp32 sums, two bf16 parts of the low-rank row, one rounding."""
    k, rank = x.shape[1], a.shape[1]
    for r in rows:
        i = int(ids[r])
        t, mag = torch.mv(a[i].to(D), x[r].to(D)), torch.mv(a[i].to(D).abs(), x[r].to(D).abs())
        e_t = mag * (2 * k + 2) * U32 + 2.0 ** -16 * t.abs()
        bi = b[i].to(D)
        want = before[r].to(D) + torch.mv(bi, t)
        bound = torch.mv(bi.abs(), e_t + (t.abs() + e_t) * (6 * rank + 8) * U32)
        bound = bound + (U16 + U32) * (want.abs() + bound) + 1e-37
        assert ((y[r].to(D) - want).abs() <= bound).all(), r


def test_adapters_of_a_large_output():
    m, k, n, rank, adapters = 40000, 64, 57344, 8, 3   # 4.6 GB
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x, a, b, y = rand(m, k), rand(adapters, rank, k), rand(adapters, n, rank), rand(m, n)
    before = y.clone()
    ids = torch.randint(-1, adapters, (m,), generator=gen, device="cuda").to(torch.int32)
    ids[0], ids[-1] = 1, 2
    adapters_call(m, k, n, rank, adapters, ids, x, a, b, y)
    none = ids < 0
    assert torch.equal(y[none], before[none])
    # (row 37449 begins behind 4 GiB)
    for r in (0, 37448, 37449, 37450, m - 1):
        if ids[r] < 0:
            continue
        adapters_check([r], ids, x, a, b, before, y)
    changed = (y != before).any(1)
    assert torch.equal(changed, ~none)


def test_adapters_of_many_large_matrices():
    m, k, n, rank, adapters = 1200, 9000, 9000, 256, 1024   # A and B of 4.7 GB each
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x, a, b, y = rand(m, k), rand(adapters, rank, k), rand(adapters, n, rank), rand(m, n)
    before = y.clone()
    ids = torch.randint(adapters, (m,), generator=gen, device="cuda").to(torch.int32)
    ids[0], ids[1], ids[2] = adapters - 1, 0, 933   # (the last one's B begins behind 4 GiB, as its A)
    adapters_call(m, k, n, rank, adapters, ids, x, a, b, y)
    adapters_check(list(range(40)) + [m - 1], ids, x, a, b, before, y)
