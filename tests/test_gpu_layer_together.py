"""GPU tests of the norm, the adapters and the head's cross entropy as they are used
together: a training step's gradients against the formulas in 64 bits, and a served
step against the same model in 64 bits."""
import importlib.util
import os

import pytest
import torch

import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D, U16 = torch.float64, 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("train_adapt_serve", os.path.join(ROOT, "examples", "train_adapt_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(s, w, eps):
    return s * w / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)


def forward(ex, p, token):
    s = p["embed"][token]
    g, u = (norm(s, p["norm1"], ex.EPS) @ p["gate_up"].T).split(ex.INTER, 1)
    return s, norm(s + (g / (1 + torch.exp(-g)) * u) @ p["down"].T, p["norm2"], ex.EPS)


def test_gradients_of_a_training_step(example):
    ex = example
    p = ex.new_parameters()
    gen = torch.Generator(device="cuda").manual_seed(3)
    token = torch.randint(ex.VOCAB, (131,), generator=gen, device="cuda")
    target = torch.randint(ex.VOCAB, (131,), generator=gen, device="cuda").to(torch.int32)
    target[::7] = -100
    loss, grads, ds = ex.loss_and_gradients(p, token, target)
    exact = {n: t.to(torch.bfloat16).to(D).requires_grad_() for n, t in p.items()}
    s, y = forward(ex, exact, token)
    s.retain_grad()
    z = y @ exact["head"].T
    rows = (target >= 0).nonzero()[:, 0]
    want = (torch.logsumexp(z, 1)[rows] - z[rows, target[rows].long()]).mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 4 * U16 * abs(want.item())
    # every tensor between two operators is rounded to bf16 once, six of them on the
    # longest way: each adds at most 2^-8 of its norm
    for name, g in grads.items():
        exact_g = exact[name].grad
        assert (g.to(D) - exact_g).norm() <= 6 * U16 * exact_g.norm(), name
    assert (ds.to(D) - s.grad).norm() <= 7 * U16 * s.grad.norm()


def test_a_served_step(example):
    ex = example
    p, (a, b) = ex.new_parameters(), ex.new_adapters()
    for m in (1, 5, 70):
        adapter = (torch.arange(m, device="cuda") % 3 - 1).to(torch.int32)
        token = torch.randint(ex.VOCAB, (m,), device="cuda")
        server = ex.Server(p, a, b, m)
        base = server(token, torch.full_like(adapter, -1)).clone()
        got = server(token, adapter).clone()
        assert torch.equal(got[adapter < 0], base[adapter < 0])
        # the adapters' share against 64 bits: fp32 rows, so only the sums' roundings
        y = server.y2.to(D)
        for i in range(ex.ADAPTERS):
            at = (adapter == i).nonzero()[:, 0]
            want = y[at] @ a[i].to(D).T @ b[i].to(D).T
            mag = y[at].abs() @ a[i].to(D).abs().T @ b[i].to(D).abs().T
            u = 2.0 ** -24
            bound = mag * (2 * ex.K + 6 * ex.RANK + 16) * u + u * got[at].to(D).abs() + 2 ** -23 * want.abs()
            assert ((got[at].to(D) - base[at].to(D) - want).abs() <= bound).all()
        # the shared layers in 8 bits: codes off by half a step of 127 per value
        exact = {n: t.to(torch.bfloat16).to(D) for n, t in p.items()}
        _, y64 = forward(ex, exact, token)
        z = y64 @ exact["head"].T
        assert (base.to(D) - z).norm() <= 0.1 * z.norm()
        again = server(token, adapter)
        assert torch.equal(again, got)


def test_the_example_runs(example):
    result = example.main(steps=3)
    assert result["kept"] and result["least_moved"] > 0
