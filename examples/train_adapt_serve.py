"""Trains a small residual block with its norms and head, then serves it in int8 with
adapters of two requests.

    python examples/train_adapt_serve.py [--steps 40]

    s = e[token],  h = act(norm(s) Wg^T) (norm(s) Wu^T),  s2 = s + h Wd^T,
    logits = norm(s2) H^T

  training   rmsnorm, ffn_gated, rmsnorm with the residual's addition,
             linear_xent for the mean loss (no logits in memory); backward:
             linear_xent_backward, rmsnorm_backward (its gradient goes past the
             block as well), ffn_gated_backward, rmsnorm_backward
  serving    rmsnorm to int8 codes, gated_gemm on them, gemm_ex, rmsnorm with the
             residual to codes and to bf16: the codes go through the shared int8
             head, the bf16 rows through the adapters of the requests that have
             one (lora), added to the same logits
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_qg_amd as qg  # noqa: E402

K, INTER, VOCAB, RANK, ADAPTERS = 256, 512, 1003, 8, 2
ACT, EPS = qg.ACT_SILU, 1e-5
BF16 = torch.bfloat16


def workspace(nbytes):
    return torch.zeros(max(nbytes, 1), dtype=torch.uint8, device="cuda")


def new_parameters(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(embed=rand(VOCAB, K), gate_up=rand(2 * INTER, K) / K ** 0.5, down=rand(K, INTER) / INTER ** 0.5,
                norm1=1 + 0.1 * rand(K), norm2=1 + 0.1 * rand(K), head=rand(VOCAB, K) / K ** 0.5)


def loss_and_gradients(p, token, target):
    """Mean loss over the targets that are a token, and the gradients of all parameters but the embedding."""
    m = len(token)
    p = {n: t.to(BF16) for n, t in p.items()}
    new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    f32 = torch.float32
    ws = workspace(max(qg.ffn_gated_workspace_size(m, K, INTER), qg.ffn_gated_backward_workspace_size(m, K, INTER),
                       qg.rmsnorm_backward_workspace_size(m, K), qg.linear_xent_workspace_size(m, K, VOCAB),
                       qg.linear_xent_backward_workspace_size(m, K, VOCAB)))
    w = (ws, ws.numel())
    s, y, h, gu = p["embed"][token].contiguous(), new(m, K), new(m, INTER), new(m, 2 * INTER, t=f32)
    s2, y2, loss, lse = new(m, K), new(m, K), new(m, t=f32), new(m, t=f32)
    qg.rmsnorm(s, qg.O_BF16, K, p["norm1"], EPS, m, K, y=y, ldy=K)
    qg.ffn_gated(y, K, p["gate_up"], K, m, K, INTER, ACT, h, INTER, *w, gu=gu, gu_type=qg.O_F32, ldgu=2 * INTER)
    out = (h.float() @ p["down"].float().T).contiguous()
    qg.rmsnorm(out, qg.O_F32, K, p["norm2"], EPS, m, K, residual=s, res_type=qg.O_BF16, ldr=K, sum=s2, lds=K, y=y2, ldy=K)
    qg.linear_xent(y2, K, p["head"], K, m, K, VOCAB, target, 1.0, loss, lse, *w)

    counts = (target >= 0).sum()
    dloss = torch.ones(m, device="cuda") / counts
    dy2, dhead, ds2, dnorm2 = new(m, K), new(VOCAB, K, t=f32), new(m, K), new(K, t=f32)
    dy, dgate_up, ds, dnorm1 = new(m, K), new(2 * INTER, K, t=f32), new(m, K), new(K, t=f32)
    qg.linear_xent_backward(y2, K, p["head"], K, m, K, VOCAB, target, 1.0, lse, dloss, dy2, K, dhead, qg.O_F32, K, *w)
    qg.rmsnorm_backward(s2, qg.O_BF16, K, p["norm2"], EPS, m, K, dy2, K, ds2, K, dnorm2, qg.O_F32, *w)
    ddown = ds2.float().T @ h.float()
    dh = (ds2.float() @ p["down"].float()).to(BF16)
    qg.ffn_gated_backward(y, K, p["gate_up"], K, dh, INTER, m, K, INTER, ACT, dy, K, dgate_up, qg.O_F32, K, *w, gu=gu,
                          gu_type=qg.O_F32, ldgu=2 * INTER)
    # what reached s past the block is added to what comes back through it
    qg.rmsnorm_backward(s, qg.O_BF16, K, p["norm1"], EPS, m, K, dy, K, ds, K, dnorm1, qg.O_F32, *w, dsum=ds2, ldds=K)
    return loss.sum() / counts, dict(gate_up=dgate_up, down=ddown, norm1=dnorm1, norm2=dnorm2, head=dhead), ds


def int8_layer(weight):
    """Codes and scales of a [channels][k] matrix, packed on the device."""
    w = weight.float().cpu()
    scale = w.abs().amax(1).clamp_min(1e-12) / 127
    codes = (w / scale[:, None]).round().clamp(-127, 127).to(torch.int8)
    desc = qg.layer_desc(qg.W_INT8, w.shape[0], w.shape[1], w.shape[1], atype=qg.A_INT8_TOKEN)
    packed = torch.empty(qg.packed_size(desc), dtype=torch.uint8, device="cuda")
    return qg.preprocess(desc, codes.numpy(), scale.numpy(), None, packed), packed


class Server:
    """The model in int8 with adapters on its head's output, for m rows."""

    def __init__(self, p, a, b, m):
        self.p, self.a, self.b, self.m = {n: t.to(BF16) for n, t in p.items()}, a, b, m
        self.gate_up, self.down, self.head = (int8_layer(p[n]) for n in ("gate_up", "down", "head"))
        new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.q, self.qs = new(m, K, t=torch.int8), new(m, t=torch.float32)
        self.h, self.out, self.s2, self.y2 = new(m, INTER), new(m, K), new(m, K), new(m, K)
        self.logits = new(m, VOCAB, t=torch.float32)
        self.sorted, self.offsets = new(m, t=torch.int32), new(ADAPTERS + 1, t=torch.int32)
        self.sort_ws = workspace(256)
        self.ws = workspace(max(qg.gated_gemm_workspace_size(self.gate_up[0], m),
                                qg.gemm_workspace_size_ex(self.down[0], m, qg.GEMM_QUANTIZE_X),
                                qg.gemm_workspace_size_ex(self.head[0], m, 0),
                                qg.lora_workspace_size(m, K, VOCAB, ADAPTERS, RANK)))

    def __call__(self, token, adapter):
        """Logits of the rows' next tokens; adapter int32 [m], -1 for none."""
        p, m, w = self.p, self.m, (self.ws, self.ws.numel())
        s = p["embed"][token].contiguous()
        qg.moe_sort(adapter, m, 1, ADAPTERS, self.sorted, self.offsets, self.sort_ws, 256)
        qg.rmsnorm(s, qg.O_BF16, K, p["norm1"], EPS, m, K, q_type=qg.A_INT8_TOKEN, q=self.q, ldq=K, q_scales=self.qs)
        qg.gated_gemm(self.gate_up[0], self.q, self.qs, m, K, self.h, qg.O_BF16, INTER, ACT, *w)
        qg.gemm_ex(self.down[0], self.h, None, m, INTER, self.out, qg.O_BF16, K, *w, qg.GEMM_QUANTIZE_X)
        qg.rmsnorm(self.out, qg.O_BF16, K, p["norm2"], EPS, m, K, residual=s, res_type=qg.O_BF16, ldr=K, sum=self.s2, lds=K, y=self.y2,
                   ldy=K, q_type=qg.A_INT8_TOKEN, q=self.q, ldq=K, q_scales=self.qs)
        qg.gemm_ex(self.head[0], self.q, self.qs, m, K, self.logits, qg.O_F32, VOCAB, *w, 0)
        qg.lora(self.y2, K, self.a, K, self.b, RANK, None, ADAPTERS, RANK, self.sorted, self.offsets, m, K, VOCAB, self.logits,
                qg.O_F32, VOCAB, *w)
        return self.logits


def new_adapters(seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return (rand(ADAPTERS, RANK, K) / K ** 0.5).to(BF16), rand(ADAPTERS, VOCAB, RANK).to(BF16)


def main(steps=40, batch=300, rate=0.05):
    p = new_parameters()
    gen = torch.Generator(device="cuda").manual_seed(2)
    successor = torch.randperm(VOCAB, generator=gen, device="cuda")
    losses = []
    for step in range(steps):
        token = torch.randint(VOCAB, (batch,), generator=gen, device="cuda")
        target = successor[token].to(torch.int32)
        target[torch.rand(batch, generator=gen, device="cuda") < 0.1] = -100   # rows that do not count
        loss, grads, _ = loss_and_gradients(p, token, target)
        for name, g in grads.items():
            p[name] -= rate * (1 - step / steps) * p[name].norm() / g.norm().clamp_min(1e-12) * g
        losses.append(loss.item())

    server = Server(p, *new_adapters(), 6)
    token = torch.arange(6, device="cuda")
    none = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    base = server(token, none).clone()
    adapted = server(token, torch.tensor([0, 0, 1, 1, -1, -1], dtype=torch.int32, device="cuda")).clone()
    moved = (adapted - base).abs().amax(1)
    result = dict(first_loss=losses[0], last_loss=losses[-1], kept=torch.equal(base[4:], adapted[4:]), least_moved=moved[:4].min().item(),
                  right=(base.argmax(1) == successor[token]).float().mean().item())
    print("loss {first_loss:.3f} -> {last_loss:.3f}; int8 next tokens right {right:.0%}; rows without an adapter kept: {kept}, "
          "the others moved by {least_moved:.2f} and more".format(**result))
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    main(**vars(ap.parse_args()))
