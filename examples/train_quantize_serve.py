"""Trains a small gated block as a next-token predictor, quantizes it to int8 and
serves it one token at a time.

    python examples/train_quantize_serve.py [--steps 60] [--tokens 32]

The model is one gated feed-forward block between an embedding and an output
head: h = act(x Wg^T) (x Wu^T), logits = h H^T.  It learns a fixed successor of
every token, which a share of the training targets contradicts.

  training   ffn_gated (pre-activations saved in fp32), the head by torch,
             token_logprobs and token_logprobs_backward for the loss
             -log p(target) - c entropy, ffn_gated_backward for dW
  serving    gate / up and head weights as int8 with one scale per channel,
             activations quantized per token inside the calls: gated_gemm, then
             gemm_ex, then token_logprobs with its alternatives picks the token
  judging    log probabilities of the same targets before and after quantizing
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_qg_amd as qg  # noqa: E402

K, INTER, VOCAB, ACT = 256, 704, 1000, qg.ACT_SILU
NOISE = 0.3   # share of targets that another token's successor replaces


def workspace(nbytes):
    return torch.zeros(max(nbytes, 1), dtype=torch.uint8, device="cuda")


class Scores:
    """Buffers of token_logprobs and its gradient for up to `rows` rows."""

    def __init__(self, rows, top=0):
        f32 = dict(dtype=torch.float32, device="cuda")
        self.rows, self.top = rows, top
        self.logp, self.entropy, self.stats = (torch.empty(s, **f32) for s in ((rows,), (rows,), (rows, 2)))
        self.ids = torch.empty(rows, max(top, 1), dtype=torch.int32, device="cuda")
        self.top_logp = torch.empty(rows, max(top, 1), **f32)
        self.ws = workspace(qg.token_logprobs_workspace_size(rows, VOCAB, top))

    def __call__(self, logits, tokens):
        out = dict(top_ids=self.ids, top_logp=self.top_logp) if self.top else {}
        qg.token_logprobs(logits, qg.O_F32, self.rows, VOCAB, logits.stride(0), tokens, 1.0, self.top, self.logp, self.entropy,
                          stats=self.stats, ws=self.ws, ws_bytes=self.ws.numel(), **out)


def int8_layer(weight):
    """Codes and scales of a [channels][k] matrix, packed on the device."""
    w = weight.float().cpu()
    scale = w.abs().amax(1).clamp_min(1e-12) / 127
    codes = (w / scale[:, None]).round().clamp(-127, 127).to(torch.int8)
    desc = qg.layer_desc(qg.W_INT8, w.shape[0], w.shape[1], w.shape[1], atype=qg.A_INT8_TOKEN)
    packed = torch.empty(qg.packed_size(desc), dtype=torch.uint8, device="cuda")
    return qg.preprocess(desc, codes.numpy(), scale.numpy(), None, packed), packed


def train(embed, head, successor, steps, batch=512, rate=0.05, entropy_weight=0.01):
    gen = torch.Generator(device="cuda").manual_seed(1)
    master = torch.randn(2 * INTER, K, generator=gen, device="cuda") / K ** 0.5
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    h, dh = torch.empty(batch, INTER, **bf16), torch.empty(batch, INTER, **bf16)
    gu = torch.empty(batch, 2 * INTER, device="cuda")
    dw = torch.empty(2 * INTER, K, device="cuda")
    dlogits = torch.empty(batch, VOCAB, device="cuda")
    scores = Scores(batch)
    ws = workspace(max(qg.ffn_gated_workspace_size(batch, K, INTER), qg.ffn_gated_backward_workspace_size(batch, K, INTER)))
    dlogp = torch.full((batch,), -1.0 / batch, device="cuda")
    dentropy = torch.full((batch,), -entropy_weight / batch, device="cuda")
    losses = []
    for step in range(steps):
        token = torch.randint(VOCAB, (batch,), generator=gen, device="cuda")
        noise = torch.rand(batch, generator=gen, device="cuda") < NOISE
        x, target = embed[token], torch.where(noise, successor[token.flip(0)], successor[token])
        w = master.to(torch.bfloat16)
        qg.ffn_gated(x, K, w, K, batch, K, INTER, ACT, h, INTER, ws, ws.numel(), gu=gu, gu_type=qg.O_F32, ldgu=2 * INTER)
        logits = h.float() @ head.float().T
        scores(logits, target)
        qg.token_logprobs_backward(logits, qg.O_F32, batch, VOCAB, VOCAB, target, 1.0, scores.stats, scores.entropy, dlogp,
                                   dentropy, dlogits, VOCAB)
        dh.copy_(dlogits @ head.float())
        qg.ffn_gated_backward(x, K, w, K, dh, INTER, batch, K, INTER, ACT, None, K, dw, qg.O_F32, K, ws, ws.numel(), gu=gu,
                              gu_type=qg.O_F32, ldgu=2 * INTER)
        master -= rate * (1 - step / steps) * master.norm() / dw.norm() * dw
        losses.append(-scores.logp.mean().item())
    return master.to(torch.bfloat16), losses


def logits_int8(x, gate_up, head, h, logits, ws):
    m, flags = x.shape[0], qg.GEMM_QUANTIZE_X
    qg.gated_gemm(gate_up, x, None, m, K, h, qg.O_BF16, INTER, ACT, ws, ws.numel(), flags)
    qg.gemm_ex(head, h, None, m, INTER, logits, qg.O_F32, VOCAB, ws, ws.numel(), flags)


def main(steps=60, tokens=32):
    gen = torch.Generator(device="cuda").manual_seed(0)
    embed = torch.randn(VOCAB, K, generator=gen, device="cuda").to(torch.bfloat16)
    head = (torch.randn(VOCAB, INTER, generator=gen, device="cuda") / INTER ** 0.5).to(torch.bfloat16)
    successor = torch.randperm(VOCAB, generator=gen, device="cuda").to(torch.int32)

    w, losses = train(embed, head, successor, steps)

    # the same targets by the bf16 block and by the int8 layers
    h = torch.empty(VOCAB, INTER, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(VOCAB, VOCAB, device="cuda")
    scores = Scores(VOCAB)
    ws = workspace(qg.ffn_gated_workspace_size(VOCAB, K, INTER))
    qg.ffn_gated(embed, K, w, K, VOCAB, K, INTER, ACT, h, INTER, ws, ws.numel())
    scores(h.float() @ head.float().T, successor)
    before = scores.logp.clone()
    (gate_up, keep0), (head8, keep1) = int8_layer(w), int8_layer(head)
    ws = workspace(max(qg.gated_gemm_workspace_size(gate_up, VOCAB, qg.GEMM_QUANTIZE_X),
                       qg.gemm_workspace_size_ex(head8, VOCAB, qg.GEMM_QUANTIZE_X)))
    logits_int8(embed, gate_up, head8, h, logits, ws)
    scores(logits, successor)
    after = scores.logp.clone()

    # greedy decoding, a token at a time
    one = Scores(1, top=4)
    token, right = torch.zeros(1, dtype=torch.int64, device="cuda"), 0
    for _ in range(tokens):
        logits_int8(embed[token], gate_up, head8, h, logits, ws)
        one(logits[:1], successor[token])
        right += int(one.ids[0, 0] == successor[token][0])
        token = one.ids[0, :1].long()
    del keep0, keep1
    result = dict(first_loss=losses[0], last_loss=losses[-1], logp_bf16=before.mean().item(), logp_int8=after.mean().item(),
                  drift=(after - before).abs().mean().item(), greedy_right=right / tokens)
    print("loss {first_loss:.3f} -> {last_loss:.3f}; mean log p bf16 {logp_bf16:.3f}, int8 {logp_int8:.3f} (mean change "
          "{drift:.4f}); greedy tokens right {greedy_right:.0%}".format(**result))
    return result


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=32)
    main(**vars(p.parse_args()))
