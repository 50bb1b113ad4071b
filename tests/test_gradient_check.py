"""The difference check of the feed-forward block's gradients accepts the right
ones and refuses mistakes planted in them (CPU)."""
import math

import pytest
import torch

from gradient_check import D, check_block_gradients, gate

REL = 2.0 ** -7


def closed_form(x, w, dh, silu, slope_term=True):
    inter = w.shape[0] // 2
    gu = x @ w.T
    g, u = gu[:, :inter], gu[:, inter:]
    z = g if silu else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    dz = 1 if silu else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    p = torch.sigmoid(z)
    da = p + (g * p * (1 - p) * dz if slope_term else 0)
    dgu = torch.cat((dh * u * da, dh * gate(g, silu)), 1)
    return dgu @ w, dgu.T @ x


def case(m=70, k=136, inter=45):
    gen = torch.Generator().manual_seed(11)
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(D)  # noqa: E731
    return bf(m, k), bf(2 * inter, k) * (1.5 / math.sqrt(k)), bf(m, inter)


@pytest.mark.parametrize("silu", [True, False])
def test_right_gradients_pass(silu):
    x, w, dh = case()
    dx, dw = closed_form(x, w, dh, silu)
    check_block_gradients(x, w, dh, silu, dx, dw, 1e-6)
    # rounded once to bf16 as well
    check_block_gradients(x, w, dh, silu, dx.to(torch.bfloat16).to(D), dw.to(torch.bfloat16).to(D), REL)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("mistake", ["no dx", "no dw", "half", "slope term", "halves swapped", "a row", "a column", "2 %"])
def test_planted_mistakes_fail(silu, mistake):
    x, w, dh = case()
    dx, dw = closed_form(x, w, dh, silu, slope_term=mistake != "slope term")
    if mistake == "no dx":
        dx = torch.zeros_like(dx)
    elif mistake == "no dw":
        dw = torch.zeros_like(dw)
    elif mistake == "half":
        dx, dw = dx / 2, dw / 2
    elif mistake == "halves swapped":
        dw = dw.roll(dw.shape[0] // 2, 0)
    elif mistake == "a row":
        dx[-1] = dx[-2]
    elif mistake == "a column":
        dw[:, 0] *= -1
    elif mistake == "2 %":
        dx = dx * 1.02
    with pytest.raises(AssertionError):
        check_block_gradients(x, w, dh, silu, dx, dw, REL)
