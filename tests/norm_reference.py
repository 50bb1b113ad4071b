"""The root-mean-square norm, its codes and its gradients by their formulas in
64 bits, and bounds on what fp32 arithmetic may differ by."""
import torch

import quantized_gemm_qg_amd as qg

D = torch.float64
U32 = 2.0 ** -24


def types(t):
    return torch.float32 if t == qg.O_F32 else torch.bfloat16


def half_step(t):
    return torch.finfo(t).eps / 2


def added(x, residual, res_type):
    """s as the library keeps it: one fp32 addition, then the type's rounding."""
    if res_type is None:
        return x.to(D)
    s = x.float() + residual.float() if residual is not None else x.float()
    return s.to(types(res_type)).to(D)


def norm(s, w, eps):
    """y and a bound on its fp32 error: the mean of k squares is off by at most
    (k / 2 + 3) roundings relative (any order of the sums; half of it after the
    root), then root, reciprocal and two products."""
    k = s.shape[1]
    y = s * w / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return y, (k / 2 + 8) * U32


def codes(y, q_type):
    """Codes as values before their rounding and scales (fp32 ones not rounded)."""
    rows, k = y.shape
    size = {qg.A_MXFP8: 32, qg.A_FP8_BLOCK: 128}.get(q_type, k)
    p = torch.zeros(rows, -(-k // size) * size, dtype=D)
    p[:, :k] = y
    p = p.view(rows, -1, size)
    most = p.abs().amax(2)
    if q_type == qg.A_MXFP8:
        scale = torch.exp2(torch.floor(torch.log2(most)) - 8)
    else:
        scale = (most / (127 if q_type == qg.A_INT8_TOKEN else 448)).clamp_min(2.0 ** -126)
    scale = torch.where(most > 0, scale, torch.ones_like(scale))
    return (p / scale[..., None]).view(rows, -1)[:, :k], scale


def gradients(s, w, eps, dy, dsum):
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    g = dy * w
    dx = r * (g - s * r * r * (g * s).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * s * r).sum(0)
