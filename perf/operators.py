"""Workloads of the integer product, the gated feed-forward block and the token log probabilities.

Four paths, each in a plain form (elementary torch operations in 32 bits) and
through the library's entry points (``own``):

- ``linear``: bf16 rows quantised per token to int8 times int8 weights with one
  scale per output channel (serving);
- ``gated``: the same product with the fused gate / up layer, the activation
  and the elementwise product (serving);
- ``ffn``: the bf16 gated block, forward (serving a model that is not
  quantised) or forward and backward (training);
- ``logprobs``: log probabilities of given tokens with entropy, rank and top
  alternatives, or, for training, log probabilities and entropy with the
  gradient of the logits.
"""
import math

import torch

own = False

# One hidden size and one feed-forward size of the repository's decode and
# large-M benchmarks (4096, 14336); odd and ragged sizes beside them.
_LISTED = (
    # a single request's decode step: latency, bound by the weight bytes
    dict(name="linear_one_token", op="linear", m=1, n=14336, k=4096, out="bf16"),
    # a small decode batch through a long-K (down) projection
    dict(name="linear_23_rows", op="linear", m=23, n=4096, k=14336, out="bf16"),
    # a short prompt, odd sizes, K that ends inside a 128-block, fp32 output (as a head's logits)
    dict(name="linear_333_rows_odd", op="linear", m=333, n=8187, k=2080, out="f32"),
    # a prefill chunk: bound by the matrix cores
    dict(name="linear_4096_rows", op="linear", m=4096, n=14336, k=4096, out="bf16"),
    # the gate / up half of the block at one token
    dict(name="gated_one_token", op="gated", m=1, inter=14336, k=4096, act="silu", out="bf16"),
    # the same in a mixed batch with an odd inner size
    dict(name="gated_1000_rows_odd", op="gated", m=1000, inter=7001, k=4096, act="gelu", out="bf16"),
    # the unquantised block at one token
    dict(name="ffn_one_token", op="ffn", m=1, inter=14336, k=4096, act="silu", train=False),
    # a small training step with odd sizes
    dict(name="ffn_train_257_rows_odd", op="ffn", m=257, inter=2817, k=1032, act="gelu", train=True),
    # a training step of a full layer: bound by the matrix cores
    dict(name="ffn_train_4096_rows", op="ffn", m=4096, inter=14336, k=4096, act="silu", train=True),
    # the log probabilities of one sampled token: latency
    dict(name="logprobs_one_row", op="logprobs", rows=1, vocab=131072, dtype="f32", top=20, temperature=1.0,
         masked=False, train=False),
    # scoring a batch of prompts, with tokens that a grammar masks out: bound by the logits' bytes
    dict(name="logprobs_2048_rows_masked", op="logprobs", rows=2048, vocab=131072, dtype="bf16", top=20,
         temperature=0.7, masked=True, train=False),
    # a policy-gradient step: log probabilities and entropy, and the logits' gradient
    dict(name="logprobs_train_1021_rows_odd", op="logprobs", rows=1021, vocab=100003, dtype="bf16", top=0,
         temperature=1.0, masked=False, train=True),
)

_MOST_PRODUCT = 4096 * 14336 * 4096   # m * inter * k of the largest training step
_MOST_LOGITS = 2048 * 131072


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "ffn", "ffn", "logprobs", "logprobs"))
    if op == "logprobs":
        train = rng.random() < 0.4
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, min(4096, _MOST_LOGITS // vocab // (2 if train else 1)))
        return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(("bf16", "f32")), top=0 if train else rng.randint(1, 32),
                    temperature=rng.choice((0.5, 1.0, 1.3)), masked=rng.random() < 0.5, train=train)
    while True:
        m = rng.choice((1, _log(rng, 1, 32), _log(rng, 16, 512), _log(rng, 256, 4096)))
        width, k = _log(rng, 200, 16384), 8 * _log(rng, 32, 2048)
        if m * width * k <= _MOST_PRODUCT:
            break
    act = rng.choice(("silu", "gelu"))
    if op == "linear":
        return dict(op=op, m=m, n=width, k=-(-k // 32) * 32, out=rng.choice(("bf16", "f32")))
    if op == "gated":
        return dict(op=op, m=m, inter=width, k=-(-k // 32) * 32, act=act, out=rng.choice(("bf16", "f32")))
    return dict(op=op, m=m, inter=width, k=k, act=act, train=rng.random() < 0.6)


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _up(v, to):
    return -(-v // to) * to


def _hidden(gen, m, k):
    """Hidden states as after a norm layer: unit rows with a few strong channels."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    strong = torch.rand(k, generator=gen, device="cuda") < 0.004
    return (x * torch.where(strong, 12.0, 1.0)).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op in ("linear", "gated"):
        m, k = case["m"], case["k"]
        n = case["n"] if op == "linear" else 2 * case["inter"]
        s["x"] = _hidden(gen, m, k)
        s["codes"] = torch.randn(n, k, generator=gen, device="cuda").mul_(36).round_().clamp_(-127, 127).to(torch.int8)
        s["scales"] = (0.5 + torch.rand(n, generator=gen, device="cuda")) / (36 * math.sqrt(k))
    elif op == "ffn":
        m, k, inter = case["m"], case["k"], case["inter"]
        s["x"] = _hidden(gen, m, k)
        s["w"] = (torch.randn(2 * inter, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
        if case["train"]:
            s["dh"] = torch.randn(m, inter, generator=gen, device="cuda").mul_(0.1).to(torch.bfloat16)
    else:
        rows, vocab = case["rows"], case["vocab"]
        # rows padded to 16 bytes, as a head layer writes them
        logits = torch.empty(rows, _up(vocab, 8), device="cuda", dtype=_type(case["dtype"]))[:, :vocab]
        sharp = 1.0 + 2.0 * torch.rand(rows, 1, generator=gen, device="cuda")
        logits.copy_(torch.randn(rows, vocab, generator=gen, device="cuda") * sharp)
        any_token = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        likely = torch.rand(rows, generator=gen, device="cuda") < 0.6
        s["tokens"] = torch.where(likely, logits.argmax(1), any_token).to(torch.int32)
        if case["masked"]:
            logits.masked_fill_(torch.rand(vocab, generator=gen, device="cuda") < 0.2, -math.inf)
            if rows > 1:
                logits[rows // 2] = -math.inf  # a row whose mask leaves nothing
        s["logits"] = logits
        if case["train"]:
            s["dlogp"] = torch.randn(rows, generator=gen, device="cuda")
            s["dentropy"] = torch.full((rows,), -0.01, device="cuda")
    if own:
        _prepare_own(s)
    return s


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------

def _prepare_own(s):
    """The packed weights, outputs and workspaces that a user's program keeps."""
    import quantized_gemm_qg_amd as qg

    c = s["case"]
    dev = dict(device="cuda")
    s["qg"], s["stream"] = qg, torch.cuda.current_stream().cuda_stream
    if c["op"] in ("linear", "gated"):
        n, k = s["codes"].shape
        desc = qg.layer_desc(qg.W_INT8, n, k, k, atype=qg.A_INT8_TOKEN)
        s["packed"] = torch.empty(qg.packed_size(desc), dtype=torch.uint8, **dev)
        s["weight"] = qg.preprocess(desc, s["codes"].cpu().numpy(), s["scales"].cpu().numpy(), None, s["packed"])
        width = n if c["op"] == "linear" else c["inter"]
        size = qg.gemm_workspace_size_ex if c["op"] == "linear" else qg.gated_gemm_workspace_size
        s["ws_bytes"] = size(s["weight"], c["m"], qg.GEMM_QUANTIZE_X)
        s["out"] = torch.empty(c["m"], _up(width, 8), dtype=_type(c["out"]), **dev)
        s["y"] = s["out"][:, :width]
        s["otype"] = qg.O_F32 if c["out"] == "f32" else qg.O_BF16
    elif c["op"] == "ffn":
        m, k, inter = c["m"], c["k"], c["inter"]
        s["h"] = torch.empty(m, _up(inter, 8), dtype=torch.bfloat16, **dev)
        s["ws_bytes"] = qg.ffn_gated_workspace_size(m, k, inter)
        if c["train"]:
            s["gu"] = torch.empty(m, _up(2 * inter, 4), **dev)
            s["dx"] = torch.empty(m, k, dtype=torch.bfloat16, **dev)
            s["dw"] = torch.empty(2 * inter, k, dtype=torch.bfloat16, **dev)
            s["ws_bytes"] = max(s["ws_bytes"], qg.ffn_gated_backward_workspace_size(m, k, inter))
    else:
        rows, top = c["rows"], c["top"]
        for name in ("logp", "entropy"):
            s[name] = torch.empty(rows, **dev)
        s["stats"] = torch.empty(rows, 2, **dev) if c["train"] else None
        if top:
            s["rank"] = torch.empty(rows, dtype=torch.int32, **dev)
            s["top_ids"] = torch.empty(rows, top, dtype=torch.int32, **dev)
            s["top_logp"] = torch.empty(rows, top, **dev)
        s["ws_bytes"] = qg.token_logprobs_workspace_size(rows, c["vocab"], top)
        if c["train"]:
            s["dlogits"] = torch.empty(rows, s["logits"].stride(0), dtype=s["logits"].dtype, **dev)
        s["ltype"] = qg.O_F32 if c["dtype"] == "f32" else qg.O_BF16
    if "act" in c:
        s["act"] = qg.ACT_SILU if c["act"] == "silu" else qg.ACT_GELU_TANH
    s["ws"] = torch.zeros(max(s["ws_bytes"], 1), dtype=torch.uint8, **dev)


def _run_own(s):
    qg, c, stream, ws = s["qg"], s["case"], s["stream"], (s["ws"], s["ws_bytes"])
    if c["op"] == "linear":
        qg.gemm_ex(s["weight"], s["x"], None, c["m"], c["k"], s["out"], s["otype"], s["out"].stride(0), *ws,
                   qg.GEMM_QUANTIZE_X, stream)
        return s["y"]
    if c["op"] == "gated":
        qg.gated_gemm(s["weight"], s["x"], None, c["m"], c["k"], s["out"], s["otype"], s["out"].stride(0), s["act"], *ws,
                      qg.GEMM_QUANTIZE_X, stream)
        return s["y"]
    if c["op"] == "ffn":
        m, k, inter = c["m"], c["k"], c["inter"]
        h = s["h"]
        if not c["train"]:
            qg.ffn_gated(s["x"], k, s["w"], k, m, k, inter, s["act"], h, h.stride(0), *ws, stream=stream)
            return h[:, :inter]
        gu = s["gu"]
        qg.ffn_gated(s["x"], k, s["w"], k, m, k, inter, s["act"], h, h.stride(0), *ws, gu=gu, gu_type=qg.O_F32,
                     ldgu=gu.stride(0), stream=stream)
        qg.ffn_gated_backward(s["x"], k, s["w"], k, s["dh"], inter, m, k, inter, s["act"], s["dx"], k, s["dw"], qg.O_BF16, k,
                              *ws, gu=gu, gu_type=qg.O_F32, ldgu=gu.stride(0), stream=stream)
        return dict(h=h[:, :inter], dx=s["dx"], dw=s["dw"])
    rows, vocab, ld, scale = c["rows"], c["vocab"], s["logits"].stride(0), 1.0 / c["temperature"]
    qg.token_logprobs(s["logits"], s["ltype"], rows, vocab, ld, s["tokens"], scale, c["top"], s["logp"], s["entropy"],
                      s["stats"], s.get("rank"), s.get("top_ids"), s.get("top_logp"), *ws, stream)
    if not c["train"]:
        return dict(logp=s["logp"], entropy=s["entropy"], rank=s["rank"], top_ids=s["top_ids"], top_logp=s["top_logp"])
    qg.token_logprobs_backward(s["logits"], s["ltype"], rows, vocab, ld, s["tokens"], scale, s["stats"], s["entropy"],
                               s["dlogp"], s["dentropy"], s["dlogits"], ld, stream)
    return dict(logp=s["logp"], entropy=s["entropy"], dlogits=s["dlogits"][:, :vocab])


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _activation(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _int8_product(s):
    x = s["x"].float()
    most = x.abs().amax(1, keepdim=True)
    scale = torch.where(most > 0, most / torch.full_like(most, 127.0), torch.ones_like(most))
    q = torch.round(x / scale).clamp(-127, 127)
    return (q @ s["codes"].float().T) * scale * s["scales"]


def _ordered(v):
    """int64 keys that sort as the fp32 values do."""
    bits = v.view(torch.int32).to(torch.int64)
    return torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)


def _plain_logprobs(s):
    c = s["case"]
    vocab = c["vocab"]
    logits = s["logits"].float()
    z = logits * (1.0 / c["temperature"])
    most = z.amax(1, keepdim=True)
    empty = most == -math.inf
    e = torch.exp(z - torch.where(empty, torch.zeros_like(most), most))
    total = e.sum(1, keepdim=True)
    lse = most + torch.log(torch.where(empty, torch.ones_like(total), total))
    p = e / torch.where(empty, torch.ones_like(total), total)
    logp_all = torch.where(z == -math.inf, z, z - lse)
    entropy = -torch.where(p > 0, p * logp_all, torch.zeros_like(p)).sum(1)
    at = s["tokens"].long().unsqueeze(1)
    logp = logp_all.gather(1, at).squeeze(1)
    if c["train"]:
        hit = torch.zeros_like(p).scatter_(1, at, 1.0)
        info = torch.where(p > 0, p * (logp_all + entropy.unsqueeze(1)), torch.zeros_like(p))
        dz = s["dlogp"].unsqueeze(1) * (hit - p) - s["dentropy"].unsqueeze(1) * info
        dz = torch.where(empty, torch.zeros_like(dz), dz) * (1.0 / c["temperature"])
        return dict(logp=logp, entropy=entropy, dlogits=dz.to(s["logits"].dtype))
    rank = (logits > logits.gather(1, at)).sum(1).to(torch.int32)
    # equal values in the order of their ids
    key = _ordered(logits) * (1 << 20) + (vocab - 1 - torch.arange(vocab, device=logits.device))
    ids = vocab - 1 - (key.topk(c["top"], dim=1).values & ((1 << 20) - 1))
    top_logp = logp_all.gather(1, ids)
    ids = torch.where(top_logp == -math.inf, torch.full_like(ids, -1), ids)
    return dict(logp=logp, entropy=entropy, rank=rank, top_ids=ids.to(torch.int32), top_logp=top_logp)


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "linear":
        return _int8_product(state).to(_type(c["out"]))
    if c["op"] == "gated":
        y = _int8_product(state)
        g, u = y[:, :c["inter"]], y[:, c["inter"]:]
        return (_activation(g, c["act"])[0] * u).to(_type(c["out"]))
    if c["op"] == "ffn":
        x, w, inter = state["x"].float(), state["w"].float(), c["inter"]
        gu = x @ w.T
        g, u = gu[:, :inter], gu[:, inter:]
        a, slope = _activation(g, c["act"])
        h = (a * u).to(torch.bfloat16)
        if not c["train"]:
            return h
        dh = state["dh"].float()
        dgu = torch.cat((dh * u * slope, dh * a), 1)
        return dict(h=h, dx=(dgu @ w).to(torch.bfloat16), dw=(dgu.T @ x).to(torch.bfloat16))
    return _plain_logprobs(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c, el = case, {"bf16": 2, "f32": 4}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=2 * m * k + n * k + 4 * n + el[c["out"]] * m * n, flops=2 * m * n * k)
    if c["op"] == "gated":
        m, n, k = c["m"], 2 * c["inter"], c["k"]
        return dict(bytes=2 * m * k + n * k + 4 * n + el[c["out"]] * m * c["inter"], flops=2 * m * n * k)
    if c["op"] == "ffn":
        m, i, k = c["m"], c["inter"], c["k"]
        if not c["train"]:
            return dict(bytes=2 * (m * k + 2 * i * k + m * i), flops=4 * m * i * k)
        return dict(bytes=2 * (2 * m * k + 4 * i * k + 2 * m * i), flops=12 * m * i * k)
    v = c["rows"] * c["vocab"]
    if c["train"]:
        return dict(bytes=2 * v * el[c["dtype"]] + 24 * c["rows"], flops=12 * v)
    return dict(bytes=v * el[c["dtype"]] + c["rows"] * (16 + 8 * c["top"]), flops=6 * v)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, d = case["op"], torch.float64
    if op in ("linear", "gated"):
        # the codes by their definition (fp32 scale and quotient, half to even), then exact sums
        x = s["x"].cpu().float().numpy()
        most = abs(x).max(1, keepdims=True)
        step = most / most.dtype.type(127)
        step[most == 0] = 1
        q = torch.from_numpy((x / step).round()).clamp_(-127, 127).cuda().to(d)
        y = torch.mm(q, s["codes"].to(d).t().contiguous())
        y *= torch.from_numpy(step).cuda().to(d)
        y *= s["scales"].to(d)[None]
        return y if op == "linear" else _gate64(y[:, :case["inter"]], case["act"])[0] * y[:, case["inter"]:]
    if op == "ffn":
        inter = case["inter"]
        x, wg, wu = s["x"].to(d), s["w"][:inter].to(d), s["w"][inter:].to(d)
        g, u = torch.mm(x, wg.t().contiguous()), torch.mm(x, wu.t().contiguous())
        a, slope = _gate64(g, case["act"])
        if not case["train"]:
            return a * u
        dh = s["dh"].to(d)
        dg, du = dh * u * slope, dh * a
        return dict(h=a * u, dx=torch.mm(dg, wg) + torch.mm(du, wu),
                    dw=torch.cat((torch.mm(dg.t().contiguous(), x), torch.mm(du.t().contiguous(), x))))
    z = s["logits"].to(d) / case["temperature"]
    lse = torch.logsumexp(z, 1)
    logq = (z - lse[:, None]).masked_fill_(z == -math.inf, -math.inf)
    p = torch.exp(logq)
    entropy = torch.special.entr(p).sum(1)
    tok = s["tokens"].long()
    logp = logq[torch.arange(len(tok), device="cuda"), tok]
    if not case["train"]:
        return dict(logp=logp, entropy=entropy, rank=None, top_ids=None, top_logp=logq.topk(case["top"], 1).values)
    grad = p * (-s["dlogp"].to(d)[:, None])
    grad -= s["dentropy"].to(d)[:, None] * (p * entropy[:, None] - torch.special.entr(p))
    grad[torch.arange(len(tok), device="cuda"), tok] += s["dlogp"].to(d)
    grad[lse == -math.inf] = 0
    return dict(logp=logp, entropy=entropy, dlogits=grad / case["temperature"])


def _gate64(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    r = math.sqrt(2 / math.pi)
    t = torch.tanh(r * g * (1 + 0.044715 * g ** 2))
    return g * (1 + t) / 2, (1 + t + g * (1 - t ** 2) * r * (1 + 0.134145 * g ** 2)) / 2
