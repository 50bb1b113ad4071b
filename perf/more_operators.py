"""Workloads of the root-mean-square norm, the low-rank adapters and the cross entropy of a head layer.

Three paths, each in a plain form (elementary torch operations in 32 bits) and
through the library's entry points (``own``):

- ``norm``: the residual's addition and the norm, to bf16 and / or to 8 bits
  with scales (serving), or forward and backward (training);
- ``lora``: low-rank adapters of many requests added in place to the output of
  a shared projection (serving);
- ``xent``: softmax cross entropy of hidden states against a head's weights
  without logits in memory: the loss alone (scoring), or with the gradients of
  both (training).
"""
import math

import torch

own = False

# The hidden size of the repository's benchmarks (4096) and its feed-forward
# size (14336); odd and ragged sizes beside them.
_LISTED = (
    # a decode step between two layers: latency
    dict(name="norm_one_token_fp8", op="norm", rows=1, k=4096, x="bf16", res="bf16", y=False, q="fp8", train=False),
    # a mixed batch, odd sizes, rows that end inside a block of 128, fp32 input from a projection; adapters read y, the product q
    dict(name="norm_333_rows_fp8_blocks", op="norm", rows=333, k=5128, x="f32", res=None, y=True, q="fp8b", train=False),
    # a prompt ahead of an int8 layer, residual stream in fp32
    dict(name="norm_1001_rows_int8", op="norm", rows=1001, k=2080, x="bf16", res="f32", y=False, q="int8", train=False),
    # a large prefill, both outputs: bound by bytes
    dict(name="norm_16384_rows_mxfp8", op="norm", rows=16384, k=4096, x="bf16", res="bf16", y=True, q="mxfp8", train=False),
    # a training step's norm, forward and backward
    dict(name="norm_train_4096_rows", op="norm", rows=4096, k=4096, x="bf16", res="bf16", y=True, q=None, train=True),
    # a single request with an adapter: latency
    dict(name="lora_one_token", op="lora", m=1, k=4096, n=4096, rank=16, adapters=8, prompts=False, out="bf16"),
    # a decode batch, most rows with an adapter of their own, some without
    dict(name="lora_decode_64", op="lora", m=64, k=4096, n=14336, rank=16, adapters=48, prompts=False, out="bf16"),
    # odd sizes, fp32 rows (a head's logits), every request its prompt
    dict(name="lora_333_rows_odd", op="lora", m=333, k=2088, n=8187, rank=24, adapters=5, prompts=True, out="f32"),
    # prompts of several requests: bound by the output's bytes
    dict(name="lora_prefill_4096", op="lora", m=4096, k=4096, n=14336, rank=64, adapters=6, prompts=True, out="bf16"),
    # scoring a short answer: bound by the weights' bytes
    dict(name="xent_61_tokens", op="xent", m=61, vocab=100003, k=2048, train=False),
    # a small training step with odd sizes
    dict(name="xent_train_257_odd", op="xent", m=257, vocab=38531, k=1032, train=True),
    # a training step of a full head: bound by the matrix cores
    dict(name="xent_train_4096", op="xent", m=4096, vocab=131072, k=4096, train=True),
)

_MOST_HEAD = 4096 * 131072 * 4096   # m * vocab * k of the largest training step
_EPS = 1e-5


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "lora", "xent"))
    if op == "norm":
        k = 32 * _log(rng, 8, 512) if rng.random() < 0.5 else 8 * _log(rng, 32, 2048)
        rows = _log(rng, 1, 16384 * 4096 // max(k, 4096))
        train = rng.random() < 0.35
        q = None if train else rng.choice((None, "int8", "fp8", "fp8b", "mxfp8" if k % 32 == 0 else "fp8b"))
        return dict(op=op, rows=rows, k=k, x=rng.choice(("bf16", "bf16", "f32")), res=rng.choice((None, "bf16", "bf16", "f32")),
                    y=train or q is None or rng.random() < 0.5, q=q, train=train)
    if op == "lora":
        m = rng.choice((_log(rng, 1, 128), _log(rng, 1, 4096)))
        return dict(op=op, m=m, k=8 * _log(rng, 32, 2048), n=_log(rng, 200, 16384), rank=8 * rng.choice((1, 2, 2, 3, 4, 8, 16)),
                    adapters=_log(rng, 1, 64), prompts=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
    while True:
        m, vocab, k = rng.choice((_log(rng, 1, 64), _log(rng, 1, 4096))), _log(rng, 1000, 200000), 8 * _log(rng, 32, 1024)
        if m * vocab * k <= _MOST_HEAD and vocab * k <= 1 << 30:
            return dict(op=op, m=m, vocab=vocab, k=k, train=rng.random() < 0.6)


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _up(v, to):
    return -(-v // to) * to


def _hidden(gen, m, k):
    """Rows as a layer writes them: unit variance with a few strong channels."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    strong = torch.rand(k, generator=gen, device="cuda") < 0.004
    return x * torch.where(strong, 12.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op, dev = case["op"], dict(device="cuda")
    if op == "norm":
        rows, k = case["rows"], case["k"]
        s["x"] = (0.3 * _hidden(gen, rows, k)).to(_type(case["x"]))
        s["residual"] = _hidden(gen, rows, k).to(_type(case["res"])) if case["res"] else None
        s["weight"] = (1 + 0.2 * torch.randn(k, generator=gen, **dev)).to(torch.bfloat16)
        if case["train"]:
            s["dy"] = (0.1 * torch.randn(rows, k, generator=gen, **dev)).to(torch.bfloat16)
            s["dsum"] = (0.1 * torch.randn(rows, k, generator=gen, **dev)).to(_type(case["res"] or case["x"]))
    elif op == "lora":
        m, k, n, rank, adapters = (case[v] for v in ("m", "k", "n", "rank", "adapters"))
        s["x"] = _hidden(gen, m, k).to(torch.bfloat16)
        s["a"] = (torch.randn(adapters, rank, k, generator=gen, **dev) / math.sqrt(k)).to(torch.bfloat16)
        s["b"] = (torch.randn(adapters, n, rank, generator=gen, **dev) * (0.3 / math.sqrt(rank))).to(torch.bfloat16)
        s["scales"] = 0.5 + torch.rand(adapters, generator=gen, **dev)
        if case["prompts"]:   # runs of rows of one request each
            starts = torch.randint(m, (2 * adapters,), generator=gen, **dev).sort().values
            owner = torch.randint(-1, adapters, (2 * adapters + 1,), generator=gen, **dev)
            ids = owner[torch.searchsorted(starts, torch.arange(m, **dev), right=True)]
        else:                 # a row each; one in eight has none
            ids = torch.randint(adapters, (m,), generator=gen, **dev)
            ids = torch.where(torch.rand(m, generator=gen, **dev) < 0.125, torch.full_like(ids, -1), ids)
        ids[0] = ids[0].clamp_min(0)
        s["ids"] = ids.to(torch.int32)
        # the projection's output, which the adapters are added to
        s["rows"] = torch.zeros(m, _up(n, 8), dtype=_type(case["out"]), **dev)
        s["y"] = s["rows"][:, :n]
        s["y"].copy_(torch.randn(m, n, generator=gen, **dev))
    else:
        m, k, vocab = case["m"], case["k"], case["vocab"]
        s["w"] = (torch.randn(vocab, k, generator=gen, **dev) / math.sqrt(k)).to(torch.bfloat16)
        target = torch.randint(vocab, (m,), generator=gen, **dev)
        # as a trained model's last states: near the target's row, for half of the tokens very near
        near = torch.where(torch.rand(m, 1, generator=gen, **dev) < 0.5, 10.0, 3.0)
        s["x"] = (_hidden(gen, m, k) + near * s["w"][target].float()).to(torch.bfloat16)
        ignored = torch.rand(m, generator=gen, **dev) < 0.1   # padding and prompts
        ignored[0] = False
        s["targets"] = torch.where(ignored, torch.full_like(target, -100), target).to(torch.int32)
        if case["train"]:
            s["dloss"] = torch.ones(m, **dev) / (~ignored).sum()   # the mean over the tokens that count
    if own:
        _prepare_own(s)
    return s


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------

def _prepare_own(s):
    """Outputs, workspaces and the batch's grouping, which a user's program keeps."""
    import quantized_gemm_qg_amd as qg

    c, dev, bf16 = s["case"], dict(device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
    s["qg"], s["stream"], s["ws_bytes"] = qg, torch.cuda.current_stream().cuda_stream, 0
    s["type"] = {None: qg.O_BF16, "bf16": qg.O_BF16, "f32": qg.O_F32}
    if c["op"] == "norm":
        rows, k = c["rows"], c["k"]
        s["sum"] = torch.empty(rows, k, dtype=_type(c["res"]), **dev) if c["res"] else None
        s["y"] = torch.empty(rows, k, **bf16) if c["y"] else None
        s["q_type"] = {None: qg.A_BF16, "int8": qg.A_INT8_TOKEN, "fp8": qg.A_FP8_TOKEN, "fp8b": qg.A_FP8_BLOCK, "mxfp8": qg.A_MXFP8}[c["q"]]
        s["q"] = torch.empty(rows, _up(k, 16), dtype=torch.int8, **dev) if c["q"] else None
        s["q_scales"] = {None: lambda: None, "mxfp8": lambda: torch.empty(rows, k // 32, dtype=torch.uint8, **dev),
                         "fp8b": lambda: torch.empty(rows, -(-k // 128), **dev)}.get(c["q"], lambda: torch.empty(rows, **dev))()
        if c["train"]:
            s["dx"] = torch.empty_like(s["dsum"])
            s["dw"] = torch.empty(k, **bf16)
            s["ws_bytes"] = qg.rmsnorm_backward_workspace_size(rows, k)
    elif c["op"] == "lora":
        m, adapters = c["m"], c["adapters"]
        # grouped once per batch: every projection of every layer uses it
        s["sorted"], s["offsets"] = torch.empty(m, dtype=torch.int32, **dev), torch.empty(adapters + 1, dtype=torch.int32, **dev)
        sort_ws = torch.empty(_up(4 * (adapters + 1), 256), dtype=torch.uint8, **dev)
        qg.moe_sort(s["ids"], m, 1, adapters, s["sorted"], s["offsets"], sort_ws, sort_ws.numel(), s["stream"])
        s["ws_bytes"] = qg.lora_workspace_size(m, c["k"], c["n"], adapters, c["rank"])
    else:
        m, k, vocab = c["m"], c["k"], c["vocab"]
        s["loss"], s["lse"] = torch.empty(m, **dev), torch.empty(m, **dev)
        s["ws_bytes"] = qg.linear_xent_workspace_size(m, k, vocab)
        if c["train"]:
            s["dx"], s["dw"] = torch.empty(m, k, **bf16), torch.empty(vocab, k, **bf16)
            s["ws_bytes"] = max(s["ws_bytes"], qg.linear_xent_backward_workspace_size(m, k, vocab))
    s["ws"] = torch.zeros(max(s["ws_bytes"], 1), dtype=torch.uint8, **dev)


def _run_own(s):
    qg, c, stream, ws = s["qg"], s["case"], s["stream"], (s["ws"], s["ws_bytes"])
    if c["op"] == "norm":
        rows, k = c["rows"], c["k"]
        qg.rmsnorm(s["x"], s["type"][c["x"]], k, s["weight"], _EPS, rows, k, residual=s["residual"], res_type=s["type"][c["res"]], ldr=k,
                   sum=s["sum"], lds=k, y=s["y"], ldy=k, q_type=s["q_type"], q=s["q"], ldq=_up(k, 16), q_scales=s["q_scales"],
                   stream=stream)
        out = dict(sum=s["sum"], y=s["y"])
        if c["train"]:
            total, kind = (s["sum"], c["res"]) if c["res"] else (s["x"], c["x"])
            qg.rmsnorm_backward(total, s["type"][kind], k, s["weight"], _EPS, rows, k, s["dy"], k, s["dx"], k, s["dw"], qg.O_BF16, *ws,
                                dsum=s["dsum"], ldds=k, stream=stream)
            out.update(dx=s["dx"], dw=s["dw"])
        if c["q"]:
            q = s["q"][:, :k]
            out["q"] = q.to(torch.bfloat16) if c["q"] == "int8" else q.view(torch.float8_e4m3fn)
            out["q_scales"] = s["q_scales"].view(torch.float8_e8m0fnu) if c["q"] == "mxfp8" else s["q_scales"]
        return out
    if c["op"] == "lora":
        k, n, rank = c["k"], c["n"], c["rank"]
        qg.lora(s["x"], k, s["a"], k, s["b"], rank, s["scales"], c["adapters"], rank, s["sorted"], s["offsets"], c["m"], k, n, s["rows"],
                s["type"][c["out"]], s["rows"].stride(0), *ws, stream=stream)
        return s["y"]
    m, k, vocab = c["m"], c["k"], c["vocab"]
    qg.linear_xent(s["x"], k, s["w"], k, m, k, vocab, s["targets"], 1.0, s["loss"], s["lse"], *ws, stream=stream)
    out = dict(loss=s["loss"], lse=s["lse"])
    if c["train"]:
        qg.linear_xent_backward(s["x"], k, s["w"], k, m, k, vocab, s["targets"], 1.0, s["lse"], s["dloss"], s["dx"], k, s["dw"],
                                qg.O_BF16, k, *ws, stream=stream)
        out.update(dx=s["dx"], dw=s["dw"])
    return out


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _quantized(y, kind):
    """Codes (as the values they are) and scales of fp32 rows."""
    rows, k = y.shape
    if kind == "mxfp8":
        most = y.reshape(rows, k // 32, 32).abs().amax(2)
        exponent = torch.where(most > 0, torch.frexp(most).exponent - 9, torch.zeros_like(most, dtype=torch.int32)).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(most), exponent)
        q = (y.reshape(rows, k // 32, 32) / scale.unsqueeze(2)).clamp(-448, 448).reshape(rows, k)
        return q.to(torch.float8_e4m3fn), (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    width = 128 if kind == "fp8b" else k
    blocks = torch.nn.functional.pad(y, (0, -k % width)).reshape(rows, -1, width)
    top = 127.0 if kind == "int8" else 448.0
    most = blocks.abs().amax(2)
    scale = torch.where(most > 0, most / torch.full_like(most, top), torch.ones_like(most))
    q = (blocks / scale.unsqueeze(2)).clamp(-top, top).reshape(rows, -1)[:, :k]
    q = torch.round(q).to(torch.bfloat16) if kind == "int8" else q.to(torch.float8_e4m3fn)
    return q, scale if kind == "fp8b" else scale.squeeze(1)


def _plain_norm(s):
    c = s["case"]
    total, out = s["x"].float(), {}
    if c["res"]:
        out["sum"] = (total + s["residual"].float()).to(_type(c["res"]))
        total = out["sum"].float()
    w = s["weight"].float()
    r = 1 / torch.sqrt((total * total).mean(1, keepdim=True) + _EPS)
    y = total * r * w
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    if c["q"]:
        out["q"], out["q_scales"] = _quantized(y, c["q"])
    if c["train"]:
        dy, unit = s["dy"].float(), total * r
        g = dy * w
        out["dx"] = (r * (g - unit * (g * unit).mean(1, keepdim=True)) + s["dsum"].float()).to(s["dsum"].dtype)
        out["dw"] = (dy * unit).sum(0).to(torch.bfloat16)
    return out


def _plain_lora(s):
    """All adapters' low-rank products at once, those of other adapters' rows replaced by zeros."""
    c = s["case"]
    rank, adapters = c["rank"], c["adapters"]
    t = s["x"].float() @ s["a"].float().reshape(adapters * rank, c["k"]).T
    mine = (s["ids"].unsqueeze(1) == torch.arange(adapters, device="cuda")) * s["scales"]
    t = t * mine.repeat_interleave(rank, 1)
    y = s["y"].float() + t @ s["b"].float().transpose(1, 2).reshape(adapters * rank, c["n"])
    return s["y"].copy_(y.to(s["y"].dtype))


def _plain_xent(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, keepdim=True)
    lse = most + torch.log(total)
    counts = s["targets"].unsqueeze(1) >= 0
    at = s["targets"].long().clamp_min(0).unsqueeze(1)
    loss = torch.where(counts, lse - z.gather(1, at), torch.zeros_like(lse)).squeeze(1)
    out = dict(loss=loss, lse=lse.squeeze(1))
    if c["train"]:
        d = torch.where(counts, s["dloss"].unsqueeze(1), torch.zeros_like(lse))
        e.mul_(d / total).scatter_add_(1, at, -d)
        out.update(dx=(e @ w).to(torch.bfloat16), dw=(e.T @ x).to(torch.bfloat16))
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "lora": _plain_lora, "xent": _plain_xent}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c, el = case, {None: 0, "bf16": 2, "f32": 4}
    if c["op"] == "norm":
        values, per = c["rows"] * c["k"], el[c["x"]] + 2 * el[c["res"]] + 2 * c["y"] + (c["q"] is not None)
        scales = {None: 0, "int8": 4, "fp8": 4, "fp8b": 4 * -(-c["k"] // 128), "mxfp8": c["k"] // 32}[c["q"]] * c["rows"]
        if c["train"]:   # dy, dsum and dx, the sum once more, dw
            kind = el[c["res"] or c["x"]]
            return dict(bytes=values * (per + 2 + 3 * kind) + 6 * c["k"], flops=20 * values)
        return dict(bytes=values * per + scales + 2 * c["k"], flops=6 * values)
    if c["op"] == "lora":
        m, k, n, rank = c["m"], c["k"], c["n"], c["rank"]
        used = min(c["adapters"], m)
        rows = m if c["prompts"] else max(1, m * 7 // 8)
        return dict(bytes=rows * (2 * k + 2 * n * el[c["out"]]) + 2 * used * rank * (k + n), flops=2 * rows * rank * (k + n))
    m, k, vocab = c["m"], c["k"], c["vocab"]
    if c["train"]:
        return dict(bytes=4 * (m * k + vocab * k) + 16 * m, flops=6 * m * k * vocab)
    return dict(bytes=2 * (m * k + vocab * k) + 12 * m, flops=2 * m * k * vocab)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _norm64, "lora": _lora64, "xent": _xent64}[case["op"]](s)


def _norm64(s):
    c, d = s["case"], torch.float64
    out, v = {}, s["x"].to(d)
    if c["res"]:
        out["sum"] = v + s["residual"].to(d)
        v = out["sum"].to(_type(c["res"])).to(d)   # the norm is that of the sum as it is kept
    w, k = s["weight"].to(d)[None], c["k"]
    r = torch.rsqrt(v.square().sum(1, keepdim=True) / k + _EPS)
    y = v * (r * w)
    if c["y"]:
        out["y"] = y
    if c["train"]:
        dy = s["dy"].to(d)
        inner = (dy * w * v).sum(1, keepdim=True) / k
        out["dx"] = dy * w * r - v * r.pow(3) * inner + s["dsum"].to(d)
        out["dw"] = (dy * v).mul_(r).sum(0)
    if c["q"]:
        size = {"mxfp8": 32, "fp8b": 128}.get(c["q"], k)
        wide = torch.zeros(c["rows"], _up(k, size), dtype=d, device="cuda")
        wide[:, :k] = y
        p = wide.view(-1, size)
        most = p.abs().amax(1)
        if c["q"] == "mxfp8":
            step = torch.exp2(torch.floor(torch.log2(most)) - 8)
        else:
            step = most / (127 if c["q"] == "int8" else 448)
        step = torch.where(most > 0, step, torch.ones_like(step))
        # the values that the e4m3 codes are the nearest of; int8 codes are whole numbers, a tie of
        # which the last bit of a scale decides
        code = (p / step[:, None]).clamp(-448, 448).view(c["rows"], -1)[:, :k]
        out["q"] = None if c["q"] == "int8" else code
        out["q_scales"] = step.view(c["rows"], -1) if c["q"] in ("mxfp8", "fp8b") else step
    return out


def _lora64(s):
    y, d = s["y"].to(torch.float64), torch.float64
    ids = s["ids"].cpu()
    for a in sorted(set(ids.tolist()) - {-1}):
        at = (ids == a).nonzero()[:, 0].cuda()
        low = torch.mm(s["x"][at].to(d), s["a"][a].to(d).t().contiguous())
        y[at] += s["scales"][a].to(d) * torch.mm(low, s["b"][a].to(d).t().contiguous())
    return y


def _xent64(s):
    c, d = s["case"], torch.float64
    x, w = s["x"].to(d), s["w"].to(d)
    z = torch.mm(x, w.t())
    lse = torch.logsumexp(z, 1)
    t = s["targets"].long()
    rows = (t >= 0).nonzero()[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, t[rows]]
    out = dict(loss=loss, lse=lse)
    if c["train"]:
        z.sub_(lse[:, None]).exp_()
        z[rows, t[rows]] -= 1
        weight = torch.zeros_like(lse)
        weight[rows] = s["dloss"][rows].to(d)
        z *= weight[:, None]
        out.update(dx=torch.mm(z, w), dw=torch.mm(z.t(), x))
    return out
