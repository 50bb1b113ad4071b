"""GPU tests of the token log probabilities (entropy, rank, alternatives) and
of the logits' gradient, against float64.

Ids and ranks are exact.  Tolerances: z is one fp32 product, the exponential
within a few ulps of its argument's size, and the sums' terms are non-negative
(at most V / 256 + 64 roundings on the way of one), so with Z the largest |z| of
the row's unmasked logits relative to its maximum and scale,
|logp - exact| <= (V / 256 + 64) 2^-24 + 2^-21 (1 + Z); the entropy's sum has
terms up to log V times as large."""
import math

import pytest
import torch

import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
D = torch.float64
INF = math.inf


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def place(l, dtype, pad, shift):
    """The logits on the device in rows of pitch vocab + pad, `shift` elements
    into a larger buffer, NaN around them."""
    rows, vocab = l.shape
    flat = torch.full((rows * (vocab + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    v = flat[shift:shift + rows * (vocab + pad)].view(rows, vocab + pad)
    v[:, :vocab] = l.to(dtype).cuda()
    return v


def forward(l, ltype, tokens, scale, top):
    rows, vocab, ld = l.shape[0], l.vocab, l.stride(0)
    o = dict(logp=torch.empty(rows), entropy=torch.empty(rows), stats=torch.empty(rows, 2), rank=torch.empty(rows, dtype=torch.int32),
             top_ids=torch.empty(rows, max(top, 1), dtype=torch.int32), top_logp=torch.empty(rows, max(top, 1)))
    o = {n: t.cuda() for n, t in o.items()}
    wsb = qg.token_logprobs_workspace_size(rows, vocab, top)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        qg.token_logprobs(l, ltype, rows, vocab, ld, tokens, scale, top, o["logp"], o["entropy"], o["stats"], o["rank"],
                          o["top_ids"] if top else None, o["top_logp"] if top else None, ws, wsb)
    return o


def reference(l, tokens, scale):
    """float64 log probabilities, entropy and rank of the (already rounded) logits."""
    z = l.to(D) * scale
    lse = torch.logsumexp(z, 1)
    logq = torch.where(z == -INF, z, z - lse[:, None])
    logq = torch.where(logq < torch.finfo(torch.float32).min, torch.tensor(-INF, dtype=D), logq)   # no fp32 number
    ent = torch.special.entr(torch.exp(logq)).sum(1)
    r = torch.arange(len(l))
    t = tokens.long()
    return logq, logq[r, t], ent, (l > l[r, t][:, None]).sum(1)


def alternatives(l, top):
    """Ids of the largest logits, equal ones by id; -1 where there is none."""
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top]
    ids = torch.where(l.gather(1, ids) == -INF, torch.full_like(ids, -1), ids)
    return torch.nn.functional.pad(ids, (0, top - ids.shape[1]), value=-1)


def tolerance(l, scale):
    z = torch.where(l == -INF, torch.zeros_like(l), l).to(D) * scale
    return (l.shape[1] / 256 + 64) * U32 + 2.0 ** -21 * (1 + 2 * z.abs().amax(1))


def make(kind, rows, vocab, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    l = torch.randn(rows, vocab, generator=gen) * 3
    if kind == "masked":
        l[torch.rand(rows, vocab, generator=gen) < 0.7] = -INF
        l[rows // 2] = -INF
    elif kind == "ties":
        l = torch.randint(-2, 3, (rows, vocab), generator=gen).float() * 0.5   # +0 and -0 among them
        l[torch.rand(rows, vocab, generator=gen) < 0.3] *= -1
    elif kind == "equal":
        l[:] = 1.25
    elif kind == "lowest":   # masks of the type's lowest value
        l[torch.rand(rows, vocab, generator=gen) < 0.5] = torch.finfo(dtype).min
        l[0] = torch.finfo(dtype).min
    elif kind == "sorted":
        l = l.sort(1, descending=bool(seed % 2)).values
    elif kind == "strided":  # every large logit in one residue class of the ids
        l[:, 5::2048] += 40
        l[:, 7::512] += 20
    l = l.to(dtype)
    tok = torch.randint(vocab, (rows,), generator=gen, dtype=torch.int32)
    tok[::2] = l.float().argmax(1).to(torch.int32)[::2]
    return l, tok


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 64), (2, 1000), (1, 32768), (4, 32769), (3, 100003), (1, 131072), (700, 300), (40, 5000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["plain", "masked", "ties", "equal", "lowest", "sorted", "strided"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_forward(rows, vocab, kind, dtype):
    print(f"logprobs rows={rows} vocab={vocab} {kind} {dtype}", flush=True)
    l, tok = make(kind, rows, vocab, dtype, rows + vocab)
    lf = l.float()
    ltype = qg.O_F32 if dtype == torch.float32 else qg.O_BF16
    for scale, top, pad, shift in ((1.0, 20, 0, 0), (0.7, 32, 5, 1), (2.0, 0, 8, 0), (1.0, 1, 3, 3)):
        d = place(l, dtype, pad, shift)
        d.vocab = vocab
        o = {n: t.cpu() for n, t in forward(d, ltype, tok.cuda(), scale, top).items()}
        logq, logp, ent, rank = reference(lf, tok, torch.tensor(scale, dtype=torch.float32).item())
        tol = tolerance(lf, scale)
        assert torch.equal(o["rank"].long(), rank)
        dead = (lf == -INF).all(1)
        assert (o["logp"][logp == -INF] == -INF).all() and (o["logp"][dead] == -INF).all()
        live = (logp > -INF) & ~dead
        assert ((o["logp"].to(D) - logp).abs()[live] <= tol[live]).all()
        ent = torch.where(dead, torch.zeros_like(ent), ent)
        assert ((o["entropy"].to(D) - ent).abs() <= tol * (2 + math.log(vocab))).all()
        if top:
            ids = alternatives(lf, top)
            assert torch.equal(o["top_ids"].long(), ids)
            want = torch.where(ids < 0, torch.full(ids.shape, -INF, dtype=D), logq.gather(1, ids.clamp(min=0)))
            got = o["top_logp"].to(D)
            assert torch.equal(got == -INF, want == -INF)
            fin = want > -INF
            assert ((got - want)[fin].abs() <= tol[:, None].expand_as(got)[fin]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,kind", [(1024, 300, "plain"), (1024, 300, "equal"), (1100, 4099, "plain"), (1100, 4099, "masked"),
                                             (1100, 4099, "ties"), (1100, 4099, "sorted"), (1025, 2500, "lowest"),
                                             (1024, 9001, "strided"), (20, 6201, "ties"), (20, 12001, "sorted"), (800, 17000, "plain")])
def test_forward_of_rows_that_a_chunk_holds(rows, vocab, kind, dtype):
    """Many short rows (a wave each), few of them (a workgroup each), and rows of
    a chunk and a piece of the next."""
    test_forward(rows, vocab, kind, dtype)


def test_repeated_calls_give_the_same_bits():
    l, tok = make("plain", 3, 131072, torch.bfloat16, 1)
    d = place(l, torch.bfloat16, 0, 0)
    d.vocab = 131072
    a = forward(d, qg.O_BF16, tok.cuda(), 1.0, 8)
    for _ in range(5):
        b = forward(d, qg.O_BF16, tok.cuda(), 1.0, 8)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_nan_and_infinities():
    l, tok = make("plain", 4, 70000, torch.float32, 3)
    l[0, 123] = float("nan")
    l[1, 69999] = INF
    l[2, 5] = -INF
    d = place(l, torch.float32, 0, 0)
    d.vocab = 70000
    o = {n: t.cpu() for n, t in forward(d, qg.O_F32, tok.cuda(), 1.0, 4).items()}
    for n in ("logp", "entropy"):
        assert torch.isnan(o[n][:2]).all() and torch.isfinite(o[n][2:]).all()
    assert torch.isnan(o["top_logp"][:2]).all()
    clean = torch.where(torch.isnan(l), torch.tensor(-INF), l)
    assert torch.equal(o["top_ids"].long(), alternatives(clean, 4))


def test_tokens_outside_the_vocabulary():
    l, tok = make("plain", 3, 999, torch.float32, 4)
    tok[0], tok[2] = -1, 999
    d = place(l, torch.float32, 1, 0)
    d.vocab = 999
    o = {n: t.cpu() for n, t in forward(d, qg.O_F32, tok.cuda(), 1.0, 2).items()}
    assert torch.isnan(o["logp"][[0, 2]]).all() and torch.isfinite(o["logp"][1])
    assert o["rank"][0] == o["rank"][2] == -1
    dl = torch.empty(3, 999, device="cuda")
    one = torch.ones(3, device="cuda")
    o = forward(d, qg.O_F32, tok.cuda(), 1.0, 0)
    qg.token_logprobs_backward(d, qg.O_F32, 3, 999, 1000, tok.cuda(), 1.0, o["stats"], o["entropy"], one, None, dl, 999)
    assert (dl[[0, 2]] == 0).all() and (dl[1] != 0).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["plain", "masked", "lowest"])
@pytest.mark.parametrize("rows,vocab,pad,shift", [(1, 1, 0, 0), (3, 7, 1, 1), (2, 1000, 0, 0), (4, 32769, 7, 0), (1, 131072, 0, 0),
                                                  (300, 257, 3, 0)])
def test_backward(rows, vocab, pad, shift, kind, dtype):
    print(f"logprobs backward rows={rows} vocab={vocab} {kind} {dtype}", flush=True)
    l, tok = make(kind, rows, vocab, dtype, rows + vocab)
    if kind == "masked" and rows > 1:   # a masked token
        tok[0] = 0
        l[0, 0] = -INF
    ltype = qg.O_F32 if dtype == torch.float32 else qg.O_BF16
    d = place(l, dtype, pad, shift)
    d.vocab = vocab
    scale = 0.75
    o = forward(d, ltype, tok.cuda(), scale, 0)
    gen = torch.Generator().manual_seed(9)
    g, e = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
    logq, _, ent, _ = reference(l.float(), tok, scale)
    p = torch.exp(logq)
    dead = (l == -INF).all(1)
    hit = torch.zeros(rows, vocab, dtype=D)
    hit[torch.arange(rows), tok.long()] = 1
    inner = torch.where(p > 0, p * (logq + ent[:, None]), torch.zeros_like(p))
    for dlogp, dent in ((g, e), (g, None), (None, e)):
        want = torch.zeros(rows, vocab, dtype=D)
        if dlogp is not None:
            want += dlogp.to(D)[:, None] * (hit - p)
        if dent is not None:
            want -= dent.to(D)[:, None] * inner
        want[dead] = 0
        want *= scale
        dl = torch.full((rows + 1, vocab + 3), 7.0, dtype=dtype, device="cuda")
        qg.token_logprobs_backward(d, ltype, rows, vocab, d.stride(0), tok.cuda(), scale, o["stats"], o["entropy"],
                                   None if dlogp is None else dlogp.cuda(), None if dent is None else dent.cuda(), dl, vocab + 3)
        assert (dl[rows:] == 7).all() and (dl[:, vocab:] == 7).all()
        got = dl[:rows, :vocab].cpu().to(D)
        # p is off by its logarithm's error
        tol = (tolerance(l.float(), scale) * (3 + math.log(vocab)))[:, None]
        parts = (g.abs().to(D)[:, None] + e.abs().to(D)[:, None] * (1 + torch.where(p > 0, logq.abs(), p) + ent[:, None].abs()))
        bound = scale * (p * parts * tol + (hit * g.to(D)[:, None]).abs() * 4 * U32) + (U16 if dtype == torch.bfloat16 else 2 * U32) * want.abs()
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= bound * (1 + U16) + 1e-37).all()
    # in place
    ref = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    args = (tok.cuda(), scale, o["stats"], o["entropy"], g.cuda(), e.cuda())
    qg.token_logprobs_backward(d, ltype, rows, vocab, d.stride(0), *args, ref, vocab)
    qg.token_logprobs_backward(d, ltype, rows, vocab, d.stride(0), *args, d, d.stride(0))
    assert torch.equal(d[:, :vocab], ref)


def test_backward_of_a_gradient_larger_than_the_caches():
    test_backward(170, 100003, 0, 0, "masked", torch.bfloat16)
    test_backward(70, 131072, 5, 1, "plain", torch.float32)


def test_gradient_against_differences():
    l, tok = make("plain", 3, 50, torch.float32, 8)
    scale = 1.5
    d = place(l, torch.float32, 0, 0)
    d.vocab = 50
    o = forward(d, qg.O_F32, tok.cuda(), scale, 0)
    g, e = torch.tensor([1.0, -2.0, 0.5]), torch.tensor([0.3, 0.1, -1.0])
    dl = torch.empty(3, 50, device="cuda")
    qg.token_logprobs_backward(d, qg.O_F32, 3, 50, 50, tok.cuda(), scale, o["stats"], o["entropy"], g.cuda(), e.cuda(), dl, 50)

    def loss(x):
        logq = torch.log_softmax(x * scale, 1)
        return (g.to(D) * logq[torch.arange(3), tok.long()]).sum() + (e.to(D) * -(logq.exp() * logq).sum(1)).sum()

    x, eps = l.to(D), 1e-5
    for r in range(3):
        for v in range(0, 50, 7):
            at = torch.zeros(3, 50, dtype=D)
            at[r, v] = eps
            slope = (loss(x + at) - loss(x - at)) / (2 * eps)
            # differences are exact to eps^2 and 2^-53 / eps
            assert abs(dl[r, v].item() - slope) <= 1e-8 + 2.0 ** -17 * scale * (g[r].abs() + e[r].abs() * 5)


def test_graph_replays():
    l, tok = make("plain", 2, 100003, torch.bfloat16, 1)
    d = place(l, torch.bfloat16, 5, 0)
    tok = tok.cuda()
    out = [torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")]
    wsb = qg.token_logprobs_workspace_size(2, 100003, 5)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    run = lambda: qg.token_logprobs(d, qg.O_BF16, 2, 100003, d.stride(0), tok, 1.0, 5, out[0], out[1], None, None, out[2], None, ws, wsb)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(3):
        d[:, :100003] = torch.randn(2, 100003, device="cuda").to(torch.bfloat16)
        run()
        eager = [t.clone() for t in out]
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))


@pytest.mark.parametrize("rows,vocab,kind,dtype", [
    (40, 131072, "plain", torch.bfloat16), (40, 131072, "masked", torch.bfloat16), (40, 131072, "ties", torch.bfloat16),
    (40, 131072, "strided", torch.bfloat16), (20, 100003, "plain", torch.float32), (20, 100003, "masked", torch.float32),
    (20, 100003, "ties", torch.float32), (20, 100003, "strided", torch.float32),
    (385, 33000, "plain", torch.bfloat16), (260, 25001, "sorted", torch.float32)])
def test_forward_of_tens_and_hundreds_of_long_rows(rows, vocab, kind, dtype):
    """Rows that a few workgroups share in large chunks: one chunk each, or a
    chunk and a piece of the next."""
    test_forward(rows, vocab, kind, dtype)


@pytest.mark.parametrize("kind", ["masked", "ties"])
def test_forward_of_rows_that_four_units_a_thread_hold(kind):
    test_forward(20, 3001, kind, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,pad,shift", [(1, 5, 0, 0), (5, 64, 1, 1), (300, 9001, 0, 0), (1100, 4099, 5, 1), (1, 131072, 0, 0),
                                                  (3, 100003, 5, 1), (40, 131072, 0, 0), (40, 131072, 3, 3), (800, 17000, 0, 0)])
def test_forward_without_statistics(rows, vocab, pad, shift, dtype):
    """The same bits as with them."""
    print(f"logprobs without stats rows={rows} vocab={vocab} {dtype}", flush=True)
    l, tok = make("masked", rows, vocab, dtype, rows + vocab)
    d = place(l, dtype, pad, shift)
    d.vocab = vocab
    ltype = qg.O_F32 if dtype == torch.float32 else qg.O_BF16
    for top in (0, 20):
        o = forward(d, ltype, tok.cuda(), 0.7, top)
        n = {name: torch.full_like(t, 7) for name, t in o.items()}
        wsb = qg.token_logprobs_workspace_size(rows, vocab, top)
        ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        qg.token_logprobs(d, ltype, rows, vocab, d.stride(0), tok.cuda(), 0.7, top, n["logp"], n["entropy"], None, n["rank"],
                          n["top_ids"] if top else None, n["top_logp"] if top else None, ws, wsb)
        for name in ("logp", "entropy", "rank") + (("top_ids", "top_logp") if top else ()):
            assert torch.equal(n[name], o[name]), name


@pytest.mark.parametrize("rows,vocab,dtype", [(520, 131072, torch.float32), (1030, 131073, torch.bfloat16), (9000, 16001, torch.bfloat16)])
def test_logits_read_past_the_caches(rows, vocab, dtype):
    """More than 256 MB of logits and no statistics: the same bits as with them."""
    print(f"logprobs past the caches rows={rows} vocab={vocab} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    l = torch.empty(rows, vocab + 3, dtype=dtype, device="cuda")
    assert rows * vocab * l.element_size() > 256 << 20
    l[:] = torch.randn(rows, vocab + 3, generator=gen, device="cuda")
    d = l[:, :vocab]
    d.vocab = vocab
    tok = torch.randint(vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    ltype = qg.O_F32 if dtype == torch.float32 else qg.O_BF16
    o = forward(d, ltype, tok, 0.7, 20)
    n = {name: torch.full_like(t, 7) for name, t in o.items()}
    wsb = qg.token_logprobs_workspace_size(rows, vocab, 20)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    qg.token_logprobs(d, ltype, rows, vocab, vocab + 3, tok, 0.7, 20, n["logp"], n["entropy"], None, n["rank"], n["top_ids"],
                      n["top_logp"], ws, wsb)
    for name in ("logp", "entropy", "rank", "top_ids", "top_logp"):
        assert torch.equal(n[name], o[name]), name
    # and a few rows against 64 bits
    some = torch.arange(0, rows, rows // 5)
    logq, logp, ent, rank = reference(d[some.cuda()].cpu().float(), tok.cpu()[some], torch.tensor(0.7).item())
    tol = tolerance(d[some.cuda()].cpu().float(), 0.7)
    assert ((n["logp"].cpu().to(D)[some] - logp).abs() <= tol).all() and torch.equal(n["rank"].cpu().long()[some], rank)
    assert ((n["entropy"].cpu().to(D)[some] - ent).abs() <= tol * (2 + math.log(vocab))).all()
    assert torch.equal(n["top_ids"].cpu().long()[some], alternatives(d[some.cuda()].cpu().float(), 20))
