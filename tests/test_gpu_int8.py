"""GPU tests of the int8 products (per-token and per-channel scales), their
quantizer and the gated form, against the definitions in 64 bits.

The codes and the scales are compared exactly.  The integer sum is exact, so a
fp32 output differs from the real value by three fp32 roundings (the sum's
conversion and two products), a bf16 one by one rounding more; the gated form
adds the activation's error, bounded below by its largest condition on g."""
import math

import numpy as np
import pytest
import torch

import quantized_gemm_qg_amd as qg
from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8   # unit roundoffs of fp32 and bf16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def quantize_ref(x):
    """Codes and scales of bf16 rows (given as float32) by definition."""
    most = np.abs(x).max(1).astype(np.float32) if x.shape[1] else np.zeros(len(x), np.float32)
    s = np.where(most > 0, most / np.float32(127), np.float32(1)).astype(np.float32)
    return np.rint((x / s[:, None]).astype(np.float32)).astype(np.int8), s


class Int8Layer:
    def __init__(self, n, k, seed=0):
        r = np.random.default_rng(seed)
        self.n, self.k = n, k
        self.codes = r.integers(-128, 128, (n, k), dtype=np.int8)
        self.scales = (r.random(n, dtype=np.float32) + 0.1) / 1000
        self.desc = qg.layer_desc(qg.W_INT8, n, k, k, atype=qg.A_INT8_TOKEN)
        self.buf = torch.empty(qg.packed_size(self.desc), dtype=torch.uint8, device="cuda")
        self.w = qg.preprocess(self.desc, self.codes, self.scales, None, self.buf)

    def product(self, q, s):
        """Exact y and the weights' float64 form."""
        acc = q.astype(np.float64) @ self.codes.astype(np.float64).T
        return acc * s.astype(np.float64)[:, None] * self.scales.astype(np.float64)[None]


def rows(m, k, seed, spread=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((m, k)).astype(np.float32)
    if spread:
        x *= np.exp(r.standard_normal((m, 1))).astype(np.float32)
    t = torch.from_numpy(x).to(torch.bfloat16)
    return t, t.float().numpy()


def out_buffer(m, n, otype, pad):
    ld = n + pad
    ld += ld % 2
    t = torch.full((m + 2, ld), 7.0, dtype=torch.float32 if otype == qg.O_F32 else torch.bfloat16, device="cuda")
    return t, ld


def untouched(t, m, n):
    assert (t[m:] == 7).all() and (t[:m, n:] == 7).all()


def check(y, ref, otype, extra=0.0):
    y = y.double().cpu().numpy()
    tol = 3.1 * U32 + (U16 if otype == qg.O_BF16 else 0)
    assert (np.abs(y - ref) <= tol * np.abs(ref) + extra + 1e-38).all()


@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (5, 4096), (2, 14336), (300, 1032), (2050, 264)])
def test_quantize_int8(m, k):
    x, xf = rows(m, k, 3 * m + k)
    xf[m // 2] = 0
    xf[0, :min(k, 8)] = [0.5, -0.5, 127, 63.5, -63.5, 1.5, -2.5, 0][:min(k, 8)]  # ties, with the scale 1 where 127 is the largest
    xf[0] = np.clip(xf[0], -127, 127)
    x = torch.from_numpy(xf).to(torch.bfloat16)
    xf = x.float().numpy()
    ldx, ldq = k + 8, k + 24
    xd = torch.full((m, ldx), float("nan"), dtype=torch.bfloat16, device="cuda")
    xd[:, :k] = x.cuda()
    q = torch.full((m + 1, ldq), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(m, dtype=torch.float32, device="cuda")
    qg.quantize_int8(xd, m, k, ldx, q, ldq, s)
    cq, cs = quantize_ref(xf)
    assert (s.cpu().numpy() == cs).all()
    assert (q[:m, :k].cpu().numpy() == cq).all()
    assert (q[m:] == 99).all() and (q[:m, k:] == 99).all()


SHAPES = [
    (1, 1, 32), (1, 17, 4096), (1, 256, 14336), (2, 100, 160), (4, 64, 1056), (5, 333, 416), (16, 130, 2080), (17, 96, 96),
    (23, 500, 3200), (33, 129, 224), (64, 320, 1024), (65, 255, 640), (100, 1000, 544), (128, 128, 128), (200, 384, 7168),
    (255, 257, 288), (513, 300, 352), (1030, 515, 192), (3000, 140, 64),
]


@pytest.mark.parametrize("otype", [qg.O_F32, qg.O_BF16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_matches_64_bits(m, n, k, otype):
    print(f"int8 product m={m} n={n} k={k} otype={otype}", flush=True)
    lay = Int8Layer(n, k, seed=n + k)
    x, xf = rows(m, k, m)
    cq, cs = quantize_ref(xf)
    ref = lay.product(cq, cs)
    # quantized inside the call, from rows with a longer pitch
    xd = torch.full((m, k + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    xd[:, :k] = x.cuda()
    y, ld = out_buffer(m, n, otype, 2)
    wsb = qg.gemm_workspace_size_ex(lay.w, m, qg.GEMM_QUANTIZE_X)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    for _ in range(2):  # the workspace serves call after call
        qg.gemm_ex(lay.w, xd, None, m, k + 8, y, otype, ld, ws, wsb, qg.GEMM_QUANTIZE_X)
        check(y[:m, :n], ref, otype)
        untouched(y, m, n)
    # on quantized rows: the same bits, and bit for bit the same whatever the batch
    q, s = torch.from_numpy(cq).cuda(), torch.from_numpy(cs).cuda()
    y2, _ = out_buffer(m, n, otype, 2)
    wsb = qg.gemm_workspace_size(lay.w, m)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    qg.gemm(lay.w, q, s, m, k, y2, otype, ld, ws, wsb)
    assert torch.equal(y, y2)
    one, _ = out_buffer(1, n, otype, 2)
    wsb = qg.gemm_workspace_size_ex(lay.w, 1, qg.GEMM_BATCH_INVARIANT)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    qg.gemm_ex(lay.w, q[m - 1:], s[m - 1:], 1, k, one, otype, ld, ws, wsb, qg.GEMM_BATCH_INVARIANT)
    assert torch.equal(one[0], y[m - 1])


def test_extreme_codes_reach_the_whole_int32_range():
    n, k, m = 48, 130816, 5   # k * 128 * 128 = 2143289344 < 2^31
    lay = Int8Layer(n, 64, 1)
    lay.n, lay.k = n, k
    lay.codes = np.full((n, k), -128, np.int8)
    lay.codes[1::2] = 127
    lay.scales = np.full(n, 2.0 ** -20, np.float32)
    lay.desc = qg.layer_desc(qg.W_INT8, n, k, k, atype=qg.A_INT8_TOKEN)
    lay.buf = torch.empty(qg.packed_size(lay.desc), dtype=torch.uint8, device="cuda")
    lay.w = qg.preprocess(lay.desc, lay.codes, lay.scales, None, lay.buf)
    for m in (1, 5, 40):
        q = np.full((m, k), -128, np.int8)
        s = np.ones(m, np.float32)
        y, ld = out_buffer(m, n, qg.O_F32, 0)
        wsb = qg.gemm_workspace_size(lay.w, m)
        ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        qg.gemm(lay.w, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), m, k, y, qg.O_F32, ld, ws, wsb)
        check(y[:m, :n], lay.product(q, s), qg.O_F32)


def act64(g, act):
    if act == qg.ACT_SILU:
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


@pytest.mark.parametrize("act", [qg.ACT_SILU, qg.ACT_GELU_TANH])
@pytest.mark.parametrize("m,inter,k", [(1, 1, 32), (1, 300, 4096), (3, 17, 96), (7, 128, 544), (16, 65, 1056), (20, 64, 128),
                                       (40, 1000, 256), (130, 333, 416), (300, 129, 2080), (1025, 80, 96)])
def test_gated_matches_64_bits(m, inter, k, act):
    print(f"int8 gated m={m} inter={inter} k={k} act={act}", flush=True)
    lay = Int8Layer(2 * inter, k, seed=inter)
    lay_scale = 3.0 / (math.sqrt(k) * 74 * lay.scales.mean())   # g of a few units
    x, xf = rows(m, k, m + 1, spread=False)
    cq, cs = quantize_ref(xf)
    cs2 = (cs * np.float32(lay_scale)).astype(np.float32)
    gu = lay.product(cq, cs2)
    g, u = gu[:, :inter], gu[:, inter:]
    ref = act64(g, act) * u
    # fp32 activation: a few ulps of its parts, of size at most 1 + |g|
    extra = 2.0 ** -20 * (1 + np.abs(g)) * np.abs(u)
    q, s = torch.from_numpy(cq).cuda(), torch.from_numpy(cs2).cuda()
    for otype in (qg.O_F32, qg.O_BF16):
        h, ld = out_buffer(m, inter, otype, 4)
        wsb = qg.gated_gemm_workspace_size(lay.w, m)
        ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        qg.gated_gemm(lay.w, q, s, m, k, h, otype, ld, act, ws, wsb)
        check(h[:m, :inter], ref, otype, extra)
        untouched(h, m, inter)
    # quantized inside the call: the same as quantized before it
    xd = x.cuda()
    qs = torch.empty(m, dtype=torch.float32, device="cuda")
    qg.quantize_int8(xd, m, k, k, q, k, qs)
    wsb = qg.gated_gemm_workspace_size(lay.w, m, qg.GEMM_QUANTIZE_X)
    ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
    a, ld = out_buffer(m, inter, qg.O_F32, 0)
    b, _ = out_buffer(m, inter, qg.O_F32, 0)
    qg.gated_gemm(lay.w, xd, None, m, k, a, qg.O_F32, ld, act, ws, wsb, qg.GEMM_QUANTIZE_X)
    qg.gated_gemm(lay.w, q, qs, m, k, b, qg.O_F32, ld, act, ws, wsb)
    assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,k", [(36, 97, 2560), (34, 75, 32), (65, 13423, 32), (1653, 148, 3712), (66, 16413, 32), (691, 1788, 4192),
                                   (999, 4854, 2016), (274, 13932, 32), (583, 18164, 32), (811, 15081, 32)])
def test_every_tile_shape(m, n, k):
    test_product_matches_64_bits(m, n, k, qg.O_F32)


@pytest.mark.parametrize("m,inter,k", [(19, 64, 2560), (36, 8848, 32), (1468, 66, 2656), (85, 9950, 32), (827, 2575, 1056),
                                       (1300, 838, 1152), (350, 7001, 96), (394, 13727, 32)])
def test_every_gated_tile_shape(m, inter, k):
    test_gated_matches_64_bits(m, inter, k, qg.ACT_GELU_TANH)


def test_another_stream_and_noalloc():
    lay = Int8Layer(320, 2048, 9)
    st = torch.cuda.Stream()
    for m in (1, 9, 70):
        x, xf = rows(m, 2048, m)
        cq, cs = quantize_ref(xf)
        q, s = torch.from_numpy(cq).cuda(), torch.from_numpy(cs).cuda()
        y, ld = out_buffer(m, 320, qg.O_F32, 0)
        st.wait_stream(torch.cuda.current_stream())
        qg.gemm_noalloc(lay.w, q, s, m, 2048, y, qg.O_F32, ld, stream=st)
        st.synchronize()
        check(y[:m, :320], lay.product(cq, cs), qg.O_F32)


def test_graph_replays():
    lay = Int8Layer(512, 1024, 4)
    for m in (1, 8, 50):
        x = rows(m, 1024, 5)[0].cuda()
        y = torch.zeros(m, 512, dtype=torch.bfloat16, device="cuda")
        wsb = qg.gemm_workspace_size_ex(lay.w, m, qg.GEMM_QUANTIZE_X)
        ws = torch.zeros(max(wsb, 1), dtype=torch.uint8, device="cuda")
        run = lambda: qg.gemm_ex(lay.w, x, None, m, 1024, y, qg.O_BF16, 512, ws, wsb, qg.GEMM_QUANTIZE_X)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for rep in range(3):
            x.copy_(rows(m, 1024, 50 + rep)[0])
            run()
            eager = y.clone()
            y.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager)


@pytest.mark.parametrize("m,n,k", [(1, 16400, 4096), (5, 16400, 4096), (2, 65600, 1024)])
def test_weights_read_past_the_caches(m, n, k):
    """Few rows of 64 MB of weights and more, quantized in the kernel and before it."""
    assert n * k >= 64 << 20
    test_product_matches_64_bits(m, n, k, qg.O_BF16)


@pytest.mark.parametrize("m,inter,k", [(1, 8200, 4096), (4, 8200, 4096)])
def test_gated_weights_read_past_the_caches(m, inter, k):
    assert 2 * inter * k >= 64 << 20
    test_gated_matches_64_bits(m, inter, k, qg.ACT_SILU)


@pytest.mark.parametrize("m,k", [(3, 16416), (2, 40000), (1, 130816), (4100, 32), (8200, 264)])
def test_quantize_rows_longer_and_more_than_one_pass_holds(m, k):
    """Rows that a workgroup's registers do not hold, and more rows than workgroups."""
    test_quantize_int8(m, k)


@pytest.mark.parametrize("m,n,k", [(1, 40, 16416), (1, 17, 65408), (1, 17, 65568), (3, 33, 40000), (4200, 48, 64)])
def test_products_that_quantize_long_rows(m, n, k):
    """In the kernel (one row up to 64 K codes, past what its threads ask for
    ahead) and by a launch of its own."""
    test_product_matches_64_bits(m, n, k, qg.O_F32)


@pytest.mark.parametrize("m,inter,k", [(1, 20, 9248), (1, 17, 40000), (2, 17, 20512)])
def test_gated_products_that_quantize_long_rows(m, inter, k):
    test_gated_matches_64_bits(m, inter, k, qg.ACT_GELU_TANH)
