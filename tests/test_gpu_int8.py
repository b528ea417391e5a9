"""gemm_int8_quantize and gemm_int8gemm against plain forms in 64 bits.

The product's integer sums are exact: in fp64 they are too (below 2^53), so with scales of one, no bias
and sums below 2^24 an fp32 output equals the sum.  Otherwise the sum's conversion to fp32, its products
with the two scales (one of them times alpha) and the additions of bias and beta * D round once each:
at most 6 units U = 2^-24 of the magnitudes added, and the output's half step (bf16 2^-8)."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def ints(rows, cols, seed, pad=0, off=0, low=-128):
    v = torch.randint(low, 128, (rows, cols), generator=torch.Generator().manual_seed(seed)).to(torch.int8)
    return Guarded((rows, cols), torch.int8, pad, off).set(v)


def sums64(a, b):
    return a.double() @ b.double().t()


def near(d, want, mag):
    unit = UBF if d.dtype == torch.bfloat16 else 0.0
    err = 6 * U32 * mag
    assert bool(((d.double() - want).abs() <= err + unit * (want.abs() + err)).all())


# tokens, channels, k: tiles of 16, 32, 64 and 128 tokens, whole and partial; one and many chunks of 1024
# of k; tiles split over clusters and not
SHAPES = [(1, 1, 1), (1, 256, 128), (16, 256, 128), (3, 5, 7), (16, 256, 1024), (17, 300, 200), (33, 257, 1040),
          (64, 512, 2048), (65, 100, 4096), (128, 256, 1152), (130, 520, 130), (16, 12288, 4096),
          (1, 4096, 4096), (1000, 1000, 999), (300, 2000, 1999), (700, 513, 3333), (128, 4096, 1024),
          (2000, 3000, 256), (40, 9000, 2100), (4097, 1031, 1280), (20, 38912, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sums_are_exact(M, N, K):
    # values of +-7 at most, so that the sums of 4096 stay below 2^24, and full ones where K allows
    for low, high in ((-7, 7), (-128, 127)) if K <= 1024 else ((-7, 7),):
        gen = torch.Generator().manual_seed(M + N + K)
        a = torch.randint(low, high + 1, (M, K), generator=gen).to(torch.int8)
        b = torch.randint(low, high + 1, (N, K), generator=gen).to(torch.int8)
        pitch = -(-K // 16) * 16
        A, B = (Guarded((n, K), torch.int8, pitch - K).set(v) for n, v in ((M, a), (N, b)))
        D = Guarded((M, N), torch.float32, 3)
        g.int8gemm(A.t, torch.ones(M, device="cuda"), B.t, torch.ones(N, device="cuda"), D.t)
        check_device_error()
        assert torch.equal(D.t.double(), sums64(A.t, B.t))
        assert D.clean_outside()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_bias_and_beta(M, N, K, out):
    A, B = ints(M, K, 1, pad=5, off=3), ints(N, K, 2, pad=16, off=16)
    sa, sb, bias = randn(M, seed=3).exp(), randn(N, seed=4).exp(), randn(N, seed=5, scale=100.0)
    D = Guarded((M, N), DTYPE[out], 1).set(randn(M, N, seed=6, scale=1000.0))
    old = D.t.double()
    g.int8gemm(A.t, sa, B.t, sb, D.t, alpha=-0.75, beta=0.5, bias=bias)
    check_device_error()
    prod = -0.75 * sums64(A.t, B.t) * sa.double()[:, None] * sb.double()
    near(D.t, prod + bias.double() + 0.5 * old, prod.abs() + bias.double().abs() + 0.5 * old.abs())
    assert D.clean_outside()


@pytest.mark.parametrize("M,N,K", [(3, 300, 131071), (130, 256, 65536), (16, 16, 100000)])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (127, 127)])
def test_largest_sums(M, N, K, a, b):
    # every product the same: partial sums reach 2^24 in a chunk and 2^31 in all
    pitch = -(-K // 16) * 16
    A, B = (torch.full((n, pitch), v, dtype=torch.int8, device="cuda")[:, :K] for n, v in ((M, a), (N, b)))
    ones = torch.ones(max(M, N), device="cuda")
    D = torch.empty(M, N, device="cuda")
    g.int8gemm(A, ones[:M], B, ones[:N], D, bias=torch.full((N,), float(-a * b * K // 2 * 2), device="cuda"))
    check_device_error()
    # one conversion to fp32, at most 2^7 off (half a unit of 2^31), and the bias's own
    assert bool((D.abs() <= 2.0 ** 8).all())
    A[:, -1] = 0   # one product fewer
    g.int8gemm(A, ones[:M], B, ones[:N], D)
    assert bool(((D.double() - a * b * (K - 1)).abs() <= U32 * abs(a * b) * K).all())


def test_partial_sums_at_the_edge_of_exactness():
    # 1024 products of 2^14 and then one of 1: 2^24 + 1 needs the integers beyond a chunk
    for K in (1024, 1025, 2048, 2049):
        A = torch.full((2, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
        B = A.clone()
        A[:, 1024:] = 1
        B[:, 1024:] = 1
        one = torch.ones(2, device="cuda")
        D = torch.empty(2, 2, device="cuda")
        g.int8gemm(A, one, B, one, D, bias=torch.full((2,), -(2.0 ** 24), device="cuda"))
        # 2^24 + odd rounds to even before the bias: at most one off
        assert bool(((D - (K - 1024)).abs() <= 1).all())
        D2 = torch.empty(2, 2, device="cuda")
        half = torch.full((2, K), 0, dtype=torch.int8, device="cuda")
        half[:, : K - 1] = A[:, : K - 1]
        if K % 16 == 0:
            g.int8gemm(half, one, B, one, D2)
            # 2^24 + 1023 is no fp32 number; its conversion, to nearest even, is the only rounding
            assert torch.equal(D2, sums64(half, B).float())


@pytest.mark.parametrize("M,N,K", [(5, 300, 200), (130, 300, 200)])
def test_unread_operands(M, N, K):
    nan = float("nan")
    D = Guarded((M, N), torch.float32, 1).set(randn(M, N, seed=1))
    A, B = ints(M, K, 1).t, ints(N, K, 2).t
    sa, sb = torch.full((M,), nan, device="cuda"), torch.full((N,), nan, device="cuda")
    old, bias = D.t.clone(), randn(N, seed=2)
    g.int8gemm(A, sa, B, sb, D.t, alpha=0.0, beta=2.0, bias=bias)
    near(D.t, 2.0 * old.double() + bias.double(), 2 * old.double().abs() + bias.double().abs())
    e = torch.empty(M, 0, dtype=torch.int8, device="cuda")
    g.int8gemm(e, sa, torch.empty(N, 0, dtype=torch.int8, device="cuda"), sb, D.t)
    assert bool((D.t == 0).all())
    D.t.fill_(nan)   # not read when beta is 0
    one = torch.ones(max(M, N), device="cuda")
    g.int8gemm(A, one[:M], B, one[:N], D.t)
    assert torch.equal(D.t.double(), sums64(A, B)) and D.clean_outside()


@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (1, 0), (0, 1), (16, 48)])
@pytest.mark.parametrize("M,N,K", [(1, 1, 37), (1, 300, 200), (30, 1, 100), (200, 300, 144)])
def test_operands_that_tma_cannot_describe(M, N, K, pad, off):
    A, B = ints(M, K, 1, pad, off), ints(N, K, 2, pad, off)
    one = torch.ones(max(M, N), device="cuda")
    D = Guarded((M, N), torch.bfloat16, pad, off)
    g.int8gemm(A.t, one[:M], B.t, one[:N], D.t)
    check_device_error()
    near(D.t, sums64(A.t, B.t), sums64(A.t, B.t).abs())
    assert D.clean_outside()


def test_streams_graph_and_same_bits():
    M, N, K = 40, 2000, 1111
    pairs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (1, 2):
        A, B = ints(M, K, seed), ints(N, K, seed + 10)   # pitch 1111: staged
        pairs.append((A.t, randn(M, seed=seed).exp(), B.t, randn(N, seed=seed).exp(), torch.empty(M, N, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(pairs, streams):
            with torch.cuda.stream(s):
                g.int8gemm(*p)
    torch.cuda.synchronize()

    def check(p):
        want = sums64(p[0], p[2]) * p[1].double()[:, None] * p[3].double()
        near(p[4], want, want.abs())

    for p in pairs:
        check(p)
    p, first = pairs[0], pairs[0][4].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        g.int8gemm(*p)
    p[4].zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p[4], first)
    p[0].copy_(ints(M, K, 77).t)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(p)
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh):
        with pytest.raises(g.GemmError) as e:
            g.int8gemm(*p)
        p[4].zero_()
    assert g.STATUS[e.value.status] == "GEMM_ERR_NO_MEMORY"
    check_device_error()
    for s in streams:
        g.gemm_release_stream(s.cuda_stream)


def test_outputs_past_two_to_the_31_elements():
    M, N, K = 300, 1000, 64
    A, B = ints(M, K, 1).t, ints(N, K, 2).t
    ld = 1 << 23
    raw = torch.empty((M - 1) * ld + N, dtype=torch.bfloat16, device="cuda")
    D = torch.as_strided(raw, (M, N), (ld, 1))
    one = torch.ones(N, device="cuda")
    g.int8gemm(A, one[:M], B, one, D)
    check_device_error()
    want = sums64(A, B)
    near(D, want, want.abs())


# ---------------------------------------------------------------- quantise
def check_s8(q, s, x):
    """q * s must be fp64 x rounded to whole multiples of its row's largest finite magnitude / 127."""
    fine = torch.isfinite(x)
    amax = torch.where(fine, x.abs(), 0.0).amax(1)
    scale = (amax / 127).clamp_min(2.0 ** -126)
    assert bool(((s.double() - scale).abs() <= U32 * scale).all())
    q = q.double()
    bound = 0.5 * scale[:, None] * (1 + 2.0 ** -18) + 4 * U32 * x.abs()
    assert bool(((q * scale[:, None] - x).abs() <= bound)[fine].all()) and bool((q.abs() <= 127).all())
    assert bool((q[torch.isnan(x)] == 0).all())
    inf = torch.isinf(x)
    assert bool((q[inf] == 127.0 * torch.sign(x[inf])).all())
    # the largest value keeps the whole range
    full = amax > 127 * 2.0 ** -126
    assert bool((q.abs().amax(1)[full] == 127).all())


QSHAPES = [(1, 1), (1, 4096), (3, 5), (7, 127), (64, 128), (130, 264), (65, 1000), (1000, 64), (300, 2049),
           (2000, 4096), (4, 16384), (3, 20000), (129, 8200), (5, 16385), (700, 30)]


@pytest.mark.parametrize("rows,cols", QSHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("pad,off", [(0, 0), (16, 16), (3, 1)])
def test_quantize(rows, cols, dtype, transpose, pad, off):
    v = randn(rows, cols, seed=rows + cols, device="cpu") * torch.exp(2.0 * randn(rows, 1, seed=1, device="cpu"))
    x = Guarded((rows, cols), DTYPE[dtype], pad, off).set(v)
    shape = (cols, rows) if transpose else (rows, cols)
    q, s = Guarded(shape, torch.int8, pad, off), Guarded((1, shape[0]), torch.float32, 0, 1)
    g.int8_quantize(x.t, q.t, s.t[0], transpose=transpose)
    check_s8(q.t, s.t[0], (x.t.t() if transpose else x.t).double())
    assert q.clean_outside() and s.clean_outside()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("cols", [256, 255])
def test_quantize_edges(transpose, cols):
    inf, nan = float("inf"), float("nan")
    x = randn(9, cols, seed=1)
    x[1] = 0.0
    x[2, 5], x[2, 9], x[3, 7], x[3, 8] = inf, -inf, nan, 1000.0
    x[4] = nan
    x[5] = inf
    x[6] *= 1e-40       # below the smallest scale
    x[7] *= 3e37
    x[8, :] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5] + [0.0] * (cols - 5))   # ties to even
    y = x.t().contiguous() if transpose else x
    q = torch.empty(9, cols, dtype=torch.int8, device="cuda")
    s = torch.empty(9, device="cuda")
    g.int8_quantize(y, q, s, transpose=transpose)
    check_s8(q, s, x.double())
    assert q[8, :5].tolist() == [127, 0, 2, 2, 0] and s[1] == 2.0 ** -126 and s[4] == 2.0 ** -126
    assert bool((q[5] == 127).all()) and s[5] == 2.0 ** -126


def test_quantize_rows_past_two_to_the_31_elements():
    rows, cols = (1 << 15) + 3, 1 << 16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn(3, cols, seed=1, dtype=torch.bfloat16)
    q, s = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    g.int8_quantize(x, q, s)
    check_s8(q[-3:], s[-3:], x[-3:].double())
    assert bool((s[:-3] == 2.0 ** -126).all())


def test_a_layer_in_8_bits():
    """Norm, int8 rows, product with weights laid out by the transposed quantiser: as served."""
    m, k, n = 70, 512, 384
    x, r = randn(m, k, seed=1, dtype=torch.bfloat16), randn(m, k, seed=2, dtype=torch.bfloat16)
    w, gain, bias = randn(k, n, seed=3, scale=k ** -0.5), 1.0 + randn(k, seed=4, scale=0.1), randn(n, seed=5)
    wq, ws = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    g.int8_quantize(w, wq, ws, transpose=True)
    q, s = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    g.layernorm(x, gain, residual=r, h=r, q=q, scales=s)
    d = torch.empty(m, n, device="cuda")
    g.int8gemm(q, s, wq, ws, d, bias=bias)
    check_device_error()
    # exactly what the 8-bit values say
    want = sums64(q, wq) * s.double()[:, None] * ws.double()
    near(d, want + bias.double(), want.abs() + bias.double().abs())
    # and near the layer in fp64: rows of 512 normal values reach 3.2 sigma or more, so a step of
    # max / 127 is off by max / 127 / sqrt(12) rms: 0.9 % (weights and rows alike), 4.5 sigma at most 1 %;
    # together sqrt(2) * 1 % = 1.5 %
    h = r.double()
    y = (h - h.mean(1, keepdim=True)) / h.var(1, unbiased=False, keepdim=True).add(1e-5).sqrt() * gain.double()
    full = y @ w.double()
    assert float((d.double() - bias.double() - full).norm() / full.norm()) <= 0.015
