"""gemm_int8gemm at sizes where both operands are widened beforehand, against sums in 64 bits: the same
bounds as for the smaller products (exact sums; six roundings of 2^-24 and the output's half step)."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, randn
from test_gpu_int8 import ints, near, sums64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def kernels(run):
    """The names of the kernels that `run` launches (the profiler may miss the first ones of a process);
    the test ends here where the profiler sees none at all."""
    for _ in range(3):
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
            run()
            torch.cuda.synchronize()
        names = " ".join(e.key for e in prof.key_averages())
        if "int8" in names:
            return names
    pytest.skip("the profiler reports no kernels")


# whole and partial tiles of 256 x 256; less than a k-block of 64, one, a chunk of 1024 and around it
SHAPES = [(4096, 4352, 64), (4100, 4099, 5), (2305, 2049, 1025), (2100, 2500, 1023), (2048, 4096, 512),
          (4097, 1031, 2048), (1031, 6000, 2113), (3000, 5000, 1999), (2561, 2560, 8200)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 3), (16, 16)])
def test_sums_scales_bias_and_beta(M, N, K, pad, off):
    A, B = ints(M, K, 1, pad=pad, off=off), ints(N, K, 2, pad=pad, off=off)
    sums = sums64(A.t, B.t)
    if K <= 1024:
        D = Guarded((M, N), torch.float32, 3)
        g.int8gemm(A.t, torch.ones(M, device="cuda"), B.t, torch.ones(N, device="cuda"), D.t)
        check_device_error()
        assert torch.equal(D.t.double(), sums)
        assert D.clean_outside()
    sa, sb, bias = randn(M, seed=3).exp(), randn(N, seed=4).exp(), randn(N, seed=5, scale=100.0)
    prod = -0.75 * sums * sa.double()[:, None] * sb.double()
    for out, beta, ld in (("f32", 0.5, 1), ("bf16", 0.5, 1), ("bf16", 0.0, 2)):
        D = Guarded((M, N), DTYPE[out], ld).set(randn(M, N, seed=6, scale=1000.0))
        old = beta * D.t.double()
        g.int8gemm(A.t, sa, B.t, sb, D.t, alpha=-0.75, beta=beta, bias=bias)
        check_device_error()
        near(D.t, prod + bias.double() + old, prod.abs() + bias.double().abs() + old.abs())
        assert D.clean_outside()


def test_which_way_a_product_goes():
    def names(M, N, K):
        A, B = ints(M, K, 1).t, ints(N, K, 2).t
        D = torch.empty(M, N, device="cuda")
        return kernels(lambda: g.int8gemm(A, torch.ones(M, device="cuda"), B, torch.ones(N, device="cuda"), D))

    found = {s: names(*s) for s in SHAPES}
    assert {s: "int8_wide_kernel" in n for s, n in found.items()} == dict.fromkeys(SHAPES, True)
    for tokens in (224, 256):   # to a tile, whichever makes the better rounds
        assert any("int8_wide_kernel<%d>" % tokens in n for n in found.values())
    small = [(16, 4096, 1024), (128, 4096, 1024), (256, 256, 4096), (1, 20000, 512)]
    assert {s: "int8_wide_kernel" in names(*s) for s in small} == dict.fromkeys(small, False)


@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (127, 127)])
@pytest.mark.parametrize("K", [1024, 1025, 16400])
def test_largest_sums(K, a, b):
    # every product the same: a chunk's sums reach 2^24
    M, N = 2304, 2304
    pitch = -(-K // 16) * 16
    A, B = (torch.full((n, pitch), v, dtype=torch.int8, device="cuda")[:, :K] for n, v in ((M, a), (N, b)))
    A[:, 0] = 1   # and an odd number in between
    A[M // 2:, K - 1] = 3
    ones = torch.ones(M, device="cuda")
    D = torch.empty(M, N, device="cuda")
    g.int8gemm(A, ones, B, ones[:N], D)
    check_device_error()
    assert torch.equal(D, sums64(A, B).float())   # the conversion, to nearest even, is the only rounding


def test_longest_rows():
    # K = 2^17 - 1, all products 2^14: just below 2^31
    K, n = 131071, 2000
    A, B = (torch.full((n, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K] for _ in range(2))
    A[:, 1] = torch.arange(n, device="cuda") % 256 - 128
    D = torch.empty(n, n, device="cuda")
    one = torch.ones(n, device="cuda")
    g.int8gemm(A, one, B, one, D)
    check_device_error()
    want = 2.0 ** 14 * (K - 1) - 128 * A[:, 1].double()
    assert torch.equal(D, want[:, None].expand(n, n).float())
    assert "int8_wide_kernel" in kernels(lambda: g.int8gemm(A, one, B, one, D))


def test_the_same_bits_in_a_capture_on_streams_and_with_the_smaller_tiles():
    M, N, K = 2100, 2500, 704
    A, B = ints(M, K, 1).t, ints(N, K, 2).t
    sa, sb = randn(M, seed=3).exp(), randn(N, seed=4).exp()

    def run(D):
        g.int8gemm(A, sa, B, sb, D)

    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    run(want)
    # row blocks of 128 tokens take the other way: the same sums, finished alike
    parts = torch.empty_like(want)
    for i in range(0, M, 128):
        g.int8gemm(A[i:i + 128], sa[i:i + 128], B, sb, parts[i:i + 128])
    assert torch.equal(parts, want)
    torch.cuda.synchronize()
    # a stream without a buffer: a capture cannot have one
    for warm in (False, True):
        s = torch.cuda.Stream()
        D, E = torch.empty_like(want), torch.empty_like(want)
        if warm:
            with torch.cuda.stream(s):
                run(E)
            s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run(D)
        D.zero_()
        E.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
            run(E)          # behind the replay, in the same buffer
            graph.replay()
        s.synchronize()
        check_device_error()
        assert torch.equal(D, want) and torch.equal(E, want)
    # two streams at once, each with a buffer of its own
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    for _ in range(4):
        for s, D in zip(streams, outs):
            with torch.cuda.stream(s):
                run(D)
    torch.cuda.synchronize()
    assert all(torch.equal(D, want) for D in outs)


def test_row_blocks_and_nothing_behind_them():
    # rows behind the last token and columns behind the last channel keep their bytes
    M, N, K = 2101, 2503, 130
    A, B = ints(M, K, 1, pad=14).t, ints(N, K, 2, pad=14).t
    for dtype in (torch.float32, torch.bfloat16):
        D = torch.full((M + 40, N + 61), 7.0, dtype=dtype, device="cuda")
        g.int8gemm(A, torch.ones(M, device="cuda"), B, torch.ones(N, device="cuda"), D[:M, :N])
        check_device_error()
        mag = sums64(A, B)
        assert bool(((D[:M, :N].double() - mag).abs() <= (UBF if dtype == torch.bfloat16 else U32) * mag.abs()).all())
        assert bool((D[M:] == 7).all()) and bool((D[:, N:] == 7).all())


# tiles of 128 tokens that widen as they go: split over a cluster, one and several tiles a CTA
@pytest.mark.parametrize("M,N,K,name", [
    (120, 12200, 4000, "<128, true>"), (128, 12288, 4097, "<128, true>"), (100, 20000, 512, "<128, false>"),
    (127, 24001, 300, "<128, false>"), (100, 50000, 140, "<128, false>"), (200, 30000, 1100, "<128, false>")])
def test_tiles_of_128_tokens(M, N, K, name):
    A, B = ints(M, K, 1, pad=-K % 16), ints(N, K, 2, pad=-K % 16)
    sa, sb, bias = randn(M, seed=3).exp(), randn(N, seed=4).exp(), randn(N, seed=5, scale=100.0)
    prod = sums64(A.t, B.t) * sa.double()[:, None] * sb.double()
    for out, beta, pad in (("f32", 0.5, 3), ("bf16", 0.0, N % 2), ("bf16", 0.0, 1 - N % 2)):
        D = Guarded((M, N), DTYPE[out], pad).set(randn(M, N, seed=6, scale=1000.0))
        old = beta * D.t.double()
        g.int8gemm(A.t, sa, B.t, sb, D.t, beta=beta, bias=bias)
        check_device_error()
        near(D.t, prod + bias.double() + old, prod.abs() + bias.double().abs() + old.abs())
        assert D.clean_outside()
    assert "int8_kernel" + name in kernels(lambda: g.int8gemm(A.t, sa, B.t, sb, D.t, bias=bias))


# 64 tokens to a tile though there are more: one tile a CTA and split ones
@pytest.mark.parametrize("M,N,K", [(128, 4096, 4096), (100, 1000, 999), (500, 4000, 1000), (513, 1000, 2100)])
def test_tiles_of_64_of_more_tokens(M, N, K):
    A, B = ints(M, K, 1, pad=-K % 16), ints(N, K, 2, pad=-K % 16)
    D = torch.empty(M, N, device="cuda")
    one = torch.ones(max(M, N), device="cuda")
    g.int8gemm(A.t, one[:M], B.t, one[:N], D)
    check_device_error()
    assert torch.equal(D, sums64(A.t, B.t).float())
    assert "int8_kernel<64" in kernels(lambda: g.int8gemm(A.t, one[:M], B.t, one[:N], D))
