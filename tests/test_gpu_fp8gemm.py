"""gemm_fp8gemm and gemm_fp8gemm_grouped against the definition in fp64.

The tensor cores sum a block's 128 products in fp32: at most 128 additions of
up to 2^-23 (they may truncate) of the block's sum of magnitudes.  The scaled
block sums are added in fp32: two roundings of the scaled value and one
addition per k-block, then alpha, beta and the output's rounding.  With
den = |alpha| sum |scaled A| |scaled B| that is

    (128 * 2^-23 + (k-blocks + 4) * 2^-24) * den + 2^-23 |beta D| + u_out |D|
"""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, fp8_matrix, offsets_of, randn, spread, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def values(q, s, block):
    return q.double() * spread(s, block, *q.shape)


def check(D, a, b, alpha, beta, D0, out):
    """D against alpha a b^T + beta D0, all fp64; a, b the scaled operands."""
    K = a.shape[1]
    want = alpha * (a @ b.t())
    den = abs(alpha) * (a.abs() @ b.abs().t())
    bound = (128 * 2 * U32 + (up(K) + 4) * U32) * den
    if beta:
        want = want + beta * D0.double()
        bound = bound + 2 * U32 * (beta * D0.double()).abs()
    unit = UBF if out == "bf16" else U32
    bound = bound + unit * (want.abs() + bound) + 1e-37
    bad = ~((D.double() - want).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())


def run(M, N, K, block, out, alpha=1.0, beta=0.0, pads=(0, 0, 0), offs=(0, 0, 0), seed=0, spad=0):
    A, sa0 = fp8_matrix(M, K, "rows", seed, pad=pads[0], off=offs[0])
    B, sb0 = fp8_matrix(N, K, block, seed + 1, pad=pads[1], off=offs[1])
    sa = Guarded(sa0.shape, torch.float32, spad).set(sa0).t
    sb = Guarded(sb0.shape, torch.float32, spad).set(sb0).t
    D0 = randn(M, N, seed=seed + 2, scale=10.0, dtype=DTYPE[out])
    D = Guarded((M, N), DTYPE[out], pads[2], offs[2])
    D.set(D0 if beta else torch.full_like(D0, float("nan")))
    g.fp8gemm(A, sa, B, sb, D.t, alpha=alpha, beta=beta)
    check_device_error()
    assert D.clean_outside()
    check(D.t, values(A, sa, "rows"), values(B, sb, block), alpha, beta, D0, out)


SHAPES = [(1, 1, 1), (1, 128, 128), (16, 4096, 4096), (17, 300, 130), (32, 256, 1000), (33, 257, 384),
          (64, 1000, 2048), (65, 512, 127), (100, 129, 129), (128, 256, 128), (129, 255, 257),
          (300, 700, 1999), (1000, 520, 640), (256, 4096, 1024), (4, 12288, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_shapes(M, N, K, block, out):
    # pitches that TMA can describe: rows padded to 16 bytes
    run(M, N, K, block, out, pads=(-K % 16, -K % 16, 0), seed=M + N + K)


@pytest.mark.parametrize("M,N,K", [(5, 70, 200), (130, 300, 333), (40, 2000, 1000)])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("pads,offs,spad", [((0, 0, 3), (0, 0, 1), 1), ((16, 1, 0), (16, 3, 0), 0),
                                            ((7, 32, 5), (5, 16, 2), 3)])
def test_pitches_and_addresses(M, N, K, block, pads, offs, spad):
    # operands that TMA cannot describe are staged; scales and D take any
    run(M, N, K, block, "f32", pads=pads, offs=offs, spad=spad, seed=3)
    run(M, N, K, block, "bf16", pads=pads, offs=offs, spad=spad, seed=4)


@pytest.mark.parametrize("M,N,K", [(20, 600, 700), (300, 300, 300)])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("alpha,beta", [(0.5, 1.0), (-2.0, 0.25), (1.0, -1.0), (0.0, 0.5), (0.0, 0.0)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_alpha_beta(M, N, K, block, alpha, beta, out):
    run(M, N, K, block, out, alpha, beta, pads=(-K % 16, -K % 16, 4), seed=5)


@pytest.mark.parametrize("M,N", [(3, 100), (200, 300)])
def test_empty_k(M, N):
    A = torch.empty(M, 0, dtype=torch.float8_e4m3fn, device="cuda")
    B = torch.empty(N, 0, dtype=torch.float8_e4m3fn, device="cuda")
    sa, sb = torch.empty(0, M, device="cuda"), torch.empty(0, N, device="cuda")
    D = randn(M, N, seed=6)
    want = 0.5 * D
    g.fp8gemm(A, sa, B, sb, D, alpha=float("inf"), beta=0.5)
    assert torch.equal(D, want)
    g.fp8gemm(A, sa, B, sb, D)
    assert (D == 0).all()


@pytest.mark.parametrize("M,N,K", [(16, 512, 4096), (200, 520, 1152), (1000, 1000, 384)])
@pytest.mark.parametrize("block", ["rows", "tiles"])
def test_integers_exact(M, N, K, block):
    # integers up to 4 in magnitude and power-of-two scales: every partial sum is exact in fp32
    gen = torch.Generator().manual_seed(7)
    A = torch.randint(-4, 5, (M, K), generator=gen).float().cuda().to(torch.float8_e4m3fn)
    B = torch.randint(-4, 5, (N, K), generator=gen).float().cuda().to(torch.float8_e4m3fn)
    sa = torch.exp2(torch.randint(-1, 2, (up(K), M), generator=gen).float()).cuda()
    sb = torch.exp2(torch.randint(-1, 2, (up(K), N if block == "rows" else up(N)), generator=gen).float()).cuda()
    D = torch.empty(M, N, device="cuda")
    g.fp8gemm(A, sa, B, sb, D)
    assert torch.equal(D.double(), values(A, sa, "rows") @ values(B, sb, block).t())


def test_every_e4m3_value():
    # each of the 254 finite codes times one, exactly
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    A = torch.zeros(254, 128, dtype=torch.uint8)
    A[:, 0] = codes
    B = torch.zeros(256, 128)
    B[:, 0] = 1.0
    D = torch.empty(254, 256, device="cuda")
    A8 = A.cuda().view(torch.float8_e4m3fn)
    g.fp8gemm(A8, torch.ones(1, 254, device="cuda"), B.cuda().to(torch.float8_e4m3fn),
              torch.ones(1, 2, device="cuda"), D)
    assert torch.equal(D, A8[:, :1].float().expand(254, 256))


def test_nan_and_infinite_scales_stay_in_their_rows():
    M, N, K = 200, 300, 256
    A, sa = fp8_matrix(M, K, "rows", 8)
    B, sb = fp8_matrix(N, K, "rows", 9)
    A.view(torch.uint8)[3, 17] = 0x7F
    sa[1, 70] = float("inf")
    sb[0, 150] = float("nan")
    D = torch.empty(M, N, device="cuda")
    g.fp8gemm(A, sa, B, sb, D)
    clean = torch.ones(M, N, dtype=torch.bool, device="cuda")
    clean[3], clean[70], clean[:, 150] = False, False, False
    assert torch.isfinite(D[clean]).all() and torch.isnan(D[3]).all() and torch.isnan(D[:, 150]).all()
    assert not torch.isfinite(D[70]).any()


@pytest.mark.parametrize("counts,start,tail", [
    ([5], 0, 0), ([0, 0, 7, 0], 0, 0), ([1, 1, 1, 1, 1], 0, 3), ([130, 0, 257, 3, 128], 2, 5),
    ([0] * 40 + [64] + [0] * 40, 0, 0), ([17] * 65, 0, 1), ([0, 0, 0], 0, 9), ([600, 1], 0, 0)])
@pytest.mark.parametrize("N,K", [(300, 200), (513, 1024)])
@pytest.mark.parametrize("block", ["rows", "tiles"])
def test_grouped(counts, start, tail, N, K, block):
    G, rows = len(counts), start + sum(counts) + tail
    A, sa = fp8_matrix(rows, K, "rows", 10, pad=-K % 16)
    B, sb = fp8_matrix(N, K, block, 11, lead=(G,), pad=-K % 16)
    off = offsets_of(counts, start)
    for out, beta in (("bf16", 0.0), ("f32", 0.5)):
        D0 = randn(rows, N, seed=12, dtype=DTYPE[out])
        D = Guarded((rows, N), DTYPE[out], 8).set(D0)
        g.fp8gemm_grouped(A, sa, B, sb, off, D.t, beta=beta)
        check_device_error()
        assert D.clean_outside()
        a = values(A, sa, "rows")
        at = start
        assert torch.equal(D.t[:start], D0[:start])
        for i, n in enumerate(counts):
            check(D.t[at:at + n], a[at:at + n], values(B[i], sb[i], block), 1.0, beta,
                  D0[at:at + n], out) if n else None
            at += n
        assert torch.equal(D.t[at:], D0[at:])


def test_grouped_staged_operands_and_strided_batches():
    G, rows, N, K = 3, 90, 130, 250
    A, sa = fp8_matrix(rows, K, "rows", 13, pad=1, off=3)
    B, sb = fp8_matrix(N, K, "tiles", 14, lead=(G,), pad=2, off=1)
    wide = torch.zeros(2 * G, N, 256, device="cuda").to(torch.float8_e4m3fn)
    wide[::2, :, :K].copy_(B)
    off = offsets_of([40, 0, 50])
    one, two = torch.empty(rows, N, device="cuda"), torch.empty(rows, N, device="cuda")
    g.fp8gemm_grouped(A, sa, B, sb, off, one)
    g.fp8gemm_grouped(A, sa, wide[::2, :, :K], sb, off, two)
    assert torch.equal(one, two)
    check(one[:40], values(A, sa, "rows")[:40], values(B[0], sb[0], "tiles"), 1.0, 0.0, one, "f32")


def test_grouped_equals_dense_for_one_group():
    M, N, K = 1000, 1024, 2048
    A, sa = fp8_matrix(M, K, "rows", 15)
    B, sb = fp8_matrix(N, K, "tiles", 16)
    one, two = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    g.fp8gemm_grouped(A, sa, B[None], sb[None], offsets_of([M]), one)
    g.fp8gemm(A, sa, B, sb, two)
    bound = 2 * (128 * 2 * U32 + 20 * U32) * (values(A, sa, "rows").abs() @ values(B, sb, "tiles").abs().t())
    assert ((one.double() - two.double()).abs() <= bound).all()


def test_offsets_out_of_order_stay_in_range():
    G, rows, N, K = 6, 100, 256, 256
    A, sa = fp8_matrix(rows, K, "rows", 17)
    B, sb = fp8_matrix(N, K, "tiles", 18, lead=(G,))
    off = torch.tensor([-5, 40, 20, 1 << 30, 60, -(1 << 31), 90], dtype=torch.int32, device="cuda")
    D = Guarded((rows, N), torch.float32, 8)
    g.fp8gemm_grouped(A, sa, B, sb, off, D.t)
    check_device_error()
    # clamped and made non-decreasing: 0, 40, 40, 100, 100, 100, 100
    a = values(A, sa, "rows")
    check(D.t[:40], a[:40], values(B[0], sb[0], "tiles"), 1.0, 0.0, None, "f32")
    check(D.t[40:], a[40:], values(B[2], sb[2], "tiles"), 1.0, 0.0, None, "f32")
    assert D.clean_outside()


def test_same_bits_on_any_stream_and_offsets_read_at_replay():
    G, rows, N, K = 4, 300, 520, 640
    A, sa = fp8_matrix(rows, K, "rows", 19)
    B, sb = fp8_matrix(N, K, "tiles", 20, lead=(G,))
    off, other = offsets_of([100, 50, 0, 150]), offsets_of([0, 250, 20, 30])
    D = torch.empty(rows, N, device="cuda")
    g.fp8gemm_grouped(A, sa, B, sb, off, D)
    first = D.clone()
    use = other.clone()
    g.fp8gemm_grouped(A, sa, B, sb, use, D)
    second = D.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            g.fp8gemm_grouped(A, sa, B, sb, use, D)
            g.fp8gemm(A, sa, B[0], sb[0], D, beta=1.0)
        for o, want in ((off, first), (other, second)):
            use.copy_(o)
            graph.replay()
            stream.synchronize()
            plus = want.clone()
            g.fp8gemm(A, sa, B[0], sb[0], plus, beta=1.0, stream=stream)
            stream.synchronize()
            assert torch.equal(D, plus)
