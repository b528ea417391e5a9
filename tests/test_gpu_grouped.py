"""bf16 products grouped by expert against their definitions in fp64.

Products of bf16 values are exact in fp32; k of them are summed with at most k
additions of up to 2^-23 (the tensor cores may truncate) of the sum of
magnitudes, then come alpha, beta and the output's rounding:

    (k * 2^-23 + 2^-23) * den + 2^-23 |beta D| + u_out |D|
"""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, offsets_of, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def check(D, a, b, alpha, beta, D0, out):
    a, b = a.double(), b.double()
    want = alpha * (a @ b)
    bound = (a.shape[1] + 1) * 2 * U32 * abs(alpha) * (a.abs() @ b.abs())
    if beta:
        want = want + beta * D0.double()
        bound = bound + 2 * U32 * (beta * D0.double()).abs()
    unit = UBF if out == "bf16" else U32
    bound = bound + unit * (want.abs() + bound) + 1e-37
    bad = ~((D.double() - want).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())


COUNTS = [([5], 0, 0), ([0, 0, 7, 0], 0, 0), ([1, 1, 1, 1, 1], 0, 3), ([130, 0, 257, 3, 128], 2, 5),
          ([0] * 40 + [64] + [0] * 40, 0, 0), ([17] * 65, 0, 1), ([0, 0, 0], 0, 9), ([600, 1], 0, 0)]


def matrices(rows, G, N, K, transpose_b, pads=(0, 0), offs=(0, 0), seed=0):
    A = Guarded((rows, K), torch.bfloat16, pads[0], offs[0]).set(randn(rows, K, seed=seed))
    B = Guarded((G, N, K) if transpose_b else (G, K, N), torch.bfloat16, pads[1], offs[1])
    B.set(randn(*B.shape, seed=seed + 1))
    return A.t, B.t


@pytest.mark.parametrize("counts,start,tail", COUNTS)
@pytest.mark.parametrize("N,K", [(300, 200), (520, 1024), (8, 8), (1, 65)])
@pytest.mark.parametrize("transpose_b", [False, True])
def test_forward_and_transposed(counts, start, tail, N, K, transpose_b):
    G, rows = len(counts), start + sum(counts) + tail
    A, B = matrices(rows, G, N, K, transpose_b, pads=(-K % 8, -(K if transpose_b else N) % 8))
    off = offsets_of(counts, start)
    for out, alpha, beta in (("bf16", 1.0, 0.0), ("f32", -0.5, 0.25)):
        D0 = randn(rows, N, seed=2, dtype=DTYPE[out])
        D = Guarded((rows, N), DTYPE[out], 8).set(D0)
        g.bf16gemm_grouped(A, B, off, D.t, alpha=alpha, beta=beta, transpose_b=transpose_b)
        check_device_error()
        assert D.clean_outside() and torch.equal(D.t[:start], D0[:start])
        at = start
        for i, n in enumerate(counts):
            if n:
                b = B[i].t() if transpose_b else B[i]
                check(D.t[at:at + n], A[at:at + n], b, alpha, beta, D0[at:at + n], out)
            at += n
        assert torch.equal(D.t[at:], D0[at:])


@pytest.mark.parametrize("counts,start,tail", COUNTS)
@pytest.mark.parametrize("N,K", [(300, 200), (513, 129), (8, 264), (1, 1)])
def test_weight_gradient(counts, start, tail, N, K):
    G, rows = len(counts), start + sum(counts) + tail
    A = Guarded((rows, K), torch.bfloat16, -K % 8).set(randn(rows, K, seed=3)).t
    dD = Guarded((rows, N), torch.bfloat16, -N % 8).set(randn(rows, N, seed=4)).t
    # rows of no group hold NaN, which must reach no sum
    A[:start], dD[:start] = float("nan"), float("nan")
    if tail:
        A[rows - tail:], dD[rows - tail:] = float("nan"), float("nan")
    off = offsets_of(counts, start)
    for out, alpha, beta in (("bf16", 1.0, 0.0), ("f32", 2.0, -0.5)):
        B0 = randn(G, K, N, seed=5, dtype=DTYPE[out])
        dB = Guarded((G, K, N), DTYPE[out], 8).set(B0 if beta else torch.full_like(B0, float("nan")))
        g.bf16gemm_grouped_wgrad(A, dD, off, dB.t, alpha=alpha, beta=beta)
        check_device_error()
        assert dB.clean_outside()
        at = start
        for i, n in enumerate(counts):
            check(dB.t[i], A[at:at + n].t(), dD[at:at + n], alpha, beta, B0[i], out)
            at += n


def test_neighbours_of_a_group_do_not_reach_it():
    # every second group holds NaN and infinities; the others' results are those without them
    G, n, N, K = 6, 37, 264, 136
    rows = G * n
    off = offsets_of([n] * G)
    A, B = matrices(rows, G, N, K, False, seed=6)
    dD = randn(rows, N, seed=8, dtype=torch.bfloat16)
    D, dB = torch.empty(rows, N, device="cuda"), torch.empty(G, K, N, device="cuda")
    g.bf16gemm_grouped(A, B, off, D)
    g.bf16gemm_grouped_wgrad(A, dD, off, dB)
    A2, B2, dD2 = A.clone(), B.clone(), dD.clone()
    for i in (1, 3, 5):
        A2[i * n:(i + 1) * n], B2[i], dD2[i * n:(i + 1) * n] = float("nan"), float("inf"), float("inf")
    D2, dB2 = torch.empty_like(D), torch.empty_like(dB)
    g.bf16gemm_grouped(A2, B2, off, D2)
    g.bf16gemm_grouped_wgrad(A2, dD2, off, dB2)
    for i in (0, 2, 4):
        assert torch.equal(D[i * n:(i + 1) * n], D2[i * n:(i + 1) * n]) and torch.equal(dB[i], dB2[i])


@pytest.mark.parametrize("pads,offs", [((0, 0), (1, 0)), ((3, 8), (0, 8)), ((8, 1), (3, 5))])
@pytest.mark.parametrize("transpose_b", [False, True])
def test_staged_operands(pads, offs, transpose_b):
    counts, N, K = [50, 0, 100, 3], 77, 190
    rows = sum(counts)
    A, B = matrices(rows, 4, N, K, transpose_b, pads, offs, seed=9)
    off = offsets_of(counts)
    D = Guarded((rows, N), torch.float32, 1, 1)
    g.bf16gemm_grouped(A, B, off, D.t, transpose_b=transpose_b)
    dD = Guarded((rows, N), torch.bfloat16, pads[1], offs[1]).set(randn(rows, N, seed=11)).t
    dB = Guarded((4, K, N), torch.float32, 3, 1)
    g.bf16gemm_grouped_wgrad(A, dD, off, dB.t)
    check_device_error()
    assert D.clean_outside() and dB.clean_outside()
    at = 0
    for i, n in enumerate(counts):
        if n:
            check(D.t[at:at + n], A[at:at + n], B[i].t() if transpose_b else B[i], 1.0, 0.0, None, "f32")
        check(dB.t[i], A[at:at + n].t(), dD[at:at + n], 1.0, 0.0, None, "f32")
        at += n


@pytest.mark.parametrize("counts", [[3, 400, 0, 129], [64, 64, 64, 64]])
def test_integers_exact(counts):
    N, K, rows = 528, 1032, sum(counts)
    gen = torch.Generator().manual_seed(12)
    A = torch.randint(-4, 5, (rows, K), generator=gen).to(torch.bfloat16).cuda()
    B = torch.randint(-4, 5, (4, K, N), generator=gen).to(torch.bfloat16).cuda()
    dD = torch.randint(-4, 5, (rows, N), generator=gen).to(torch.bfloat16).cuda()
    off = offsets_of(counts)
    D, dA = torch.empty(rows, N, device="cuda"), torch.empty(rows, K, device="cuda")
    dB = torch.empty(4, K, N, device="cuda")
    g.bf16gemm_grouped(A, B, off, D)
    g.bf16gemm_grouped(dD, B, off, dA, transpose_b=True)
    g.bf16gemm_grouped_wgrad(A, dD, off, dB)
    at = 0
    for i, n in enumerate(counts):
        a, d, b = A[at:at + n].double(), dD[at:at + n].double(), B[i].double()
        assert torch.equal(D[at:at + n].double(), a @ b)
        assert torch.equal(dA[at:at + n].double(), d @ b.t())
        assert torch.equal(dB[i].double(), a.t() @ d)
        at += n


def test_gradients_against_differences():
    # L = sum(dD * D) is linear in A and in B: the difference of two forward passes along a
    # direction E is the gradient's product with E, but for the rounding of both (bounds above)
    counts, N, K = [20, 0, 45, 1], 136, 72
    rows = sum(counts)
    off = offsets_of(counts)
    A, B = matrices(rows, 4, N, K, False, seed=13)
    dD, E, F = (randn(*s, seed=14 + i, dtype=torch.bfloat16) for i, s in
                enumerate([(rows, N), (rows, K), (4, K, N)]))
    dA, dB, D = (torch.empty(*s, device="cuda") for s in [(rows, K), (4, K, N), (rows, N)])
    g.bf16gemm_grouped(dD, B, off, dA, transpose_b=True)
    g.bf16gemm_grouped_wgrad(A, dD, off, dB)

    def magnitude(a, b):  # sum over t, k, n of |dD[t, n]| |a[t, k]| |b[g, k, n]|
        total, at = 0.0, 0
        for i, n in enumerate(counts):
            p = a[at:at + n].double().abs() @ b[i].double().abs()
            total += float((dD[at:at + n].double().abs() * p).sum())
            at += n
        return total

    g.bf16gemm_grouped(E, B, off, D)
    apart = float((dD.double() * D.double()).sum() - (dA.double() * E.double()).sum())
    assert abs(apart) <= ((K + 2) + (N + 2)) * 2 * U32 * magnitude(E, B)
    g.bf16gemm_grouped(A, F, off, D)
    apart = float((dD.double() * D.double()).sum() - (dB.double() * F.double()).sum())
    assert abs(apart) <= ((K + 2) + (rows + 2)) * 2 * U32 * magnitude(A, F)


def test_degenerate_sizes():
    off = offsets_of([2, 3])
    A, B = matrices(5, 2, 16, 0, False)
    D = randn(5, 16, seed=15)
    want = 0.5 * D
    g.bf16gemm_grouped(A, B, off, D, alpha=float("inf"), beta=0.5)
    assert torch.equal(D, want)
    A, B = matrices(5, 2, 16, 8, False)
    g.bf16gemm_grouped(A, B, off, D, alpha=0.0)
    assert (D == 0).all()
    dB = randn(2, 8, 16, seed=16)
    want = 2.0 * dB
    none = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    g.bf16gemm_grouped_wgrad(none, torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"),
                             offsets_of([0, 0]), dB, beta=2.0)
    assert torch.equal(dB, want)
    g.bf16gemm_grouped(none, torch.empty(2, 8, 16, dtype=torch.bfloat16, device="cuda"), off,
                       torch.empty(0, 16, device="cuda"))
    check_device_error()


def test_offsets_out_of_order_stay_in_range():
    G, rows, N, K = 6, 100, 256, 128
    A, B = matrices(rows, G, N, K, False, seed=17)
    off = torch.tensor([-5, 40, 20, 1 << 30, 60, -(1 << 31), 90], dtype=torch.int32, device="cuda")
    D, dB = Guarded((rows, N), torch.float32, 8), Guarded((G, K, N), torch.float32, 8)
    g.bf16gemm_grouped(A, B, off, D.t)
    dD = randn(rows, N, seed=18, dtype=torch.bfloat16)
    g.bf16gemm_grouped_wgrad(A, dD, off, dB.t)
    check_device_error()
    assert D.clean_outside() and dB.clean_outside()
    check(D.t[:40], A[:40], B[0], 1.0, 0.0, None, "f32")
    check(D.t[40:], A[40:], B[2], 1.0, 0.0, None, "f32")
    check(dB.t[2], A[40:].t(), dD[40:], 1.0, 0.0, None, "f32")
    assert all((dB.t[i] == 0).all() for i in (1, 3, 4, 5))


def test_most_groups_and_a_graph():
    G, N, K = 1024, 24, 64
    counts = [i % 3 for i in range(G)]
    rows = sum(counts)
    off, use = offsets_of(counts), offsets_of(counts[::-1])
    A, B = matrices(rows, G, N, K, False, seed=19)
    dD = randn(rows, N, seed=21, dtype=torch.bfloat16)
    D, dB = torch.empty(rows, N, device="cuda"), torch.empty(G, K, N, device="cuda")

    def work(o):
        g.bf16gemm_grouped(A, B, o, D)
        g.bf16gemm_grouped_wgrad(A, dD, o, dB)

    work(off)
    first = (D.clone(), dB.clone())
    at = 0
    for i, n in enumerate(counts):
        if n and i % 50 < 3:
            check(D[at:at + n], A[at:at + n], B[i], 1.0, 0.0, None, "f32")
            check(dB[i], A[at:at + n].t(), dD[at:at + n], 1.0, 0.0, None, "f32")
        at += n
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            work(use)
        use.copy_(off)
        graph.replay()
        stream.synchronize()
    assert torch.equal(D, first[0]) and torch.equal(dB, first[1])


@pytest.mark.parametrize("counts,start,tail", [([600], 0, 0), ([513, 1, 1537, 0, 1000], 3, 4),
                                               ([1025, 999], 0, 1), ([16, 2000, 15, 47], 1, 0),
                                               ([0, 0, 3000], 7, 9)])
@pytest.mark.parametrize("N,K", [(300, 200), (520, 1024), (256, 129), (2048, 700), (9, 385)])
def test_weight_gradient_of_long_groups(counts, start, tail, N, K):
    G, rows = len(counts), start + sum(counts) + tail
    A = Guarded((rows, K), torch.bfloat16, -K % 8).set(randn(rows, K, seed=6)).t
    dD = Guarded((rows, N), torch.bfloat16, -N % 8).set(randn(rows, N, seed=7)).t
    off, ends = offsets_of(counts, start), [start + sum(counts[:i]) for i in range(G + 1)]
    for out, alpha, beta in (("bf16", 1.0, 0.0), ("f32", 2.0, -0.5)):
        for keep in (0, 1):  # every other group holds NaN, and the rows of none: neither reaches the rest
            a, d = A.clone(), dD.clone()
            a[:start], d[ends[-1]:] = float("nan"), float("nan")
            for i in range(G):
                if i % 2 != keep:
                    a[ends[i]:ends[i + 1]], d[ends[i]:ends[i + 1]] = float("nan"), float("nan")
            B0 = randn(G, K, N, seed=8, dtype=DTYPE[out])
            dB = Guarded((G, K, N), DTYPE[out], 8).set(B0 if beta else torch.full_like(B0, float("nan")))
            g.bf16gemm_grouped_wgrad(a, d, off, dB.t, alpha=alpha, beta=beta)
            check_device_error()
            assert dB.clean_outside()
            for i in range(keep, G, 2):
                check(dB.t[i], a[ends[i]:ends[i + 1]].t(), d[ends[i]:ends[i + 1]], alpha, beta, B0[i], out)
