"""Products of matrices of one row: a single row's pitch says nothing, so TMA can
read it whatever its length is.  Such calls need no staging copy, hence no
buffer: they can be captured on a stream that has none.  Results are compared
with the formulas in fp64.

Products are exact in fp32; K of them are summed with at most K additions of up
to 2^-23 of the sum of magnitudes (fp8: 128 to a block, then two roundings and
an addition per block), alpha and the fp32 output add two units:

    (K + 2) * 2^-23 * den
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


def captured(run, *outs):
    """Runs `run` from a graph captured on a stream for which the library holds nothing."""
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert g.gemm_release_stream(stream.cuda_stream) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            run()
        graph.replay()
        stream.synchronize()
    check_device_error()
    assert all(o.clean_outside() for o in outs)


def check(D, a, b, out):
    a, b = a.double(), b.double()
    bound = (a.shape[1] + 2) * 2 * U32 * (a.abs() @ b.abs())
    want = a @ b
    bound = bound + (UBF if out == "bf16" else 0.0) * (want.abs() + bound)
    assert bool(((D.double() - want).abs() <= bound).all())


def values(q, s, block):
    return q.double() * spread(s, block, *q.shape)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1999), (1, 1, 129), (70, 1, 333), (1, 4097, 1001)])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_fp8(M, N, K, block, out):
    A, sa = fp8_matrix(M, K, "rows", 1, pad=-K % 16)
    B, sb = fp8_matrix(N, K, block, 2, pad=-K % 16)
    D = Guarded((M, N), DTYPE[out], 3)
    captured(lambda: g.fp8gemm(A, sa, B, sb, D.t), D)
    check(D.t, values(A, sa, "rows"), values(B, sb, block).t(), out)


@pytest.mark.parametrize("N,K", [(1, 1999), (130, 333)])
def test_fp8_grouped(N, K):
    G = 3
    A, sa = fp8_matrix(1, K, "rows", 3, pad=-K % 16)
    B, sb = fp8_matrix(N, K, "rows", 4, lead=(G,), pad=-K % 16)
    D = Guarded((1, N), torch.float32, 5)
    off = offsets_of([0, 1, 0])
    captured(lambda: g.fp8gemm_grouped(A, sa, B, sb, off, D.t), D)
    check(D.t, values(A, sa, "rows"), values(B[1], sb[1], "rows").t(), "f32")


@pytest.mark.parametrize("rows,N,K,transpose_b", [(1, 77, 1999, False), (1, 1, 65, True),
                                                  (90, 1, 1001, True), (90, 333, 1, False),
                                                  (1, 4097, 129, True)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_bf16_grouped(rows, N, K, transpose_b, out):
    A = Guarded((rows, K), torch.bfloat16, -K % 8).set(randn(rows, K, seed=5)).t
    B = Guarded((3, N, K) if transpose_b else (3, K, N), torch.bfloat16, -(K if transpose_b else N) % 8)
    B.set(randn(*B.shape, seed=6))
    D = Guarded((rows, N), DTYPE[out], 3)
    off = offsets_of([0, rows, 0])
    captured(lambda: g.bf16gemm_grouped(A, B.t, off, D.t, transpose_b=transpose_b), D)
    check(D.t, A, B.t[1].t() if transpose_b else B.t[1], out)


@pytest.mark.parametrize("rows,N,K", [(1, 77, 1999), (1, 1, 1), (1, 4097, 3), (50, 300, 1)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_gradient(rows, N, K, out):
    A = Guarded((rows, K), torch.bfloat16, -K % 8).set(randn(rows, K, seed=7)).t
    dD = Guarded((rows, N), torch.bfloat16, -N % 8).set(randn(rows, N, seed=8)).t
    for G, counts in ((1, [rows]), (2, [0, rows])):
        dB = Guarded((G, K, N), DTYPE[out], 3)
        off = offsets_of(counts)
        captured(lambda: g.bf16gemm_grouped_wgrad(A, dD, off, dB.t), dB)
        check(dB.t[-1], A.t(), dD, out)
        assert G == 1 or bool((dB.t[0] == 0).all())
