"""A captured graph holds the addresses of its stream's buffers: they stay
allocated, with the graph's results, when a later call on the stream outgrows
them, until the stream is released.

Whether a buffer is still there is read from the device's default memory pool
(the library's buffers are its only users here): growth adds the new buffer's
bytes and takes none away.  Replays come only after that has been checked.
"""
import ctypes

import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import fp8_matrix, offsets_of, randn

pytestmark = pytest.mark.gpu
USED_MEM_CURRENT = 7  # CU_MEMPOOL_ATTR_USED_MEM_CURRENT


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def pool_used():
    """Bytes allocated from the device's default memory pool once the device is idle."""
    torch.cuda.synchronize()
    driver = ctypes.CDLL("libcuda.so.1")
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert driver.cuDeviceGetDefaultMemPool(ctypes.byref(pool), torch.cuda.current_device()) == 0
    assert driver.cuMemPoolGetAttribute(pool, USED_MEM_CURRENT, ctypes.byref(used)) == 0
    return used.value


def norm_gradient(rows, dim):
    x, dy = (randn(rows, dim, seed=i, dtype=torch.bfloat16) for i in (1, 2))
    w, rstd = 1.0 + randn(dim, seed=3, scale=0.1), x.float().square().mean(-1).rsqrt()
    dh, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    return lambda: g.rmsnorm_backward(dy, x, w, rstd, dh, dw), (dh, dw)


def fp8_product(M, K):
    A, sa = fp8_matrix(M, K, "rows", 4, pad=1)  # an odd pitch: staged
    B, sb = fp8_matrix(200, K, "tiles", 5, pad=-K % 16)
    D = torch.empty(M, 200, device="cuda")
    return lambda: g.fp8gemm(A, sa, B, sb, D), (D,)


def grouped_gradient(rows, K):
    A, dD = (randn(rows, n, seed=n, dtype=torch.bfloat16) for n in (K, 72))
    off, dB = offsets_of([rows - 5, 5]), torch.empty(2, K, 72, device="cuda")
    return lambda: g.bf16gemm_grouped_wgrad(A, dD, off, dB), (dB,)


def dense_staged(M, K):
    A, B = (randn(*s, seed=7, dtype=torch.bfloat16) for s in ((M, K), (K, 256)))
    C = torch.empty(M, 256, device="cuda")
    return lambda: g.bf16gemm(A, B, C), (C,)


@pytest.mark.parametrize("make,small,large", [(norm_gradient, (256, 1024), (4096, 4096)),
                                              (fp8_product, (100, 384), (1500, 1024)),
                                              (grouped_gradient, (300, 129), (3000, 1025)),
                                              (dense_staged, (256, 257), (1024, 1025))])
def test_outgrown_buffer_of_a_graph_is_kept(make, small, large):
    run_small, out_small = make(*small)
    run_large, out_large = make(*large)
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (stream, other):  # handles are reused: start without buffers
        assert g.gemm_release_stream(s.cuda_stream) == 0
    nothing = pool_used()
    with torch.cuda.stream(other):
        run_large()
    bytes_large = pool_used() - nothing
    want_large = [t.clone() for t in out_large]
    assert bytes_large > 0 and g.gemm_release_stream(other.cuda_stream) == 0
    assert pool_used() == nothing

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        run_small()
        stream.synchronize()
        want_small = [t.clone() for t in out_small]
        with torch.cuda.graph(graph, stream=stream):
            run_small()
    bytes_small = pool_used() - nothing
    assert 0 < bytes_small < bytes_large
    with torch.cuda.stream(stream):
        run_large()
    assert pool_used() - nothing == bytes_small + bytes_large
    with torch.cuda.stream(stream):
        for _ in range(3):
            for t in (*out_small, *out_large):
                t.fill_(float("nan"))
            graph.replay()
            run_large()
            graph.replay()
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out_small, want_small))
            assert all(torch.equal(a, b) for a, b in zip(out_large, want_large))
    check_device_error()
    assert g.gemm_release_stream(stream.cuda_stream) == 0
    assert pool_used() == nothing


def test_buffer_without_a_graph_is_replaced():
    run_small, _ = fp8_product(100, 384)
    run_large, _ = fp8_product(1500, 1024)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert g.gemm_release_stream(stream.cuda_stream) == 0
    nothing = pool_used()
    with torch.cuda.stream(stream):
        run_large()
        bytes_large = pool_used() - nothing
        assert g.gemm_release_stream(stream.cuda_stream) == 0
        run_small()
        run_large()
        assert pool_used() - nothing == bytes_large
    assert g.gemm_release_stream(stream.cuda_stream) == 0
    check_device_error()
