"""Which kernel an int8 product takes, read from the graph that a call is captured into: both ways give the same
bits, so that their values cannot tell them apart."""
import ctypes
import re

import pytest
import torch

import dense_gemm_12_gb300 as g
from test_gpu_int8_large import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def captured(M, N, K, path, warm=True):
    """(kernel, its first template argument) of the product in a capture on a stream with a buffer (`warm`)
    or without."""
    pitch = -(-K // 16) * 16
    A, B = (torch.ones(n, pitch, dtype=torch.int8, device="cuda")[:, :K] for n in (M, N))
    one, D = torch.ones(max(M, N), device="cuda"), torch.empty(M, N, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(s):
            g.int8gemm(A, one[:M], B, one[:N], D)
        s.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=s):
        g.int8gemm(A, one[:M], B, one[:N], D)
    D.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph.replay()
    s.synchronize()
    assert bool((D == K).all())
    dump = ctypes.CDLL("libcuda.so.1").cuGraphDebugDotPrint
    assert dump(ctypes.c_void_p(graph.raw_cuda_graph()), str(path).encode(), ctypes.c_uint(1)) == 0
    text = path.read_text()
    found = set(re.findall(r"(int8_wide_kernel|int8_kernel)(?:ILi|<\(?i?n?t?\)?)(\d+)", text))
    assert len(found) == 1, text[:2000]
    del graph
    g.gemm_release_stream(s.cuda_stream)
    return found.pop()


def test_large_products_are_widened_beforehand(tmp_path):
    found = {s: captured(*s, tmp_path / "graph.dot") for s in SHAPES}
    assert {s: k for s, (k, _) in found.items()} == dict.fromkeys(SHAPES, "int8_wide_kernel")
    assert {int(t) for _, t in found.values()} == {224, 256}


@pytest.mark.parametrize("M,N,K,tokens", [
    (16, 4096, 1024, 16), (1, 20000, 512, 16), (17, 300, 200, 32), (64, 512, 2048, 64), (128, 4096, 4096, 64),
    (500, 4000, 1000, 64), (120, 12200, 4000, 128), (100, 20000, 512, 128), (200, 30000, 1100, 128)])
def test_tokens_to_a_tile_of_smaller_products(tmp_path, M, N, K, tokens):
    assert captured(M, N, K, tmp_path / "graph.dot") == ("int8_kernel", str(tokens))


def test_a_capture_without_the_buffer_takes_the_way_without_copies(tmp_path):
    assert captured(2100, 2500, 704, tmp_path / "graph.dot")[0] == "int8_wide_kernel"
    assert captured(2100, 2500, 704, tmp_path / "graph.dot", warm=False)[0] == "int8_kernel"
