"""The operators around the GEMMs on views whose elements lie more than 2^31
elements apart: row pitches, batch strides and scales' pitches far beyond the
rows.  Results must equal, bit for bit, those on compact copies."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import fp8_matrix, offsets_of, randn, up

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield
    torch.cuda.empty_cache()


def far(t, pitch):
    """A copy of t (2-D, or a batch with pitch between its matrices) with that pitch."""
    strides = (pitch, 1) if t.dim() == 2 else (pitch, t.shape[2], 1)
    store = torch.empty((t.shape[0] - 1) * pitch + t[0].numel() + 16, dtype=t.dtype, device="cuda")
    assert store.numel() > 1 << 31
    return torch.as_strided(store, t.shape, strides).copy_(t)


def same(a, b):
    check_device_error()
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("dim,pitch", [(200, 32768), (2048, 32768), (201, 32769)])
def test_norm_and_its_gradient(dim, pitch):
    rows = 66000
    x, r = randn(rows, dim, seed=1, dtype=BF), randn(rows, dim, seed=2, dtype=BF)
    w = 1.0 + randn(dim, seed=3, scale=0.2)
    results = []
    for place in (lambda t: t.clone(), lambda t: far(t, pitch)):
        h, y, q = place(r), place(x), place(torch.zeros(rows, dim, dtype=F8, device="cuda"))
        s, rstd = torch.empty(up(dim), rows, device="cuda"), torch.empty(rows, device="cuda")
        g.rmsnorm(y, w, residual=h, h=h, y=y, q=q, scales=s, rstd=rstd)
        dh, dw = place(x), torch.empty(dim, device="cuda")
        g.rmsnorm_backward(dh, h, w, rstd, dh, dw, residual_grad=y)
        results.append((h, y, q, s, rstd, dh, dw))
    for a, b in zip(*results):
        same(a, b)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("cols,pitch", [(200, 32768), (131, 32769)])
def test_quantisation(cols, pitch, block, transpose):
    rows = 66000
    x = randn(rows, cols, seed=4, dtype=BF)
    qr, qc = (cols, rows) if transpose else (rows, cols)
    results = []
    for big in (False, True):
        q = torch.zeros(qr, qc, dtype=F8, device="cuda")
        if big:
            q = far(q, (1 << 31) // (qr - 1) // 16 * 16 + 16 + pitch % 2)
        s = torch.empty(up(qc), up(qr) if block == "tiles" else qr, device="cuda")
        g.fp8_quantize(far(x, pitch) if big else x, q, s, block=block, transpose=transpose)
        results.append((q, s))
    for a, b in zip(*results):
        same(a, b)


@pytest.mark.parametrize("block", ["rows", "tiles"])
def test_fp8_product(block):
    M, N, K = 66000, 300, 256
    A, sa = fp8_matrix(M, K, "rows", 5)
    B, sb = fp8_matrix(N, K, block, 6)
    D = torch.empty(M, N, dtype=BF, device="cuda")
    g.fp8gemm(A, sa, B, sb, D)
    far_s = torch.as_strided(torch.empty((1 << 31) + M + 64, device="cuda"), sa.shape, ((1 << 31) - 8, 1))
    far_d = far(torch.zeros_like(D), 32768)
    g.fp8gemm(far(A, 32768), far_s.copy_(sa), B, sb, far_d)
    same(D, far_d)


def test_grouped_products():
    counts, N, K = [300, 0, 5, 700, 64, 1, 130, 0, 600], 264, 200
    G, rows, far_batch = len(counts), sum(counts), (1 << 28) + 64
    off = offsets_of(counts)
    A, B = randn(rows, K, seed=7, dtype=BF), randn(G, K, N, seed=8, dtype=BF)
    D, dB = (torch.empty(*s, dtype=BF, device="cuda") for s in ((rows, N), (G, K, N)))
    far_d, far_b = far(torch.zeros_like(D), 1 << 21), far(B, far_batch)
    far_db = far(torch.zeros_like(dB), far_batch)
    g.bf16gemm_grouped(A, B, off, D)
    g.bf16gemm_grouped(far(A, 1 << 21), far_b, off, far_d)
    same(D, far_d)
    g.bf16gemm_grouped_wgrad(A, D, off, dB)
    g.bf16gemm_grouped_wgrad(A, far_d, off, far_db)
    same(dB, far_db)
    g.bf16gemm_grouped(A, B.transpose(1, 2).contiguous(), off, D, transpose_b=True)
    g.bf16gemm_grouped(A, far(B.transpose(1, 2).contiguous(), far_batch), off, far_d, transpose_b=True)
    same(D, far_d)


def test_grouped_fp8_product():
    counts, N, K = [30, 0, 5, 170, 64, 1, 13, 0, 60], 264, 208
    G, rows = len(counts), sum(counts)
    off = offsets_of(counts)
    A, sa = fp8_matrix(rows, K, "rows", 9)
    B, sb = fp8_matrix(N, K, "tiles", 10, lead=(G,))
    D = torch.empty(rows, N, device="cuda")
    g.fp8gemm_grouped(A, sa, B, sb, off, D)
    far_d = torch.empty_like(D)
    g.fp8gemm_grouped(A, sa, far(B, (1 << 28) + 64), sb, off, far_d)
    same(D, far_d)
