"""What follows a row of an output stays as it was, also where the row's pitch is
made for 16-byte pieces but the row ends inside one.  (A TMA store clips along a
row to whole 16-byte pieces.)  Outputs are integers, exactly known; the bytes
around every row are compared."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, Guarded, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def small(*shape, seed):
    """Integers up to 2: sums of 30 products are exact in bf16 too (120 < 256)."""
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=gen).to(torch.bfloat16).cuda()


def aligned(t):
    """A copy whose rows TMA can read (pitch of whole 16-byte pieces)."""
    return Guarded(t.shape, t.dtype, -t.shape[-1] % 8).set(t).t


# every remainder of a row's length by the 8 (bf16) or 4 (fp32) elements of a piece; ends in
# the first and the last chunk of 32 of a tile of 256, just before and after a tile's end
WIDTHS = [1, 2, 3, 31, 33, 77, 100, 225, 254, 255, 257, 262, 301, 515]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("more", [0, 32])
def test_grouped(N, out, more):
    counts, K = [64, 0, 37, 200], 30
    rows = sum(counts)
    off = offsets_of(counts)
    A, B, dD = small(rows, K, seed=1), small(4, K, N, seed=2), small(rows, N, seed=3)
    pad = -N % (8 if out == "bf16" else 4) + more
    D, dB = Guarded((rows, N), DTYPE[out], pad), Guarded((4, K, N), DTYPE[out], pad)
    ends = [sum(counts[:i]) for i in range(5)]
    want = torch.cat([A[ends[i]:ends[i + 1]].double() @ B[i].double() for i in range(4)])
    g.bf16gemm_grouped(aligned(A), aligned(B), off, D.t)
    check_device_error()
    assert D.clean_outside() and torch.equal(D.t.double(), want)
    g.bf16gemm_grouped(aligned(A), aligned(B.transpose(1, 2).contiguous()), off, D.t, transpose_b=True)
    check_device_error()
    assert D.clean_outside() and torch.equal(D.t.double(), want)
    # the weight gradient sums up to 200 rows: exact in fp32, one rounding in bf16
    want = torch.stack([A[ends[i]:ends[i + 1]].double().t() @ dD[ends[i]:ends[i + 1]].double()
                        for i in range(4)])
    g.bf16gemm_grouped_wgrad(aligned(A), aligned(dD), off, dB.t)
    check_device_error()
    assert dB.clean_outside() and torch.equal(dB.t.double(), want.to(DTYPE[out]).double())


@pytest.mark.parametrize("N", [77, 254, 301, 2049])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_pairs(N, out):
    # long groups: CTA pairs in all three products
    counts, K = [1100, 1500], 30
    rows = sum(counts)
    off = offsets_of(counts)
    A, B, dD = small(rows, K, seed=4), small(2, K, N, seed=5), small(rows, N, seed=6)
    pad = -N % (8 if out == "bf16" else 4)
    D = Guarded((rows, N), DTYPE[out], pad)
    g.bf16gemm_grouped(aligned(A), aligned(B), off, D.t)
    assert D.clean_outside()
    want = torch.cat([A[:1100].double() @ B[0].double(), A[1100:].double() @ B[1].double()])
    assert torch.equal(D.t.double(), want)
    wide, ragged = small(rows, 700, seed=7), aligned(dD)
    dB = Guarded((2, 700, N), DTYPE[out], pad)
    g.bf16gemm_grouped_wgrad(wide, ragged, off, dB.t)
    check_device_error()
    want = torch.stack([wide[:1100].double().t() @ dD[:1100].double(),
                        wide[1100:].double().t() @ dD[1100:].double()])
    assert dB.clean_outside() and torch.equal(dB.t.double(), want.to(DTYPE[out]).double())


@pytest.mark.parametrize("M,N,K", [(700, 77, 64), (1000, 301, 520), (777, 30, 200), (640, 1001, 4096),
                                   (2048, 2049, 512), (600, 258, 1024)])
@pytest.mark.parametrize("cfg", [None, {"kernel": "single_cta", "split": 1},
                                 {"kernel": "single_cta", "split": 3}, {"kernel": "cta_pair", "split": 1},
                                 {"kernel": "cta_pair", "split": 2}])
@pytest.mark.parametrize("more", [0, 4])
def test_dense_bf16(M, N, K, cfg, more):
    A, B = small(M, K, seed=8), aligned(small(K, N, seed=9))
    C = Guarded((M, N), torch.float32, -N % 4 + more)
    st = g.gemm_bf16gemm_config(M, N, K, 1.0, A.data_ptr(), K, B.data_ptr(), B.stride(0), 0.0,
                                C.t.data_ptr(), C.pitch, cfg, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    check_device_error()
    assert C.clean_outside() and torch.equal(C.t.double(), A.double() @ B.double())
