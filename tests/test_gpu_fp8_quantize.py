"""gemm_fp8_quantize against its definition in fp64: scales within two fp32
units of the blocks' largest magnitude / 448, and every value E4M3's nearest to
within the few fp32 roundings before it (see ops_ref.check_fp8)."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, Guarded, check_fp8, randn, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


SIZES = [(1, 1), (1, 128), (128, 1), (1, 4096), (127, 129), (128, 128), (129, 257), (300, 1000),
         (1999, 300), (16, 8192), (1024, 1536), (5, 100000), (70000, 3)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,pad,off", [("bf16", 0, 0), ("f32", 8, 0), ("bf16", 3, 1)])
def test_quantize(rows, cols, block, transpose, dtype, pad, off):
    x = Guarded((rows, cols), DTYPE[dtype], pad, off).set(
        randn(rows, cols, seed=rows + cols) * torch.exp(3 * randn(1, cols, seed=5)))
    qr, qc = (cols, rows) if transpose else (rows, cols)
    q = Guarded((qr, qc), torch.float8_e4m3fn, (-qc) % 16 if pad != 3 else 5, off)
    s = Guarded((up(qc), up(qr) if block == "tiles" else qr), torch.float32, pad)
    g.fp8_quantize(x.t, q.t, s.t, block=block, transpose=transpose)
    check_device_error()
    assert x.clean_outside() and q.clean_outside() and s.clean_outside()
    want = x.t.double().t() if transpose else x.t.double()
    check_fp8(q.t, s.t, want.contiguous(), block, torch.zeros_like(want))


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("transpose", [False, True])
def test_special_values(block, transpose):
    x = randn(256, 384, seed=1)
    x[0, 0], x[1, 130], x[130, 7], x[255, 383] = (float("nan"), float("inf"), -float("inf"),
                                                   float("nan"))
    x[:, 256:] = 0.0            # blocks of zeros
    x[3, 5] = 1e-42             # below the normal range
    x[128:, 128:256] *= 1e-43   # blocks whose scale is the smallest one
    x[64:100, 20] = 3e38
    q = torch.empty((384, 256) if transpose else (256, 384), dtype=torch.float8_e4m3fn, device="cuda")
    qr, qc = q.shape
    s = torch.empty(up(qc), up(qr) if block == "tiles" else qr, device="cuda")
    g.fp8_quantize(x, q, s, block=block, transpose=transpose)
    want = (x.t() if transpose else x).double().contiguous()
    # below 2^-126 the fp32 products may lose bits: one subnormal unit of the scaled value
    check_fp8(q, s, want, block, torch.full_like(want, 2.0 ** -149))


def test_integers_and_powers_of_two_are_exact():
    # a largest magnitude of 448 gives scale 1, and small integers are E4M3 values
    x = torch.randint(-16, 17, (256, 512), generator=torch.Generator().manual_seed(3)).float().cuda()
    x[:, ::128] = 448.0
    q, s = torch.empty(256, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, 256, device="cuda")
    g.fp8_quantize(x, q, s)
    assert (s == 1.0).all() and torch.equal(q.float(), x)
    g.fp8_quantize(x * 2.0 ** 20, q, s)
    assert (s == 2.0 ** 20).all() and torch.equal(q.float(), x)


def test_transposed_is_the_transpose_quantised():
    x = randn(700, 900, seed=4, dtype=torch.bfloat16)
    for block in ("rows", "tiles"):
        a = torch.empty(900, 700, dtype=torch.float8_e4m3fn, device="cuda")
        sa = torch.empty(6, 8 if block == "tiles" else 900, device="cuda")
        b, sb = torch.empty_like(a), torch.empty_like(sa)
        g.fp8_quantize(x, a, sa, block=block, transpose=True)
        g.fp8_quantize(x.t().contiguous(), b, sb, block=block)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa, sb)


def test_empty():
    q, s = torch.empty(0, 128, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, 0, device="cuda")
    g.fp8_quantize(torch.empty(0, 128, device="cuda"), q, s)
    check_device_error()
