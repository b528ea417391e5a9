"""The quantiser reads nothing past a row's end, also where the row's pitch is made
for 16-byte pieces (so that tiles come by TMA) and the row ends inside one: the
bytes that follow are large numbers, which would set the scales."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, Guarded, check_fp8, randn, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


@pytest.mark.parametrize("rows,cols", [(1, 3), (130, 1), (127, 129), (300, 1001), (257, 254), (1000, 643)])
@pytest.mark.parametrize("block,transpose", [("rows", False), ("rows", True), ("tiles", False), ("tiles", True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [0, 32])
def test_quantiser(rows, cols, block, transpose, dtype, more):
    x = Guarded((rows, cols), DTYPE[dtype], -cols % 8 + more).set(randn(rows, cols, seed=rows))
    qr, qc = (cols, rows) if transpose else (rows, cols)
    q = Guarded((qr, qc), torch.float8_e4m3fn, -qc % 16 + more)
    s = Guarded((up(qc), up(qr) if block == "tiles" else qr), torch.float32, 1)
    g.fp8_quantize(x.t, q.t, s.t, block=block, transpose=transpose)
    check_device_error()
    assert x.clean_outside() and q.clean_outside() and s.clean_outside()
    want = (x.t.t() if transpose else x.t).double().contiguous()
    check_fp8(q.t, s.t, want, block, torch.zeros_like(want))
