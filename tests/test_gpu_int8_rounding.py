"""Bytes of the int8 quantiser and of layer norm's int8 output, one by one.

The factor 127 / a, a value's product with it and the whole number nearest to that are each rounded to
nearest even, so every byte follows from the fp32 value and its row's largest magnitude: the same along
the rows and transposed, and whatever else is in the row."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, Guarded, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def bytes_of(x):
    """q and scales of the rows of x (float32 or bfloat16), in fp32 operations on the CPU."""
    x = x.float().cpu()
    fine = torch.isfinite(x)
    amax = torch.where(fine, x.abs(), torch.zeros(())).amax(1)
    factor = (torch.tensor(127.0) / amax).clamp_max(2.0 ** 126)
    v = (x * factor[:, None]).round()
    q = torch.where(torch.isnan(v), torch.zeros(()), v).clamp(-127, 127)
    return q.to(torch.int8), (amax / 127).clamp_min(2.0 ** -126)


def rows_of(rows, cols, dtype, seed=0):
    """Normal values; from the second on every third row has many of half its largest magnitude (63.5 steps,
    where the factor was rounded a little more or less), and its largest at the end."""
    v = randn(rows, cols, seed=seed + rows + cols, device="cpu").to(DTYPE[dtype])
    for r in range(1, rows, 3):
        v[r, ::2] = v[r, ::2].sign() * (v[r].abs().amax() / 2)
    return v


# one, two, four chunks a thread, and rows too long for that; few rows and many; with and without vectors
SHAPES = [(4, 100), (40, 127), (400, 256), (400, 300), (400, 512), (350, 1024), (330, 1001), (5, 4096),
          (5, 8192), (5, 8191), (4, 16384), (4, 16001), (4, 20000), (4, 20001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_byte_along_rows_and_transposed(rows, cols, dtype):
    v = rows_of(rows, cols, dtype)
    want, scales = bytes_of(v)
    for turned in (False, True):
        x = Guarded((cols, rows) if turned else (rows, cols), DTYPE[dtype]).set(v.t() if turned else v)
        q, s = Guarded((rows, cols), torch.int8), torch.empty(rows, device="cuda")
        g.int8_quantize(x.t, q.t, s, transpose=turned)
        check_device_error()
        assert torch.equal(s.cpu(), scales)
        assert torch.equal(q.t.cpu(), want)


@pytest.mark.parametrize("cols", [256, 255, 8192, 20000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite_changes_no_other(cols, bad):
    v = rows_of(12, cols, "bf16", seed=5).float()
    v[:, cols // 2] = 0.0
    before, after = (torch.empty(12, cols, dtype=torch.int8, device="cuda") for _ in range(2))
    s = torch.empty(12, device="cuda")
    g.int8_quantize(v.cuda(), before, s)
    v[:, cols // 2] = bad
    g.int8_quantize(v.cuda(), after, s)
    check_device_error()
    want, scales = bytes_of(v)
    assert torch.equal(after.cpu(), want) and torch.equal(s.cpu(), scales)
    before[:, cols // 2] = after[:, cols // 2]
    assert torch.equal(before, after)


# rows in registers and through rings, longer ones, with and without vectors
@pytest.mark.parametrize("rows,dim", [(4, 4096), (9, 1001), (400, 200), (2500, 4096), (9000, 576), (5, 8192),
                                      (3, 16384), (3, 20000), (3, 20001)])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", None)])
def test_layer_norm_rounds_its_unrounded_values_alike(rows, dim, xt, rt):
    x = randn(rows, dim, seed=1, dtype=DTYPE[xt])
    r = None if rt is None else randn(rows, dim, seed=2, scale=3, dtype=DTYPE[rt])
    w, b = 1.0 + randn(dim, seed=3, scale=0.2), randn(dim, seed=4)
    y, q = torch.empty(rows, dim, device="cuda"), torch.empty(rows, dim, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    g.layernorm(x, w, b, residual=r, y=y, q=q, scales=s)
    check_device_error()
    want, scales = bytes_of(y)
    assert torch.equal(s.cpu(), scales)
    assert torch.equal(q.cpu(), want)
    # rows of two values that are each other's negative: y is +-rstd * d, the half of it is a tie
    h = torch.zeros(6, dim, device="cuda")
    h[:, 0::2], h[:, 1::2] = 3.0, -3.0
    h[:, dim - 1] = 0.0 if dim % 2 else -3.0
    gain = torch.full((dim,), 0.5, device="cuda")
    gain[0] = 1.0
    y, q, s = torch.empty(6, dim, device="cuda"), torch.empty(6, dim, dtype=torch.int8, device="cuda"), s[:1].repeat(6)
    g.layernorm(h, gain, y=y, q=q, scales=s)
    check_device_error()
    want, scales = bytes_of(y)
    assert torch.equal(q.cpu(), want) and torch.equal(s.cpu(), scales)
