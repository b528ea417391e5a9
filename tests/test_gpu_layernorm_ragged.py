"""Layer norm of rows that 16-byte pieces do not fit, at the row plans that test_gpu_layernorm.py's sizes do not
reach: two and four chunks a thread over several warps, several rows to a CTA's loop, and rows that are
looked at again after the sums (the gradient of 4097 to 8192 elements).  The bounds are that file's."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from ops_ref import randn
from test_gpu_layernorm import EPS, backward, forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


# (rows, dim, elements between the rows); 9 x 8192 and 1500 x 2048 are ragged by their pitch alone
SHAPES = [(4000, 5001, 3), (3, 5001, 3), (3, 8191, 3), (700, 8191, 1), (3, 12289, 3), (320, 12289, 7), (4000, 1999, 3),
          (2000, 300, 3), (9000, 300, 1), (9, 8192, 1), (1500, 2048, 1), (320, 20001, 3)]


@pytest.mark.parametrize("rows,dim,pad", SHAPES)
@pytest.mark.parametrize("xt,rt,out", [("bf16", "bf16", "s8"), ("f32", None, "fp8"), ("bf16", None, "bf16"),
                                       ("f32", "f32", "f32")])
def test_forward(rows, dim, pad, xt, rt, out):
    forward(rows, dim, xt, rt, out, pad)


@pytest.mark.parametrize("rows,dim,pad", SHAPES)
@pytest.mark.parametrize("dyt,ht,rt,out", [("bf16", "bf16", "bf16", "bf16"), ("f32", "f32", None, "f32"),
                                           ("bf16", "f32", "f32", "f32")])
def test_backward(rows, dim, pad, dyt, ht, rt, out):
    backward(rows, dim, dyt, ht, rt, out, pad)


@pytest.mark.parametrize("rows,dim", [(4000, 5001), (3, 8191), (2000, 300)])
def test_backward_in_place(rows, dim):
    dy, h, rg = (randn(rows, dim, seed=s, dtype=torch.bfloat16) for s in (1, 2, 3))
    w = 1.0 + randn(dim, seed=4, scale=0.2)
    mean = h.float().mean(-1)
    rstd = ((h.float() - mean[:, None]).square().mean(-1) + EPS).rsqrt()
    want, dw, db = torch.empty_like(h), torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    g.layernorm_backward(dy, h, w, mean, rstd, want, dw, db, residual_grad=rg)
    for k in range(3):
        a = [dy.clone(), h.clone(), rg.clone()]
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        g.layernorm_backward(a[0], a[1], w, mean, rstd, a[k], dw2, db2, residual_grad=a[2])
        assert torch.equal(a[k], want) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("rows,dim", [(4000, 5001), (3, 8191), (3, 12289)])
def test_forward_in_place(rows, dim):
    x, r = randn(rows, dim, seed=4, dtype=torch.bfloat16), randn(rows, dim, seed=5)
    w, b = 1.0 + randn(dim, seed=6, scale=0.2), randn(dim, seed=7)
    h, y = torch.empty_like(r), torch.empty_like(x)
    g.layernorm(x, w, b, eps=EPS, residual=r, h=h, y=y)
    g.layernorm(x, w, b, eps=EPS, residual=r, h=r, y=x)
    assert torch.equal(h, r) and torch.equal(y, x)
