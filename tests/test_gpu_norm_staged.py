"""The norm and its gradients on many rows, where rows come through a ring in
shared memory: sizes at which every CTA takes six rows or more through a ring of
two to four, so that each of its places is filled again, and the last round is
not full.  Against the formulas in fp64, with the bounds of test_gpu_norm.py.

Also the row quantiser where a thread takes a second unit and a second turn.
"""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, check_fp8, up

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed, scale=1.0, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def rel(dim):
    return (dim / 64 + 32) * U32


# (rows, dim): on 152 SMs a ring takes 152 to 2432 CTAs, the more the shorter the row
SIZES = [(15000, 520), (15001, 1000), (8001, 2048), (4001, 4096), (3001, 5000), (2001, 8192)]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("xt,rt,out", [("bf16", None, "bf16"), ("f32", None, "fp8"), ("bf16", "bf16", "fp8"),
                                       ("bf16", "f32", "f32"), ("f32", "bf16", "fp8"), ("f32", "f32", "bf16")])
def test_forward(rows, dim, xt, rt, out):
    x = Guarded((rows, dim), DTYPE[xt], 16).set(randn(rows, dim, seed=1))
    r = None if rt is None else Guarded((rows, dim), DTYPE[rt], 8).set(randn(rows, dim, seed=2, scale=3))
    w = 1.0 + randn(dim, seed=3, scale=0.2)
    h = None if rt is None else Guarded((rows, dim), DTYPE[rt], 16)
    rstd = torch.full((rows,), -1.0, device="cuda")
    y, fp8 = Guarded((rows, dim), DTYPE[out], 16), out == "fp8"
    s = Guarded((up(dim), rows), torch.float32, 5) if fp8 else None
    g.rmsnorm(x.t, w, eps=EPS, residual=r and r.t, h=h and h.t, y=None if fp8 else y.t,
              q=y.t if fp8 else None, scales=s and s.t, rstd=rstd)
    check_device_error()
    for buf in (x, r, h, y, s):
        assert buf is None or buf.clean_outside()
    h64 = x.t.double() + (r.t.double() if r else 0.0)
    rstd64 = (h64.square().mean(-1) + EPS).rsqrt()
    assert ((rstd.double() - rstd64).abs() <= rel(dim) * rstd64).all()
    if h is not None:
        unit = UBF if rt == "bf16" else U32
        assert ((h.t.double() - h64).abs() <= (unit + U32) * h64.abs() + 1e-40).all()
    y64 = h64 * rstd64[:, None] * w.double()
    err = rel(dim) * y64.abs() + 1e-37
    if fp8:
        check_fp8(y.t, s.t, y64, "rows", err)
    else:
        unit = UBF if out == "bf16" else 0.0
        assert ((y.t.double() - y64).abs() <= err + unit * (y64.abs() + err)).all()


@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_in_place(rows, dim):
    x, r = randn(rows, dim, seed=4, dtype=torch.bfloat16), randn(rows, dim, seed=5)
    w = 1.0 + randn(dim, seed=6, scale=0.2)
    h64 = x.double() + r.double()
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.double()
    g.rmsnorm(x, w, eps=EPS, residual=r, h=r, y=x)
    check_device_error()
    err = rel(dim) * y64.abs() + 1e-37
    assert ((r.double() - h64).abs() <= U32 * h64.abs()).all()
    assert ((x.double() - y64).abs() <= err + UBF * (y64.abs() + err)).all()


def check_gradients(dh, dw, dy, h, w, rstd, rg, out):
    rows, dim = dy.shape
    dy, r, w = dy.double(), rstd.double()[:, None], w.double()
    xh = h.double() * r
    gw = dy * w
    mean = (gw * xh).mean(-1, keepdim=True)
    dh64 = r * (gw - xh * mean)
    if rg is not None:
        dh64 = dh64 + rg.double()
    mean_err = (dim / 32 + 40) * U32 * (gw * xh).abs().mean(-1, keepdim=True)
    terms = r * (gw.abs() + xh.abs() * mean.abs())
    bound = r * xh.abs() * mean_err + 6 * U32 * (terms + dh64.abs())
    if out == "bf16":
        bound = bound + UBF * (dh64.abs() + bound)
    assert ((dh.double() - dh64).abs() <= bound + 1e-37).all()
    dw_bound = (rows + 64) * U32 * (dy * xh).abs().sum(0)
    assert ((dw.double() - (dy * xh).sum(0)).abs() <= dw_bound + 1e-37).all()


TYPES = [(a, b, c) for a in ("bf16", "f32") for b in ("bf16", "f32") for c in (None, "bf16", "f32")]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dyt,ht,rt", TYPES)
def test_backward(rows, dim, dyt, ht, rt):
    out = ht
    dy = Guarded((rows, dim), DTYPE[dyt], 16).set(randn(rows, dim, seed=8))
    h = Guarded((rows, dim), DTYPE[ht], 8).set(randn(rows, dim, seed=9, scale=2))
    rg = None if rt is None else Guarded((rows, dim), DTYPE[rt], 16).set(randn(rows, dim, seed=10))
    w = 1.0 + randn(dim, seed=11, scale=0.2)
    rstd = (h.t.float().square().mean(-1) + EPS).rsqrt()
    dh, dw = Guarded((rows, dim), DTYPE[out], 16), Guarded((1, dim), torch.float32, 7)
    g.rmsnorm_backward(dy.t, h.t, w, rstd, dh.t, dw.t[0], residual_grad=rg and rg.t)
    check_device_error()
    assert all(b is None or b.clean_outside() for b in (dy, h, rg, dh, dw))
    check_gradients(dh.t, dw.t[0], dy.t, h.t, w, rstd, rg and rg.t, out)


@pytest.mark.parametrize("rows,dim", [(15001, 1000), (4001, 4096), (2001, 8192)])
@pytest.mark.parametrize("which", ["dy", "h", "residual_grad"])
def test_backward_in_place(rows, dim, which):
    args = {"dy": randn(rows, dim, seed=12), "h": randn(rows, dim, seed=13, scale=2),
            "residual_grad": randn(rows, dim, seed=14)}
    w = 1.0 + randn(dim, seed=15, scale=0.2)
    rstd = (args["h"].square().mean(-1) + EPS).rsqrt()
    before, dw = {k: v.clone() for k, v in args.items()}, torch.empty(dim, device="cuda")
    g.rmsnorm_backward(args["dy"], args["h"], w, rstd, args[which], dw, residual_grad=args["residual_grad"])
    check_device_error()
    check_gradients(args[which], dw, before["dy"], before["h"], w, rstd, before["residual_grad"], "f32")
    assert all(torch.equal(args[k], before[k]) for k in args if k != which)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(5001, 1280), (9001, 1536), (9001, 1032), (9001, 1031)])
def test_row_quantiser_with_many_units(rows, cols, dtype):
    x = randn(rows, cols, seed=16, dtype=DTYPE[dtype]) * torch.exp(3 * randn(1, cols, seed=17)).to(DTYPE[dtype])
    q, s = Guarded((rows, cols), torch.float8_e4m3fn, -cols % 16), Guarded((up(cols), rows), torch.float32, 3)
    g.fp8_quantize(x, q.t, s.t)
    check_device_error()
    assert q.clean_outside() and s.clean_outside()
    want = x.double()
    check_fp8(q.t, s.t, want, "rows", torch.zeros_like(want))
