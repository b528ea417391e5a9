"""gemm_rmsnorm and gemm_rmsnorm_backward against their formulas in fp64.

The kernels compute in fp32.  With n terms summed in at most n / 32 + 32
successive additions (a lane's own and the shuffles; rows that do not fit the
registers: n / 512 a lane), the sum of squares -- all of one sign -- is off by
at most that many units of 2^-24, and rstd by half of it plus the reciprocal
root's two units and the mean's two; three more products make y.  So y is
within (n / 64 + 32) * 2^-24 of itself, plus what h = x + r is rounded by.
"""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, FILL, U32, UBF, Guarded, check_fp8, e4m3_round, randn, up

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def rel(dim):
    return (dim / 64 + 32) * U32


def forward64(x, r, w, eps=EPS):
    h = x.double() + (r.double() if r is not None else 0.0)
    rstd = (h.square().mean(-1) + eps).rsqrt()
    return h, rstd, h * rstd[:, None] * w.double()


ROWS_DIM = [(1, 1), (1, 128), (3, 127), (5, 129), (1, 4096), (7, 1000), (33, 512), (400, 64),
            (700, 200), (1000, 1024), (330, 4096), (320, 5000), (2, 8192), (3, 12288), (2, 16384),
            (3, 16385), (2, 20000), (310, 16392)]


@pytest.mark.parametrize("rows,dim", ROWS_DIM)
@pytest.mark.parametrize("xt,rt,out", [("bf16", "bf16", "fp8"), ("f32", None, "bf16"),
                                       ("bf16", "f32", "f32"), ("f32", "bf16", "fp8")])
def test_forward(rows, dim, xt, rt, out):
    pad = 16 if dim % 8 == 0 else 3
    x = Guarded((rows, dim), DTYPE[xt], pad).set(randn(rows, dim, seed=1))
    r = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad).set(randn(rows, dim, seed=2, scale=3))
    w = 1.0 + randn(dim, seed=3, scale=0.2)
    h = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad)
    rstd = torch.full((rows,), -1.0, device="cuda")
    y = Guarded((rows, dim), DTYPE[out], pad)
    s = Guarded((up(dim), rows), torch.float32, 5) if out == "fp8" else None
    g.rmsnorm(x.t, w, eps=EPS, residual=None if r is None else r.t, h=None if h is None else h.t,
              y=None if out == "fp8" else y.t, q=y.t if out == "fp8" else None,
              scales=None if s is None else s.t, rstd=rstd)
    check_device_error()
    h64, rstd64, y64 = forward64(x.t, None if r is None else r.t, w)
    assert ((rstd.double() - rstd64).abs() <= rel(dim) * rstd64).all()
    for buf in (x, r, h, y, s):
        assert buf is None or buf.clean_outside()
    if h is not None:
        unit = UBF if rt == "bf16" else U32
        assert ((h.t.double() - h64).abs() <= (unit + U32) * h64.abs() + 1e-40).all()
    err = rel(dim) * y64.abs() + 1e-37
    if out == "fp8":
        check_fp8(y.t, s.t, y64, "rows", err)
    else:
        unit = UBF if out == "bf16" else 0.0
        assert ((y.t.double() - y64).abs() <= err + unit * (y64.abs() + err)).all()


@pytest.mark.parametrize("rows,dim", [(4, 4096), (400, 96), (330, 1001), (2, 20000)])
def test_in_place_and_several_outputs(rows, dim):
    # h over the residual and y over x, with q, all from one call
    x, r = randn(rows, dim, seed=4, dtype=torch.bfloat16), randn(rows, dim, seed=5)
    w = 1.0 + randn(dim, seed=6, scale=0.2)
    h64, _, y64 = forward64(x, r, w)
    q = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(up(dim), rows, device="cuda")
    g.rmsnorm(x, w, eps=EPS, residual=r, h=r, y=x, q=q, scales=s)
    check_device_error()
    err = rel(dim) * y64.abs() + 1e-37
    assert ((r.double() - h64).abs() <= U32 * h64.abs()).all()
    assert ((x.double() - y64).abs() <= err + UBF * (y64.abs() + err)).all()
    check_fp8(q, s, y64, "rows", err)


def test_zero_rows_and_zero_values():
    w = torch.ones(256, device="cuda")
    g.rmsnorm(torch.empty(0, 256, device="cuda"), w, y=torch.empty(0, 256, device="cuda"))
    x = torch.zeros(3, 256, device="cuda")
    q = torch.full((3, 256), 1.0, device="cuda").to(torch.float8_e4m3fn)
    s, rstd = torch.empty(2, 3, device="cuda"), torch.empty(3, device="cuda")
    g.rmsnorm(x, w, eps=0.0, y=None, q=q, scales=s)       # 0 * inf: NaN, as the formula has it
    assert torch.isnan(q.float()).all() and (s == 2.0 ** -126).all()
    g.rmsnorm(x, w, eps=1e-6, q=q, scales=s, rstd=rstd)
    assert (q.float() == 0).all() and (s == 2.0 ** -126).all() and torch.allclose(rstd, torch.tensor(1e3))


def test_nan_and_infinity_stay_in_their_row():
    x = randn(6, 1024, seed=7)
    x[1, 5], x[3, 700] = float("nan"), float("inf")
    w = torch.ones(1024, device="cuda")
    y = torch.empty_like(x)
    q, s = torch.empty(6, 1024, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(8, 6, device="cuda")
    g.rmsnorm(x, w, eps=EPS, y=y, q=q, scales=s)
    _, _, y64 = forward64(x, None, w)
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all()
    assert torch.isnan(y[3, 700]) and (y[3, :700] == 0).all()
    good = [0, 2, 4, 5]
    assert ((y[good].double() - y64[good]).abs() <= rel(1024) * y64[good].abs()).all()
    check_fp8(q[good], s[:, good], y64[good], "rows", rel(1024) * y64[good].abs())


def backward64(dy, h, w, rstd, rg):
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    gw, xh = dy * w, h * rstd
    dh = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    if rg is not None:
        dh = dh + rg.double()
    return dh, (dy * xh).sum(0), rstd, gw, xh


@pytest.mark.parametrize("rows,dim", ROWS_DIM)
@pytest.mark.parametrize("dyt,ht,rt,out", [("bf16", "bf16", "bf16", "bf16"),
                                           ("f32", "f32", None, "f32"), ("bf16", "f32", "f32", "f32")])
def test_backward(rows, dim, dyt, ht, rt, out):
    pad = 16 if dim % 8 == 0 else 3
    dy = Guarded((rows, dim), DTYPE[dyt], pad).set(randn(rows, dim, seed=8))
    h = Guarded((rows, dim), DTYPE[ht], pad).set(randn(rows, dim, seed=9, scale=2))
    rg = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad).set(randn(rows, dim, seed=10))
    w = 1.0 + randn(dim, seed=11, scale=0.2)
    rstd = (h.t.float().square().mean(-1) + EPS).rsqrt()
    dh, dw = Guarded((rows, dim), DTYPE[out], pad), Guarded((1, dim), torch.float32, 7)
    g.rmsnorm_backward(dy.t, h.t, w, rstd, dh.t, dw.t[0],
                       residual_grad=None if rg is None else rg.t)
    check_device_error()
    dh64, dw64, r64, gw, xh = backward64(dy.t, h.t, w, rstd, None if rg is None else rg.t)
    assert all(b is None or b.clean_outside() for b in (dy, h, rg, dh, dw))
    # the mean of n signed terms: (n / 32 + 32) units of the sum of magnitudes; then a handful of
    # roundings of the terms that are subtracted and added
    mean_err = (dim / 32 + 40) * U32 * (gw * xh).abs().mean(-1, keepdim=True)
    terms = r64 * (gw.abs() + xh.abs() * (gw * xh).mean(-1, keepdim=True).abs())
    bound = r64 * xh.abs() * mean_err + 6 * U32 * (terms + dh64.abs())
    if out == "bf16":
        bound = bound + UBF * (dh64.abs() + bound)
    assert ((dh.t.double() - dh64).abs() <= bound + 1e-37).all()
    # a column's sum over the rows: at most rows + 64 successive additions
    dw_bound = (rows + 64) * U32 * ((dy.t.double() * xh).abs()).sum(0)
    assert ((dw.t[0].double() - dw64).abs() <= dw_bound + 1e-37).all()


@pytest.mark.parametrize("dim", [64, 640, 4097])
def test_backward_against_differences(dim):
    # central differences of L = sum(dy * y) + sum(c * h) in fp64, along random directions
    rows, step = 5, 1e-4
    x, dy = randn(rows, dim, seed=12), randn(rows, dim, seed=13)
    w, c = 1.0 + randn(dim, seed=14, scale=0.2), randn(rows, dim, seed=15)
    rstd = torch.empty(rows, device="cuda")
    y = torch.empty_like(x)
    g.rmsnorm(x, w, eps=EPS, y=y, rstd=rstd)
    dh, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    g.rmsnorm_backward(dy, x, w, rstd, dh, dw, residual_grad=c)

    def loss(x_, w_):
        h, _, y_ = forward64(x_, None, w_)
        return float((dy.double() * y_).sum() + (c.double() * h).sum())

    for seed in range(3):
        e = randn(rows, dim, seed=20 + seed).double()
        num = (loss(x.double() + step * e, w) - loss(x.double() - step * e, w)) / (2 * step)
        got = float((dh.double() * e).sum())
        # third derivatives of y are O(rstd^2): the difference quotient is good to step^2 of the
        # gradient's size, the gradient to fp32's bound above
        size = float((dh.double() * e).abs().sum())
        assert abs(num - got) <= (10 * step ** 2 + (dim / 32 + 64) * U32) * size + 1e-9 * size
        f = randn(dim, seed=30 + seed).double()
        num = (loss(x.double(), w.double() + step * f) - loss(x.double(), w.double() - step * f)) / (2 * step)
        size = float((dw.double() * f).abs().sum()) + float((dy * y).double().abs().sum())
        assert abs(num - float((dw.double() * f).sum())) <= ((dim / 32 + 128) * U32 + 1e-9) * size


@pytest.mark.parametrize("dim", [768, 10000, 20000])
def test_backward_in_place(dim):
    x, dy, c = randn(40, dim, seed=16), randn(40, dim, seed=17), randn(40, dim, seed=18)
    w, rstd = 1.0 + randn(dim, seed=19, scale=0.2), torch.empty(40, device="cuda")
    g.rmsnorm(x, w, eps=EPS, rstd=rstd)
    dh, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    g.rmsnorm_backward(dy, x, w, rstd, dh, dw, residual_grad=c)
    for which in range(3):  # over dy, h, residual_grad
        args = [dy.clone(), x.clone(), c.clone()]
        dw2 = torch.empty_like(dw)
        g.rmsnorm_backward(args[0], args[1], w, rstd, args[which], dw2, residual_grad=args[2])
        assert torch.equal(args[which], dh) and torch.equal(dw2, dw)


def test_backward_without_weight_gradient_and_without_rows():
    x, dy, c = randn(40, 768, seed=16), randn(40, 768, seed=17), randn(40, 768, seed=18)
    w, rstd = 1.0 + randn(768, seed=19, scale=0.2), torch.empty(40, device="cuda")
    g.rmsnorm(x, w, eps=EPS, rstd=rstd)
    dh, dw = torch.empty_like(x), torch.empty(768, device="cuda")
    g.rmsnorm_backward(dy, x, w, rstd, dh, dw, residual_grad=c)
    over = c.clone()
    g.rmsnorm_backward(dy, x, w, rstd, over, residual_grad=over)
    assert torch.equal(over, dh)
    none = torch.empty(0, 768, device="cuda")
    g.rmsnorm_backward(none, none, w, torch.empty(0, device="cuda"), none, dw)
    assert (dw == 0).all()


def test_same_bits_on_any_stream_and_in_a_graph():
    rows, dim = 1000, 2304
    x, r = randn(rows, dim, seed=21, dtype=torch.bfloat16), randn(rows, dim, seed=22)
    w, dy = 1.0 + randn(dim, seed=23, scale=0.2), randn(rows, dim, seed=24, dtype=torch.bfloat16)
    q, s = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(18, rows, device="cuda")
    h, rstd = torch.empty_like(r), torch.empty(rows, device="cuda")
    dh, dw = torch.empty_like(x), torch.empty(dim, device="cuda")

    def work():
        g.rmsnorm(x, w, eps=EPS, residual=r, h=h, q=q, scales=s, rstd=rstd)
        g.rmsnorm_backward(dy, h, w, rstd, dh, dw, residual_grad=dy)

    outs = (h, q.view(torch.uint8), s, rstd, dh, dw)
    work()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for t in outs:
            t.fill_(0)
        work()
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            work()
        for t in outs:
            t.fill_(0)
        graph.replay()
        stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
