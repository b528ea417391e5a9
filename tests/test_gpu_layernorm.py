"""gemm_layernorm and gemm_layernorm_backward against their formulas in fp64.

The kernels compute in fp32 (unit U = 2^-24).  With n terms summed in at most n / 32 + 40 successive
additions: the sum h = x + r is off by U |h|; the differences d from the rounded mean by U |d|, and
their own mean, which is taken off them, by (n / 32 + 40) U mean|d|; so a value less the mean is off by

    e = U (|h| + mean|h|) + 2 U |d| + (n / 32 + 40) U mean|d|

The variance, a sum of one sign, is off by (n / 32 + 40) U of itself and by 2 U mean|d h|, 1 / sqrt by
half of that and three units; y by four more roundings of its terms.
"""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import DTYPE, U32, UBF, Guarded, check_fp8, randn, up

pytestmark = pytest.mark.gpu
EPS = 1e-5
TYPES = {**DTYPE, "s8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


def forward64(x, r, w, b, eps=EPS):
    """h, mean, rstd, y in fp64, and bounds of the last three."""
    h = x.double() + (r.double() if r is not None else 0.0)
    n = h.shape[1]
    mean = h.mean(-1, keepdim=True)
    d = h - mean
    var = d.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    w = 1.0 if w is None else w.double()
    b = 0.0 if b is None else b.double()
    y = d * rstd * w + b
    ad = d.abs().mean(-1, keepdim=True)
    e = U32 * (h.abs() + h.abs().mean(-1, keepdim=True) + 2 * d.abs() + (n / 32 + 40) * ad)
    rel = (n / 64 + 24) * U32 + U32 * (d * h).abs().mean(-1, keepdim=True) * rstd ** 2
    y_err = rstd * e * abs(w) + (rel + 5 * U32) * (d * rstd * w).abs() + 2 * U32 * abs(b) + 1e-37
    mean_err = (n / 32 + 44) * U32 * h.abs().mean(-1) + 1e-37
    return h, mean[:, 0], rstd[:, 0], y, mean_err, (rel * rstd)[:, 0], y_err


def check_s8(q, s, want, err):
    """q * s must be `want`, known to within err, rounded to whole multiples of the row's largest
    magnitude / 127: half a step, and the three fp32 roundings of the scale and the quotient."""
    amax = want.abs().amax(1)
    off = err.amax(1)
    scale = (amax / 127).clamp_min(2.0 ** -126)
    assert bool(((s.double() - scale).abs() <= off / 127 + 2 * U32 * scale).all()), "scales"
    assert int(q.min()) >= -127
    got = q.double() * s.double()[:, None]
    bound = err + off[:, None] + 4 * U32 * want.abs() + 0.5 * s.double()[:, None] * (1 + 2.0 ** -18)
    assert bool(((got - want).abs() <= bound).all())


ROWS_DIM = [(1, 1), (1, 128), (3, 127), (5, 129), (1, 4096), (7, 1000), (33, 512), (400, 64),
            (700, 200), (1000, 1024), (330, 4096), (320, 5000), (2, 8192), (3, 12288), (2, 16384),
            (3, 16385), (2, 20000), (310, 16392), (40, 33000)]
# rows through the ring: several to a CTA, stages of two to four places
STAGED = [(4000, 1024), (2500, 4096), (1300, 8192), (5000, 520), (6001, 2048), (9001, 1032), (2431, 4104),
          (3001, 6144), (9000, 576)]


def forward(rows, dim, xt, rt, out, pad, mean=0.0, weight=True, bias=True):
    x = Guarded((rows, dim), DTYPE[xt], pad).set(randn(rows, dim, seed=1) + mean)
    r = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad).set(randn(rows, dim, seed=2, scale=3))
    w = 1.0 + randn(dim, seed=3, scale=0.2) if weight else None
    b = randn(dim, seed=4) if bias else None
    h = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad)
    mu, rstd = (Guarded((1, rows), torch.float32, 3) for _ in range(2))
    y = Guarded((rows, dim), TYPES[out], pad)
    eight = out in ("fp8", "s8")
    s = Guarded((up(dim), rows) if out == "fp8" else (1, rows), torch.float32, 5) if eight else None
    g.layernorm(x.t, w, b, eps=EPS, residual=None if r is None else r.t, h=None if h is None else h.t,
                y=None if eight else y.t, q=y.t if eight else None,
                scales=None if s is None else s.t if out == "fp8" else s.t[0], mean=mu.t[0], rstd=rstd.t[0])
    check_device_error()
    h64, m64, r64, y64, m_err, r_err, y_err = forward64(x.t, None if r is None else r.t, w, b)
    for buf in (x, r, h, y, s, mu, rstd):
        assert buf is None or buf.clean_outside()
    assert bool(((mu.t[0].double() - m64).abs() <= m_err).all())
    assert bool(((rstd.t[0].double() - r64).abs() <= r_err + U32 * r64).all())
    if h is not None:
        unit = UBF if rt == "bf16" else 0.0
        assert bool(((h.t.double() - h64).abs() <= (unit + U32) * h64.abs() * (1 + U32) + 1e-40).all())
    if out == "fp8":
        check_fp8(y.t, s.t, y64, "rows", y_err)
    elif out == "s8":
        check_s8(y.t, s.t[0], y64, y_err)
    else:
        unit = UBF if out == "bf16" else 0.0
        assert bool(((y.t.double() - y64).abs() <= y_err + unit * (y64.abs() + y_err)).all())


@pytest.mark.parametrize("rows,dim", ROWS_DIM + STAGED)
@pytest.mark.parametrize("xt,rt,out", [("bf16", "bf16", "s8"), ("f32", None, "bf16"), ("bf16", None, "s8"),
                                       ("bf16", "f32", "f32"), ("f32", "bf16", "fp8"), ("f32", "f32", "s8")])
def test_forward(rows, dim, xt, rt, out):
    forward(rows, dim, xt, rt, out, 16 if dim % 8 == 0 else 3)


@pytest.mark.parametrize("rows,dim,pad", [(9, 1024, 4), (9, 1000, 1), (2500, 4096, 0), (9, 4096, 7)])
@pytest.mark.parametrize("out", ["f32", "s8", "fp8"])
def test_forward_without_weight_or_bias(rows, dim, pad, out):
    forward(rows, dim, "bf16", "bf16", out, pad, weight=False, bias=False)
    forward(rows, dim, "bf16", None, out, pad, bias=False)


@pytest.mark.parametrize("rows,dim", [(4, 100), (3, 4096), (2500, 4096), (2, 20000), (40, 512)])
@pytest.mark.parametrize("mean", [300.0, -30000.0])
def test_mean_far_from_zero(rows, dim, mean):
    # the squares' mean less the mean's square would have no digit left
    forward(rows, dim, "f32", None, "f32", 0, mean=mean)


@pytest.mark.parametrize("rows,dim", [(4, 4096), (400, 96), (330, 1001), (2, 20000), (2500, 4096)])
def test_in_place_and_several_outputs(rows, dim):
    x, r = randn(rows, dim, seed=4, dtype=torch.bfloat16), randn(rows, dim, seed=5)
    w, b = 1.0 + randn(dim, seed=6, scale=0.2), randn(dim, seed=7)
    h64, _, _, y64, _, _, err = forward64(x, r, w, b)
    q, s = torch.empty(rows, dim, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    g.layernorm(x, w, b, eps=EPS, residual=r, h=r, y=x, q=q, scales=s)
    check_device_error()
    assert bool(((r.double() - h64).abs() <= U32 * h64.abs()).all())
    assert bool(((x.double() - y64).abs() <= err + UBF * (y64.abs() + err)).all())
    check_s8(q, s, y64, err)


def test_zero_rows_and_constant_rows():
    w = torch.ones(256, device="cuda")
    g.layernorm(torch.empty(0, 256, device="cuda"), w, y=torch.empty(0, 256, device="cuda"))
    x = torch.full((3, 256), 7.0, device="cuda")
    x[1] = 0.0
    q, s = torch.ones(3, 256, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    mu, rstd, y = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty_like(x)
    g.layernorm(x, w, eps=1e-6, y=y, q=q, scales=s, mean=mu, rstd=rstd)
    assert bool((y == 0).all()) and bool((q == 0).all()) and bool((s == 2.0 ** -126).all())
    assert mu.tolist() == [7.0, 0.0, 7.0] and torch.allclose(rstd, torch.full_like(rstd, 1e3))
    g.layernorm(x, None, torch.full((256,), 2.0, device="cuda"), eps=1e-6, q=q, scales=s)
    assert bool((q == 127).all())
    g.layernorm(x[:, :1].contiguous(), None, eps=1e-6, y=y[:, :1], rstd=rstd)   # rows of one value
    assert bool((y[:, 0] == 0).all())


def test_nan_and_infinity_stay_in_their_row():
    x = randn(6, 1024, seed=7)
    x[1, 5], x[3, 700] = float("nan"), float("inf")
    y, q, s = torch.empty_like(x), torch.empty(6, 1024, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    rstd = torch.empty(6, device="cuda")
    g.layernorm(x, None, eps=EPS, y=y, q=q, scales=s, rstd=rstd)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all() and torch.isnan(rstd[[1, 3]]).all()
    assert bool((q[[1, 3]] == 0).all()) and bool((s[[1, 3]] == 2.0 ** -126).all())
    good = [0, 2, 4, 5]
    _, _, _, y64, _, _, err = forward64(x[good], None, None, None)
    assert bool(((y[good].double() - y64).abs() <= err).all())
    check_s8(q[good], s[good], y64, err)


def backward64(dy, h, w, mean, rstd, rg):
    dy, h, mean, rstd = dy.double(), h.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (h - mean) * rstd
    gw = dy * w.double() if w is not None else dy
    dh = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    if rg is not None:
        dh = dh + rg.double()
    return dh, (dy * xh).sum(0), dy.sum(0), rstd, gw, xh


def backward(rows, dim, dyt, ht, rt, out, pad, weight=True):
    dy = Guarded((rows, dim), DTYPE[dyt], pad).set(randn(rows, dim, seed=8))
    h = Guarded((rows, dim), DTYPE[ht], pad).set(randn(rows, dim, seed=9, scale=2) + 1.0)
    rg = None if rt is None else Guarded((rows, dim), DTYPE[rt], pad).set(randn(rows, dim, seed=10))
    w = 1.0 + randn(dim, seed=11, scale=0.2) if weight else None
    mean = h.t.float().mean(-1)
    rstd = ((h.t.float() - mean[:, None]).square().mean(-1) + EPS).rsqrt()
    dh = Guarded((rows, dim), DTYPE[out], pad)
    dw, db = (Guarded((1, dim), torch.float32, 7) for _ in range(2))
    more = dict(residual_grad=None if rg is None else rg.t)
    g.layernorm_backward(dy.t, h.t, w, mean, rstd, dh.t, dw.t[0], db.t[0], **more)
    check_device_error()
    dh64, dw64, db64, r64, gw, xh = backward64(dy.t, h.t, w, mean, rstd, None if rg is None else rg.t)
    assert all(b is None or b.clean_outside() for b in (dy, h, rg, dh, dw, db))
    # means of n signed terms: (n / 32 + 40) units of the sum of magnitudes (xh itself two units);
    # then a handful of roundings of the terms that are subtracted and added
    unit = (dim / 32 + 44) * U32
    err_g, err_x = unit * gw.abs().mean(-1, keepdim=True), unit * (gw * xh).abs().mean(-1, keepdim=True)
    terms = r64 * (gw.abs() + gw.mean(-1, keepdim=True).abs() + xh.abs() * (gw * xh).mean(-1, keepdim=True).abs())
    bound = r64 * (err_g + xh.abs() * err_x) + 8 * U32 * (terms + dh64.abs())
    if out == "bf16":
        bound = bound + UBF * (dh64.abs() + bound)
    assert bool(((dh.t.double() - dh64).abs() <= bound + 1e-37).all())
    # a column's sum over the rows: at most rows + 64 successive additions
    assert bool(((dw.t[0].double() - dw64).abs() <= (rows + 68) * U32 * (dy.t.double() * xh).abs().sum(0) + 1e-37).all())
    assert bool(((db.t[0].double() - db64).abs() <= (rows + 64) * U32 * dy.t.double().abs().sum(0) + 1e-37).all())
    # each alone gives the same bits; neither leaves them as they are
    for one in ("dweight", "dbias"):
        v = torch.full((dim,), 3.0, device="cuda")
        g.layernorm_backward(dy.t, h.t, w, mean, rstd, dh.t, **{one: v}, **more)
        assert torch.equal(v, (dw if one == "dweight" else db).t[0])
    first = dh.t.clone()
    g.layernorm_backward(dy.t, h.t, w, mean, rstd, dh.t, **more)
    assert torch.equal(dh.t, first)


@pytest.mark.parametrize("rows,dim", ROWS_DIM + STAGED)
@pytest.mark.parametrize("dyt,ht,rt,out", [("bf16", "bf16", "bf16", "bf16"), ("f32", "f32", None, "f32"),
                                           ("bf16", "f32", "f32", "f32"), ("f32", "bf16", "bf16", "bf16")])
def test_backward(rows, dim, dyt, ht, rt, out):
    backward(rows, dim, dyt, ht, rt, out, 16 if dim % 8 == 0 else 3)


@pytest.mark.parametrize("rows,dim,pad", [(9, 1024, 4), (9, 1000, 1), (2500, 4096, 0), (2, 20000, 0)])
def test_backward_without_weight(rows, dim, pad):
    backward(rows, dim, "bf16", "bf16", "f32", "f32", pad, weight=False)


@pytest.mark.parametrize("rows,dim", [(4, 1024), (330, 1001), (2, 20000), (2500, 4096)])
def test_backward_in_place(rows, dim):
    dy, h, rg = (randn(rows, dim, seed=s) for s in (1, 2, 3))
    w = 1.0 + randn(dim, seed=4, scale=0.2)
    mean = h.mean(-1)
    rstd = ((h - mean[:, None]).square().mean(-1) + EPS).rsqrt()
    want, dw, db = torch.empty_like(h), torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    g.layernorm_backward(dy, h, w, mean, rstd, want, dw, db, residual_grad=rg)
    for k in range(3):
        a = [dy.clone(), h.clone(), rg.clone()]
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        g.layernorm_backward(a[0], a[1], w, mean, rstd, a[k], dw2, db2, residual_grad=a[2])
        assert torch.equal(a[k], want) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_backward_no_rows():
    e, v = torch.empty(0, 64, device="cuda"), torch.empty(0, device="cuda")
    dw, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    g.layernorm_backward(e, e, None, v, v, e, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_backward_against_differences():
    rows, dim = 5, 40
    x, dy = randn(rows, dim, seed=1) + 0.5, randn(rows, dim, seed=2)
    w, b = 1.0 + randn(dim, seed=3, scale=0.2), randn(dim, seed=4)
    mean, rstd, dh = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    dw, db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    g.layernorm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    g.layernorm_backward(dy, x, w, mean, rstd, dh, dw, db)

    def loss(x, w, b):
        d = x - x.mean(-1, keepdim=True)
        return ((d * (d.square().mean(-1, keepdim=True) + EPS).rsqrt() * w + b) * dy.double()).sum(-1)

    x, w, b = x.double(), w.double(), b.double()
    step = 1e-5
    scale = float(dy.abs().sum(1).max())
    # differences in fp64: step^2 times a third derivative, 2^-52 / step; the kernels' fp32: some 100 U
    tol = (1e-8 + 200 * U32) * scale
    for i in range(dim):
        e = torch.zeros(dim, dtype=torch.float64, device="cuda")
        e[i] = step
        assert bool((((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * step) - dh[:, i]).abs() <= tol).all())
        assert abs(float((loss(x, w + e, b) - loss(x, w - e, b)).sum()) / (2 * step) - float(dw[i])) <= rows * tol
        assert abs(float((loss(x, w, b + e) - loss(x, w, b - e)).sum()) / (2 * step) - float(db[i])) <= rows * tol


def test_streams_and_graph():
    """Forward and backward on two streams at once, and captured and replayed on other values."""
    rows, dim = 700, 1024
    w, b = 1.0 + randn(dim, seed=1, scale=0.2), randn(dim, seed=2)

    class Work:
        def __init__(self, seed):
            self.x, self.dy = randn(rows, dim, seed=seed), randn(rows, dim, seed=seed + 1)
            self.y, self.dh = torch.empty_like(self.x), torch.empty_like(self.x)
            self.mean, self.rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            self.dw, self.db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")

        def run(self):
            g.layernorm(self.x, w, b, eps=EPS, y=self.y, mean=self.mean, rstd=self.rstd)
            g.layernorm_backward(self.dy, self.x, w, self.mean, self.rstd, self.dh, self.dw, self.db)

        def check(self):
            _, _, _, y64, _, _, err = forward64(self.x, None, w, b)
            assert bool(((self.y.double() - y64).abs() <= err).all())
            _, dw64, db64, _, _, xh = backward64(self.dy, self.x, w, self.mean, self.rstd, None)
            unit = (rows + 68) * U32
            assert bool(((self.dw.double() - dw64).abs() <= unit * (self.dy * xh).abs().sum(0)).all())
            assert bool(((self.db.double() - db64).abs() <= unit * self.dy.double().abs().sum(0)).all())

    works, streams = [Work(1), Work(3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, s in zip(works, streams):
            with torch.cuda.stream(s):
                k.run()
    torch.cuda.synchronize()
    for k in works:
        k.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        works[0].run()
    for seed in (21, 22):
        works[0].x.copy_(randn(rows, dim, seed=seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        works[0].check()
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh):
        with pytest.raises(g.GemmError) as e:
            works[1].run()
    assert g.STATUS[e.value.status] == "GEMM_ERR_NO_MEMORY"
    check_device_error()
    for s in streams:
        g.gemm_release_stream(s.cuda_stream)


def test_rows_past_two_to_the_31_elements():
    dim, rows = 1 << 16, (1 << 15) + 9
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    x[: rows - 9].zero_()
    x[rows - 9:] = randn(9, dim, seed=1, dtype=torch.bfloat16)
    tail = x[rows - 9:].clone()
    g.layernorm(x, None, eps=EPS, y=x)
    _, _, _, y64, _, _, err = forward64(tail, None, None, None)
    assert bool(((x[rows - 9:].double() - y64).abs() <= err + UBF * (y64.abs() + err)).all())
    assert bool((x[: rows - 9] == 0).all())
