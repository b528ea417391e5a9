"""The router, the pairs sorted by expert, and the experts' rows there and back, against plain forms in
64 bits.

Bounds.  fp32 rounds by at most U = 2^-24 of the value, bf16 by 2^-8.  A share exp(l - m) / sum: the
difference is off by |l - m| U, expf by 2 ulp (4 U), the sum by its terms' errors -- the largest term is
1, and |x| e^-|x| <= 1/e -- and G/32 + 5 additions, the quotient and its use by 2 U: (|l - m| + 64) U
covers it for G <= 1024.  Sums of products: as many U of the summed magnitudes as additions follow one
another."""
import pytest
import torch

from ops_ref import DTYPE, FILL, Guarded, U32, UBF, randn

pytestmark = pytest.mark.gpu
I32 = torch.int32
NEG = float("-inf")


def half_step(dtype):
    return U32 if dtype == torch.float32 else UBF


def top_of(l, top):
    """The largest of each row of fp64 logits, one after the other, the first of equal ones."""
    left = torch.where(torch.isnan(l), NEG, l)
    out = []
    for _ in range(top):
        best = left.amax(1, keepdim=True)
        at = (left == best).int().argmax(1, keepdim=True)
        out.append(torch.where(best > NEG, at, -1))
        left = left.scatter(1, at, NEG)
    return torch.cat(out, 1) if out else torch.zeros(l.shape[0], 0, dtype=torch.long, device=l.device)


def shares(l):
    m = l.amax(1, keepdim=True)
    x = torch.where(torch.isinf(m), NEG, l - m)
    e = x.exp()
    return torch.nan_to_num(e / e.sum(1, keepdim=True)), x


def logits_for(rows, G, kind, seed=0):
    l = randn(rows, G, seed=seed, scale=4.0, device="cpu")
    if kind == "ties":
        l = l.round()
    if kind == "masked":   # some experts, whole rows, all but one of a row
        l[torch.rand(rows, G, generator=torch.Generator().manual_seed(seed)) < 0.6] = NEG
        l[::5] = NEG
        if rows > 1:
            l[1] = NEG
            l[1, G - 1] = -3.0
    if kind == "lowest":   # the type's lowest value is a value like any other
        l[:, ::2] = torch.finfo(torch.float32).min
        l[::3] = torch.finfo(torch.float32).min
    if kind == "far":
        l *= 25.0
    return l


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("rows,G,top,dtype,kind,pad", [
    (1, 1, 1, "f32", "plain", 0), (7, 2, 2, "f32", "plain", 3), (16, 64, 8, "f32", "plain", 0),
    (33, 60, 6, "bf16", "ties", 1), (1000, 32, 1, "f32", "ties", 0), (501, 128, 4, "bf16", "masked", 0),
    (77, 33, 32, "f32", "masked", 2), (40, 256, 8, "f32", "lowest", 0), (300, 384, 8, "f32", "far", 0),
    (65, 1024, 32, "f32", "plain", 0), (19, 1000, 7, "bf16", "ties", 5), (20000, 256, 8, "f32", "plain", 0)])
def test_route(gemm_lib, cuda_device, rows, G, top, dtype, kind, pad, normalize):
    buf = Guarded((rows, G), DTYPE[dtype], pad, off=1)
    buf.set(logits_for(rows, G, kind))
    expert, weight = Guarded((rows, top), I32, 0, 1), Guarded((rows, top), torch.float32, 0, 1)
    gemm_lib.expert_route(buf.t, expert.t, weight.t, normalize=normalize)
    l = buf.t.double()
    want = top_of(l, top)
    assert torch.equal(expert.t.long(), want)
    p, x = shares(l)
    real = want >= 0
    w = torch.where(real, p.gather(1, want.clamp_min(0)), 0.0)
    far = torch.where(real, x.gather(1, want.clamp_min(0)).abs(), 0.0)
    if normalize:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    # a share below the normal numbers may be flushed; of the normalised ones, each part may be
    assert bool(((weight.t.double() - w).abs() <= (far + 64) * U32 * w + 2.0 ** -125).all())
    assert expert.clean_outside() and weight.clean_outside()


def test_route_nan_and_infinity(gemm_lib, cuda_device):
    nan, inf = float("nan"), float("inf")
    l = torch.tensor([[1.0, nan, 3.0, 2.0], [nan, nan, nan, nan], [1.0, inf, 0.0, NEG],
                      [nan, NEG, NEG, 5.0]], device="cuda")
    e, w = torch.empty(4, 2, dtype=I32, device="cuda"), torch.empty(4, 2, device="cuda")
    gemm_lib.expert_route(l, e, w)
    assert e.tolist() == [[2, 3], [-1, -1], [1, 0], [3, -1]]
    assert torch.isnan(w[0]).all() and w[1].tolist() == [0.0, 0.0] and torch.isnan(w[2]).all()
    assert torch.isnan(w[3, 0]) and w[3, 1] == 0.0
    gemm_lib.expert_route(l, e, w, normalize=True)   # the weights the NaN does not enter
    want = torch.softmax(torch.tensor([3.0, 2.0], dtype=torch.float64), 0).cuda()
    assert bool(((w[0].double() - want).abs() <= 64 * U32).all())
    assert w[3].tolist() == [1.0, 0.0]


def route_grad(l, e, dw, normalize):
    """(gradient, magnitude of its terms) from the formula, in fp64."""
    p, x = shares(l)
    G = l.shape[1]
    real = (e >= 0) & (e < G)
    at = torch.where(real, e.long(), 0)
    pj = torch.where(real, p.gather(1, at), 0.0)
    dw = torch.where(real, dw.double(), 0.0)
    if normalize:
        pj = torch.nan_to_num(pj / pj.sum(1, keepdim=True))
        dot, mag = (pj * dw).sum(1, keepdim=True), (pj * dw.abs()).sum(1, keepdim=True)
        out, m = torch.zeros_like(l), torch.zeros_like(l)
        return (out.scatter_add(1, at, torch.where(real, pj * (dw - dot), 0.0)),
                m.scatter_add(1, at, torch.where(real, pj * (dw.abs() + mag), 0.0)), x)
    g = torch.zeros_like(l).scatter_add(1, at, dw)
    ga = torch.zeros_like(l).scatter_add(1, at, dw.abs())
    return p * (g - (pj * dw).sum(1, keepdim=True)), p * (ga + (pj * dw.abs()).sum(1, keepdim=True)), x


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("rows,G,top,dtype,out,kind", [
    (1, 1, 1, "f32", "f32", "plain"), (16, 64, 8, "f32", "f32", "plain"), (33, 60, 6, "bf16", "bf16", "ties"),
    (100, 33, 32, "f32", "bf16", "masked"), (40, 256, 8, "f32", "f32", "lowest"),
    (300, 384, 8, "f32", "f32", "far"), (65, 1024, 32, "f32", "f32", "plain")])
def test_route_backward(gemm_lib, cuda_device, rows, G, top, dtype, out, kind, normalize):
    g = gemm_lib
    l = logits_for(rows, G, kind).to(DTYPE[dtype]).cuda()
    e, w = torch.empty(rows, top, dtype=I32, device="cuda"), torch.empty(rows, top, device="cuda")
    g.expert_route(l, e, w, normalize=normalize)
    dw = randn(rows, top, seed=1)
    dl = Guarded((rows, G), DTYPE[out], 3, off=1)
    g.expert_route_backward(l, e, dw, dl.t, normalize=normalize)
    want, mag, x = route_grad(l.double(), e, dw, normalize)
    far = torch.where(torch.isfinite(x), x.abs(), 0.0).clamp_max(110.0)
    # both products and the dot carry a share's error each
    err = (3 * far.amax(1, keepdim=True) + 200) * U32 * mag
    assert bool(((dl.t.double() - want).abs() <= err + half_step(DTYPE[out]) * (want.abs() + err) + 2.0 ** -125).all())
    assert dl.clean_outside()


@pytest.mark.parametrize("normalize", [False, True])
def test_route_backward_against_differences(gemm_lib, cuda_device, normalize):
    g = gemm_lib
    rows, G, top = 9, 20, 5
    l, dw = randn(rows, G, seed=3), randn(rows, top, seed=4)
    e, w = torch.empty(rows, top, dtype=I32, device="cuda"), torch.empty(rows, top, device="cuda")
    g.expert_route(l, e, w, normalize=normalize)
    dl = g.expert_route_backward(l, e, dw, torch.empty_like(l), normalize=normalize).double()

    def loss(v):   # the chosen experts' weights for fp64 logits
        p, _ = shares(v)
        p = p.gather(1, e.long())
        return ((p / p.sum(1, keepdim=True) if normalize else p) * dw.double()).sum(1)

    step = 1e-5
    for i in range(G):
        d = torch.zeros(G, dtype=torch.float64, device="cuda")
        d[i] = step
        diff = (loss(l.double() + d) - loss(l.double() - d)) / (2 * step)
        # differences: step^2 times the third derivative (below 10), and 2^-52 / step
        assert bool(((dl[:, i] - diff).abs() <= 1e-9 + 1e-10 + 400 * U32 * dw.abs().sum(1).double()).all())


def test_route_backward_edges(gemm_lib, cuda_device):
    g = gemm_lib
    l = randn(3, 8, seed=1)
    # the same expert twice, ids that name none
    e = torch.tensor([[2, 2, 5], [-1, 8, 3], [-1, -7, 1 << 30]], dtype=I32, device="cuda")
    dw = randn(3, 3, seed=2)
    for normalize in (False, True):
        dl = g.expert_route_backward(l, e, dw, torch.empty_like(l), normalize=normalize)
        if normalize:   # the sum runs over choices, the same expert twice counts twice
            p, _ = shares(l.double())
            pj = p[0, e[0].long()]
            pj = pj / pj.sum()
            want = torch.zeros(8, dtype=torch.float64, device="cuda")
            want.index_add_(0, e[0].long(), pj * (dw[0].double() - (pj * dw[0].double()).sum()))
            assert bool(((dl[0].double() - want).abs() <= 400 * U32).all())
        else:
            want, mag, _ = route_grad(l.double(), e, dw, False)
            assert bool(((dl.double() - want).abs() <= 400 * U32 * mag + 1e-30).all())
        assert bool((dl[2] == 0).all())
    # in place
    l2 = l.clone()
    g.expert_route_backward(l2, e, dw, l2)
    assert torch.equal(l2, g.expert_route_backward(l, e, dw, torch.empty_like(l)))


def sorted_pairs(expert, G):
    flat = expert.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= G), G, flat)
    order = key.sort(stable=True).indices
    n = flat.numel()
    live = int((key < G).sum())
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(n, device=flat.device)
    slot[key == G] = -1
    source = order.clone()
    source[live:] = -1
    counts = torch.bincount(key, minlength=G + 1)[:G]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return slot.view(expert.shape).to(I32), offsets.to(I32), source.to(I32)


@pytest.mark.parametrize("rows,top,G,kind", [
    (0, 4, 8, "any"), (5, 0, 8, "any"), (1, 1, 1, "any"), (3, 2, 0, "any"), (16, 8, 64, "any"),
    (100, 5, 7, "bad"), (1023, 8, 60, "any"), (1024, 8, 256, "any"), (1025, 8, 256, "bad"),
    (5000, 8, 1024, "any"), (16384, 8, 256, "any"), (40001, 3, 1000, "bad"), (300000, 4, 128, "any"),
    (9000, 2, 513, "one"), (2000, 4, 512, "none"), (150000, 8, 64, "skew")])
def test_sort(gemm_lib, cuda_device, rows, top, G, kind):
    gen = torch.Generator().manual_seed(rows + G)
    e = torch.randint(0, max(G, 1), (rows, top), generator=gen)
    if kind == "bad":
        m = torch.rand(rows, top, generator=gen)
        e[m < 0.1] = -1
        e[m > 0.95] = G
        e[0, 0], e[-1, -1] = -(1 << 31), (1 << 31) - 1
    if kind == "one":
        e[:] = G - 1
    if kind == "none":
        e[:] = -1
    if kind == "skew":
        e = (e * torch.rand(rows, top, generator=gen) ** 3).long()
    expert = e.to(I32).cuda()
    slot, off, src = Guarded((rows, top), I32, 0, 1), Guarded((1, G + 1), I32, 0, 1), Guarded(
        (1, rows * top), I32, 0, 1)
    gemm_lib.expert_sort(expert, slot.t, off.t[0], source=src.t[0])
    want = sorted_pairs(expert, G)
    assert torch.equal(slot.t, want[0]) and torch.equal(off.t[0], want[1]) and torch.equal(src.t[0], want[2])
    assert slot.clean_outside() and off.clean_outside() and src.clean_outside()
    slot2 = torch.empty_like(want[0])
    gemm_lib.expert_sort(expert, slot2, off.t[0])   # without source
    assert torch.equal(slot2, want[0])


def places(rows, top, n, seed, drop=0.2):
    """Distinct rows out of n for the pairs, some pairs without one."""
    gen = torch.Generator().manual_seed(seed)
    pairs = rows * top
    at = torch.randperm(max(n, pairs), generator=gen)[:pairs]
    at[at >= n] = -1
    m = torch.rand(pairs, generator=gen)
    at[m < drop / 2] = -1
    at[(m > 1 - drop / 2) & (at >= 0)] += n    # beyond the last row
    return at.view(rows, top).to(I32).cuda()


def rows_at(a, slot):
    """(rows, top, dim) fp64 rows of the pairs, zero where there is none."""
    n = a.shape[0]
    real = (slot >= 0) & (slot < n)
    if n == 0:
        return torch.zeros(*slot.shape, a.shape[1], dtype=torch.float64, device="cuda"), real
    v = a.double()[torch.where(real, slot, 0).long()]
    return torch.where(real[..., None], v, torch.zeros_like(v)), real


SHAPES = [(1, 1, 1, 1), (3, 2, 9, 8), (16, 8, 128, 4096), (5, 4, 17, 1999), (100, 3, 310, 264),
          (2001, 2, 4002, 129), (7, 32, 200, 520), (33, 1, 20, 2048), (64, 6, 384, 8200), (3, 0, 5, 64),
          (4, 2, 0, 64), (1000, 8, 8000, 1024), (2, 2, 4, 20000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "s8"])
@pytest.mark.parametrize("rows,top,n,dim", SHAPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (16, 16), (3, 1)])
def test_dispatch(gemm_lib, cuda_device, rows, top, n, dim, dtype, pad, off):
    t = {**DTYPE, "s8": torch.int8}[dtype]
    x, a = Guarded((rows, dim), t, pad, off), Guarded((n, dim), t, pad, off)
    x.t.view(torch.uint8).copy_(torch.randint(0, 255, x.t.view(torch.uint8).shape, dtype=torch.uint8))
    slot = places(rows, top, n, dim)
    kb = -(-dim // 128)
    xs, sa = Guarded((kb, rows), torch.float32, 1, 1), Guarded((kb, n), torch.float32, 2, 1)
    xs.set(randn(kb, rows, seed=5))
    more = dict(x_scales=xs.t, a_scales=sa.t) if dtype == "fp8" else {}
    gemm_lib.expert_dispatch(x.t, slot, a.t, **more)
    want = torch.full_like(a.t.contiguous().view(torch.uint8), FILL)
    scales = sa.t.clone()
    scales.view(torch.uint8).fill_(FILL)
    for j in range(top):
        real = ((slot[:, j] >= 0) & (slot[:, j] < n)).nonzero()[:, 0]
        want[slot[real, j].long()] = x.t.contiguous().view(torch.uint8)[real]
        scales[:, slot[real, j].long()] = xs.t[:, real]
    assert torch.equal(a.t.contiguous().view(torch.uint8), want) and a.clean_outside()
    if more:
        assert torch.equal(sa.t.contiguous().view(torch.uint8), scales.view(torch.uint8)) and sa.clean_outside()


@pytest.mark.parametrize("ta,tr,to", [("bf16", "bf16", "bf16"), ("f32", None, "f32"), ("bf16", None, "f32"),
                                      ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("rows,top,n,dim", SHAPES)
@pytest.mark.parametrize("pad,weighted", [(0, True), (8, False), (3, True)])
def test_combine(gemm_lib, cuda_device, rows, top, n, dim, ta, tr, to, pad, weighted):
    a = Guarded((n, dim), DTYPE[ta], pad, pad).set(randn(n, dim, seed=1))
    slot = places(rows, top, n, dim)
    w = randn(rows, top, seed=2) if weighted else None
    r = None if tr is None else Guarded((rows, dim), DTYPE[tr], pad, pad).set(randn(rows, dim, seed=3))
    out = Guarded((rows, dim), DTYPE[to], pad, pad)
    gemm_lib.expert_combine(a.t, slot, out.t, weight=w, residual=None if r is None else r.t)
    v, _ = rows_at(a.t, slot)
    if weighted:
        v = v * w.double()[..., None]
    base = torch.zeros(rows, dim, dtype=torch.float64, device="cuda") if r is None else r.t.double()
    want, mag = base + v.sum(1), base.abs() + v.abs().sum(1)
    err = (top + 1) * U32 * mag
    assert bool(((out.t.double() - want).abs() <= err + half_step(DTYPE[to]) * (want.abs() + err)).all())
    assert out.clean_outside()
    if tr == to:   # onto the residual itself
        gemm_lib.expert_combine(a.t, slot, r.t, weight=w, residual=r.t)
        assert torch.equal(r.t, out.t)


@pytest.mark.parametrize("td,ta,to", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "f32"),
                                      ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("rows,top,n,dim", SHAPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_combine_backward(gemm_lib, cuda_device, rows, top, n, dim, td, ta, to, pad):
    g = gemm_lib
    dout = Guarded((rows, dim), DTYPE[td], pad, pad).set(randn(rows, dim, seed=1))
    a = Guarded((n, dim), DTYPE[ta], pad, pad).set(randn(n, dim, seed=2))
    slot, w = places(rows, top, n, dim), randn(rows, top, seed=3)
    da, dw = Guarded((n, dim), DTYPE[to], pad, pad), Guarded((rows, top), torch.float32, 0, 1)
    g.expert_combine_backward(dout.t, a.t, slot, w, da.t, dw.t)
    v, real = rows_at(a.t, slot)
    prod = v * dout.t.double()[:, None]
    want, mag = prod.sum(-1), prod.abs().sum(-1)
    assert bool(((dw.t.double() - want).abs() <= (dim / 32 + 24) * U32 * mag).all()) and dw.clean_outside()
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    for j in range(top):
        r = real[:, j].nonzero()[:, 0]
        at = slot[r, j].long()
        named[at] = True
        one = w[r, j, None].double() * dout.t[r].double()
        assert bool(((da.t[at].double() - one).abs() <= (U32 + half_step(DTYPE[to]) * (1 + U32)) * one.abs()).all())
    assert bool((da.t[~named].contiguous().view(torch.uint8) == FILL).all()) and da.clean_outside()
    # one without the other, and da in a's place
    dw2 = torch.empty_like(w)
    g.expert_combine_backward(dout.t, a.t, slot, w, None, dw2)
    assert torch.equal(dw2, dw.t)
    da2 = torch.zeros_like(da.t)
    g.expert_combine_backward(dout.t, a.t, slot, w, da2)
    assert torch.equal(da2[named], da.t[named])
    if ta == to:
        g.expert_combine_backward(dout.t, a.t, slot, w, a.t, dw2)
        assert torch.equal(a.t[named], da.t[named]) and torch.equal(dw2, dw.t)


def test_combine_is_dispatch_gradient(gemm_lib, cuda_device):
    # <dispatch(x), y> = <x, combine(y)> in whole numbers, exactly
    g = gemm_lib
    rows, top, dim = 50, 3, 200
    n = rows * top
    gen = torch.Generator().manual_seed(0)
    x = torch.randint(-8, 9, (rows, dim), generator=gen).float().cuda()
    y = torch.randint(-8, 9, (n, dim), generator=gen).float().cuda()
    slot = places(rows, top, n, 0)
    a, back = torch.zeros(n, dim, device="cuda"), torch.empty_like(x)
    g.expert_dispatch(x, slot, a)
    g.expert_combine(y, slot, back)
    assert float((a.double() * y.double()).sum()) == float((x.double() * back.double()).sum())


def test_unnamed_rows_and_weights_do_not_enter(gemm_lib, cuda_device):
    # rows no pair names, and the weights of pairs without a row, may hold anything
    g = gemm_lib
    nan = float("nan")
    a = torch.full((6, 64), nan, device="cuda")
    a[2], a[4] = 1.0, 2.0
    slot = torch.tensor([[2, -1], [9, 4], [-5, 6]], dtype=I32, device="cuda")
    w = torch.tensor([[0.5, nan], [nan, 3.0], [nan, nan]], device="cuda")
    out = torch.empty(3, 64, device="cuda")
    g.expert_combine(a, slot, out, weight=w)
    assert out[:, 0].tolist() == [0.5, 6.0, 0.0] and bool((out == out[:, :1]).all())
    dw, dout = torch.full_like(w, 7.0), torch.ones(3, 64, device="cuda")
    g.expert_combine_backward(dout, a, slot, w, None, dw)
    assert dw.tolist() == [[64.0, 0.0], [0.0, 128.0], [0.0, 0.0]]


def test_slots_past_two_to_the_31_elements(gemm_lib, cuda_device):
    # the last rows of an array of more than 2^31 elements
    g = gemm_lib
    dim, n = 1 << 16, (1 << 15) + 40
    a = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
    x = randn(2, dim, seed=1, dtype=torch.bfloat16)
    slot = torch.tensor([[n - 1, 3], [n - 2, (1 << 15) + 1]], dtype=I32, device="cuda")
    g.expert_dispatch(x, slot, a)
    assert torch.equal(a[n - 1], x[0]) and torch.equal(a[3], x[0]) and torch.equal(a[(1 << 15) + 1], x[1])
    out, w = torch.empty_like(x), torch.tensor([[2.0, 1.0], [4.0, -1.0]], device="cuda")
    g.expert_combine(a, slot, out, weight=w)
    assert torch.equal(out[1], (3.0 * x[1].float()).bfloat16())
    dw = torch.empty_like(w)
    g.expert_combine_backward(x, a, slot, w, a, dw)
    assert torch.equal(a[n - 2], (4.0 * x[1].float()).bfloat16())


def test_streams_and_graph(gemm_lib, cuda_device):
    """Sort, dispatch and combine on two streams at once, and captured and replayed with other ids."""
    g = gemm_lib
    rows, top, G, dim = 4000, 4, 64, 256
    n = rows * top

    class Work:
        def __init__(self, seed):
            self.e = torch.randint(-1, G, (rows, top), generator=torch.Generator().manual_seed(seed)).to(I32).cuda()
            self.x, self.w = randn(rows, dim, seed=seed), randn(rows, top, seed=seed + 1)
            self.slot, self.off = torch.empty_like(self.e), torch.empty(G + 1, dtype=I32, device="cuda")
            self.a, self.out = torch.zeros(n, dim, device="cuda"), torch.empty(rows, dim, device="cuda")

        def run(self):
            g.expert_sort(self.e, self.slot, self.off)
            g.expert_dispatch(self.x, self.slot, self.a)
            g.expert_combine(self.a, self.slot, self.out, weight=self.w)

        def check(self):
            slot, off, _ = sorted_pairs(self.e, G)
            assert torch.equal(self.slot, slot) and torch.equal(self.off, off)
            s = torch.where(self.e >= 0, self.w.double(), 0.0).sum(1, keepdim=True)
            mag = self.w.double().abs().sum(1, keepdim=True) * self.x.double().abs()
            assert bool(((self.out.double() - s * self.x.double()).abs() <= 6 * U32 * mag).all())

    works, streams = [Work(1), Work(3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, s in zip(works, streams):
            with torch.cuda.stream(s):
                w.run()
    torch.cuda.synchronize()
    for w in works:
        w.check()
    w, s = works[0], streams[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        w.run()
    for seed in (11, 12):
        w.e.copy_(torch.randint(-1, G, (rows, top), generator=torch.Generator().manual_seed(seed)).to(I32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        w.check()
    # without counters a capture is refused, and nothing is queued
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh):
        with pytest.raises(g.GemmError) as e:
            g.expert_sort(w.e, w.slot, w.off)
        w.out.zero_()
    assert g.STATUS[e.value.status] == "GEMM_ERR_NO_MEMORY"
    for s in streams:
        g.gemm_release_stream(s.cuda_stream)


def test_same_bits_every_time(gemm_lib, cuda_device):
    g = gemm_lib
    rows, top, n, dim = 3000, 8, 24000, 520
    a, slot, w = randn(n, dim, seed=1), places(rows, top, n, 2), randn(rows, top, seed=3)
    dout = randn(rows, dim, seed=4)
    first = None
    for _ in range(3):
        out, dw = torch.empty(rows, dim, device="cuda"), torch.empty_like(w)
        g.expert_combine(a, slot, out, weight=w)
        g.expert_combine_backward(dout, a, slot, w, None, dw)
        if first is not None:
            assert torch.equal(out, first[0]) and torch.equal(dw, first[1])
        first = out, dw
