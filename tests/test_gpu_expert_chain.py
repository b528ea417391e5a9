"""The operators of a layer of experts one after another, as they are served and trained: routing, sorting,
gathering, the grouped product and adding up, in one captured graph and in eager mode, against a plain form
in 64 bits that goes row by row and choice by choice."""
import pytest
import torch

import dense_gemm_12_gb300 as g
from gpu_helpers import check_device_error
from ops_ref import UBF, U32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gemm_lib, cuda_device):
    yield


class Chain:
    def __init__(self, rows, dim, out, experts, top, seed):
        self.logits = torch.empty(rows, experts, device="cuda")
        self.x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
        self.fill(seed)
        self.w = randn(experts, dim, out, seed=3, scale=dim ** -0.5, dtype=torch.bfloat16)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.expert, self.slot = torch.empty(rows, top, **i32), torch.empty(rows, top, **i32)
        self.weight, self.offsets = torch.empty(rows, top, device="cuda"), torch.empty(experts + 1, **i32)
        # rows behind the last pair: NaN, which must not enter
        self.a = torch.full((rows * top, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.b = torch.full((rows * top, out), float("nan"), device="cuda")
        self.y = torch.empty(rows, out, device="cuda")
        self.dy = randn(rows, out, seed=4)
        self.db, self.dweight = torch.zeros(rows * top, out, device="cuda"), torch.empty(rows, top, device="cuda")
        self.dlogits = torch.empty(rows, experts, device="cuda")

    def fill(self, seed):
        rows, experts = self.logits.shape
        self.logits.copy_(randn(rows, experts, seed=seed, scale=2.0))
        if rows > 2:   # a padded batch: rows that no expert gets, and one expert that gets nothing
            self.logits[rows // 2] = float("-inf")
            self.logits[-1] = float("-inf")
        if experts > 8:
            self.logits[:, 5] = float("-inf")
        self.x.copy_(randn(*self.x.shape, seed=seed + 1, dtype=torch.bfloat16))

    def run(self):
        g.expert_route(self.logits, self.expert, self.weight, normalize=True)
        g.expert_sort(self.expert, self.slot, self.offsets)
        g.expert_dispatch(self.x, self.slot, self.a)
        g.bf16gemm_grouped(self.a, self.w, self.offsets, self.b)
        g.expert_combine(self.b, self.slot, self.y, self.weight)
        g.expert_combine_backward(self.dy, self.b, self.slot, self.weight, da=self.db, dweight=self.dweight)
        g.expert_route_backward(self.logits, self.expert, self.dweight, self.dlogits, normalize=True)

    def check(self):
        rows, top = self.expert.shape
        z = self.logits.double()
        value, index = z.topk(top, dim=-1)
        keep = value > float("-inf")
        assert torch.equal(self.expert.long(), torch.where(keep, index, -1))
        top_z = torch.where(keep, value, -1e300)
        p = torch.where(keep, (top_z - top_z[:, :1]).exp(), 0.0)
        p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
        # exp of a difference below 2^5: 2^5 U32 for it, 3 for the function, the sum and the quotient
        assert bool(((self.weight.double() - p).abs() <= 64 * U32 * p + 1e-30).all())
        # every kept pair has a row of its own, in its expert's range
        rows_of = self.slot.long()[keep]
        assert torch.equal(rows_of.sort().values, torch.arange(int(keep.sum()), device="cuda"))
        e, off = self.expert.long()[keep], self.offsets.long()
        assert bool((off[e] <= rows_of).all()) and bool((rows_of < off[e + 1]).all())
        assert bool((self.slot[~keep] == -1).all())
        # products: fp32 sums of dim products in any order
        per = torch.zeros(rows, top, self.w.shape[2], dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(per)
        token = torch.arange(rows, device="cuda")[:, None].expand(rows, top)[keep]
        xs, ws = self.x.double()[token], self.w.double()
        for i in range(ws.shape[0]):
            m = e == i
            if bool(m.any()):
                at = keep.nonzero()[m]
                per[at[:, 0], at[:, 1]] = xs[m] @ ws[i]
                mag[at[:, 0], at[:, 1]] = xs[m].abs() @ ws[i].abs()
        wt = self.weight.double()
        err = (self.x.shape[1] * U32 * mag * wt[..., None]).sum(1) + (top + 1) * U32 * (mag * wt[..., None]).sum(1)
        assert bool(((self.y.double() - (per * wt[..., None]).sum(1)).abs() <= err).all())
        assert bool((self.y[~keep.any(1)] == 0).all())
        # gradients
        dw = (per * self.dy.double()[:, None]).sum(-1)
        dmag = (mag * self.dy.double().abs()[:, None]).sum(-1)
        werr = (self.x.shape[1] + self.w.shape[2]) * U32 * dmag
        assert bool(((self.dweight.double() - dw).abs() <= werr).all())
        want_db = (self.dy.double()[:, None] * wt[..., None])[keep]
        assert bool(((self.db.double()[rows_of] - want_db).abs() <= 2 * U32 * want_db.abs()).all())
        dws = self.dweight.double()
        inner = p * (dws - (p * dws).sum(1, keepdim=True))
        want = torch.zeros_like(z).scatter_add(1, torch.where(keep, index, 0), torch.where(keep, inner, 0.0))
        size = (p * (dws.abs() + (p * dws.abs()).sum(1, keepdim=True)))
        bound = torch.zeros_like(z).scatter_add(1, torch.where(keep, index, 0), torch.where(keep, size, 0.0))
        # p as above (64), once more in the inner sum, top additions and the products around them
        assert bool(((self.dlogits.double() - want).abs() <= (128 + top + 8) * U32 * bound).all())


SIZES = [(1, 264, 136, 16, 2), (4, 512, 256, 64, 8), (33, 100, 50, 7, 3), (600, 384, 640, 32, 4),
         (1031, 256, 264, 128, 6), (5, 64, 72, 4, 4)]


@pytest.mark.parametrize("rows,dim,out,experts,top", SIZES)
def test_chain(rows, dim, out, experts, top):
    c = Chain(rows, dim, out, experts, top, 10)
    c.run()
    check_device_error()
    c.check()


@pytest.mark.parametrize("rows,dim,out,experts,top", SIZES[:2] + SIZES[3:5])
def test_two_captured_chains_and_an_eager_one(rows, dim, out, experts, top):
    # both graphs are captured on one stream, whose workspace they share
    s = torch.cuda.Stream()
    chains = [Chain(rows, dim, out, experts, top, 20 + i) for i in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        chains[0].run()
    s.synchronize()
    graphs = []
    for c in chains[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.run()
        graphs.append(graph)
    for seed in (31, 41):
        for i, c in enumerate(chains):
            c.fill(seed + i)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[1].replay()
            chains[2].run()
            graphs[0].replay()
        s.synchronize()
        check_device_error()
        for c in chains:
            c.check()
    first = chains[0].dlogits.clone(), chains[0].y.clone()
    with torch.cuda.stream(s):
        graphs[0].replay()
    s.synchronize()
    assert torch.equal(first[0], chains[0].dlogits) and torch.equal(first[1], chains[0].y)
    g.gemm_release_stream(s.cuda_stream)


def test_a_served_chain_in_8_bits():
    # layer norm to fp8, its rows with their scales, the grouped fp8 product
    rows, dim, out, experts, top = 70, 384, 264, 8, 2
    x, logits = randn(rows, dim, seed=1, dtype=torch.bfloat16), randn(rows, experts, seed=2)
    kb = -(-dim // 128)
    q, s = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(kb, rows, device="cuda")
    g.layernorm(x, q=q, scales=s)
    w = randn(experts, dim, out, seed=3, scale=dim ** -0.5)
    wq = torch.empty(experts, out, dim, dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.empty(experts, kb, -(-out // 128), device="cuda")
    for i in range(experts):
        g.fp8_quantize(w[i], wq[i], ws[i], block="tiles", transpose=True)
    expert = torch.empty(rows, top, dtype=torch.int32, device="cuda")
    slot, weight = torch.empty_like(expert), torch.empty(rows, top, device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    g.expert_route(logits, expert, weight)
    g.expert_sort(expert, slot, offsets)
    n = rows * top
    a, a_s = torch.empty(n, dim, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(kb, n, device="cuda")
    g.expert_dispatch(q, slot, a, x_scales=s, a_scales=a_s)
    b, y = torch.empty(n, out, device="cuda"), torch.empty(rows, out, dtype=torch.bfloat16, device="cuda")
    g.fp8gemm_grouped(a, a_s, wq, ws, offsets, b)
    g.expert_combine(b, slot, y, weight)
    check_device_error()
    qv = q.double() * s.double().t().repeat_interleave(128, 1)
    wv = wq.double() * ws.double().transpose(1, 2).repeat_interleave(128, 1)[:, :out].repeat_interleave(128, 2)
    per = torch.einsum("rk,rjnk->rjn", qv, wv[expert.long()])
    mag = torch.einsum("rk,rjnk->rjn", qv.abs(), wv[expert.long()].abs())
    want = (per * weight.double()[..., None]).sum(1)
    err = (dim + 16) * U32 * (mag * weight.double()[..., None]).sum(1)
    assert bool(((y.double() - want).abs() <= err + UBF * (want.abs() + err)).all())
