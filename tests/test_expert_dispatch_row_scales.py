"""gemm_expert_dispatch of rows with one scale each, as int8 rows from layer norm or the quantiser have."""
import pytest
import torch

INVALID, UNSUPPORTED = 1, 3
P = 1 << 20  # an address that is only ever looked at
DISPATCH = dict(rows=10, top=4, n=40, dim=256, size=1, x=P, ldx=256, slot=P, a=P, lda=256, xs=P, ldxs=0,
                sas=P, ldas=0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would launch")
def test_row_scales_pass_the_checks(gemm_lib):
    assert gemm_lib.gemm_expert_dispatch(*DISPATCH.values()) == UNSUPPORTED   # no device


@pytest.mark.parametrize("kw", [dict(ldxs=10), dict(ldas=40), dict(xs=0), dict(sas=0), dict(xs=P + 2),
                                dict(sas=P + 1), dict(ldxs=-1), dict(ldas=-1), dict(ldxs=-1, ldas=-1)])
def test_refusals(gemm_lib, kw):
    assert gemm_lib.gemm_expert_dispatch(*{**DISPATCH, **kw}.values()) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("rows,top,dim,pad", [(1, 1, 16, 0), (16, 8, 4096, 0), (300, 4, 1000, 8), (5000, 2, 129, 15),
                                              (700, 1, 8192, 0), (9, 32, 64, 0)])
def test_int8_rows_move_with_their_scales(gemm_lib, cuda_device, rows, top, dim, pad):
    g = gemm_lib
    n = rows * top + 7
    gen = torch.Generator().manual_seed(rows + dim)
    x = torch.empty(rows, dim + pad, dtype=torch.int8, device="cuda")[:, :dim]
    x.copy_(torch.randint(-127, 128, (rows, dim), generator=gen).to(torch.int8))
    s = torch.rand(rows, generator=gen).cuda()
    slot = torch.randperm(n, generator=gen)[: rows * top].view(rows, top).to(torch.int32)
    slot[torch.rand(rows, top, generator=gen) < 0.1] = -1     # pairs without a row
    slot[-1, -1] = n                                          # and one that is none
    a = torch.full((n, dim + pad), 0x5A, dtype=torch.int8, device="cuda")
    raw = torch.full((n + 2,), -5.0, device="cuda")
    g.expert_dispatch(x, slot.cuda(), a[:, :dim], x_scales=s, a_scales=raw[1:-1])
    assert g.gemm_check_device_error(0) == 0
    want, scales = torch.full_like(a, 0x5A), torch.full_like(raw, -5.0)
    for j in range(top):
        at = slot[:, j].cuda().long()
        real = (at >= 0) & (at < n)
        want[at[real], :dim] = x[real]
        scales[1:-1][at[real]] = s[real]
    assert torch.equal(a, want) and torch.equal(raw, scales)


@pytest.mark.gpu
def test_norm_to_experts_product_in_8_bits(gemm_lib, cuda_device):
    """Layer norm's int8 rows through dispatch into each expert's product, as they would be used."""
    g = gemm_lib
    rows, dim, out, experts, top = 70, 512, 96, 3, 2
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(rows, dim, generator=gen).cuda().bfloat16()
    q, s = torch.empty(rows, dim, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    y = torch.empty(rows, dim, device="cuda")
    g.layernorm(x, y=y, q=q, scales=s)
    w = torch.randint(-127, 128, (experts, out, dim), generator=gen).to(torch.int8).cuda()
    ws = torch.rand(experts, out, generator=gen).cuda()
    expert = torch.empty(rows, top, dtype=torch.int32, device="cuda")
    weight, slot = torch.empty(rows, top, device="cuda"), torch.empty_like(expert)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    g.expert_route(torch.randn(rows, experts, generator=gen).cuda(), expert, weight)
    g.expert_sort(expert, slot, offsets)
    a, a_s = torch.empty(rows * top, dim, dtype=torch.int8, device="cuda"), torch.empty(rows * top, device="cuda")
    g.expert_dispatch(q, slot, a, x_scales=s, a_scales=a_s)
    d = torch.empty(rows * top, out, device="cuda")
    ends = offsets.tolist()
    for e in range(experts):
        at = slice(ends[e], ends[e + 1])
        g.int8gemm(a[at], a_s[at], w[e], ws[e], d[at])
    assert g.gemm_check_device_error(0) == 0
    for j in range(top):
        e = expert[:, j].long()
        # the sums are exact, and below 2^23 (512 * 127^2); two products round once each
        want = torch.einsum("rk,rnk->rn", q.double(), w[e].double()) * s.double()[:, None] * ws[e].double()
        assert bool(((d[slot[:, j].long()].double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all())


@pytest.mark.gpu
def test_tensor_helper_refuses_other_scales(gemm_lib, cuda_device):
    g = gemm_lib
    slot = torch.zeros(4, 2, dtype=torch.int32, device="cuda")

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    x, a = z(4, 256, dtype=torch.int8), z(8, 256, dtype=torch.int8)
    f8 = torch.float8_e4m3fn
    for error, call in (
            (ValueError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(4), a_scales=z(2, 8))),
            (ValueError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(4), a_scales=z(7))),
            (ValueError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(5), a_scales=z(8))),
            (ValueError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(4, 2)[:, 0], a_scales=z(8))),
            (TypeError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(4).double(), a_scales=z(8))),
            (ValueError, lambda: g.expert_dispatch(x, slot, a, x_scales=z(4))),
            # an fp8 row has a scale for each of its blocks
            (ValueError, lambda: g.expert_dispatch(x.view(f8), slot, a.view(f8), x_scales=z(4), a_scales=z(8)))):
        with pytest.raises(error):
            call()
