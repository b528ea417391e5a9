"""Arguments that the router's and the experts' rows' operators refuse (no GPU: every check comes
before the first device call)."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 3
P = 1 << 20  # an address that is only ever looked at
F32, BF16, E4M3 = 0, 1, 2
BIG = 1 << 31

needs_no_device = pytest.mark.skipif(torch.cuda.is_available(),
                                     reason="calls that pass the checks would launch")

ROUTE = dict(rows=10, G=64, top=4, logits=P, ld=64, type=F32, normalize=0, expert=P, weight=P)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(G=-1), INVALID), (dict(top=-1), INVALID), (dict(top=65), INVALID),
    (dict(logits=0), INVALID), (dict(logits=P + 2), INVALID), (dict(ld=63), INVALID),
    (dict(type=E4M3), INVALID), (dict(expert=0), INVALID), (dict(weight=0), INVALID),
    (dict(expert=P + 2), INVALID), (dict(weight=P + 1), INVALID), (dict(rows=BIG), INVALID),
    (dict(rows=1 << 30, top=2), INVALID), (dict(G=1025, ld=1025), UNSUPPORTED),
    (dict(top=33), UNSUPPORTED), (dict(rows=0, logits=0), OK), (dict(top=0, expert=0), OK)])
def test_route_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_route(*{**ROUTE, **kw}.values()) == status


ROUTEG = dict(rows=10, G=64, top=4, logits=P, ld=64, type=F32, normalize=1, expert=P, dweight=P, dlogits=P,
              ldd=64, dtype=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(top=65), INVALID), (dict(logits=0), INVALID), (dict(ld=1), INVALID),
    (dict(dlogits=0), INVALID), (dict(dlogits=P + 1), INVALID), (dict(ldd=63), INVALID),
    (dict(dtype=3), INVALID), (dict(expert=0), INVALID), (dict(dweight=0), INVALID),
    (dict(top=33), UNSUPPORTED), (dict(rows=0, dlogits=0), OK)])
def test_route_backward_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_route_backward(*{**ROUTEG, **kw}.values()) == status


SORT = dict(n=100, G=8, expert=P, slot=P, offsets=P, source=0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(G=-1), INVALID), (dict(n=BIG), INVALID), (dict(expert=0), INVALID),
    (dict(slot=0), INVALID), (dict(offsets=0), INVALID), (dict(offsets=P + 2), INVALID),
    (dict(source=P + 1), INVALID), (dict(slot=P + 2), INVALID), (dict(G=1025), UNSUPPORTED)])
def test_sort_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_sort(*{**SORT, **kw}.values()) == status


DISPATCH = dict(rows=10, top=4, n=40, dim=256, size=1, x=P, ldx=256, slot=P, a=P, lda=256, xs=P, ldxs=10,
                sas=P, ldas=40)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(top=-1), INVALID), (dict(n=-1), INVALID), (dict(dim=-1), INVALID),
    (dict(size=3), INVALID), (dict(size=8), INVALID), (dict(x=0), INVALID), (dict(a=0), INVALID),
    (dict(slot=0), INVALID), (dict(slot=P + 2), INVALID), (dict(ldx=255), INVALID),
    (dict(lda=255), INVALID), (dict(size=2, x=P + 1), INVALID), (dict(size=4, a=P + 2), INVALID),
    (dict(xs=0), INVALID), (dict(sas=0), INVALID), (dict(ldxs=9), INVALID), (dict(ldas=39), INVALID),
    (dict(xs=P + 2), INVALID), (dict(rows=1 << 30), INVALID), (dict(rows=BIG), INVALID),
    (dict(top=33), UNSUPPORTED), (dict(rows=0, x=0), OK), (dict(n=0, a=0), OK), (dict(dim=0), OK)])
def test_dispatch_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_dispatch(*{**DISPATCH, **kw}.values()) == status


COMBINE = dict(rows=10, top=4, n=40, dim=256, a=P, lda=256, a_type=BF16, slot=P, weight=P, residual=P,
               ldr=256, r_type=F32, out=P, ldo=256, o_type=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(dim=(1 << 30) + 1, lda=BIG - 1, ldo=BIG - 1, ldr=BIG - 1), INVALID),
    (dict(a=0), INVALID), (dict(a=P + 1), INVALID), (dict(lda=255), INVALID), (dict(a_type=2), INVALID),
    (dict(slot=0), INVALID), (dict(weight=P + 2), INVALID), (dict(ldr=255), INVALID),
    (dict(r_type=3), INVALID), (dict(residual=P + 2), INVALID), (dict(out=0), INVALID),
    (dict(ldo=10), INVALID), (dict(o_type=2), INVALID), (dict(out=P + 1), INVALID),
    (dict(top=33), UNSUPPORTED), (dict(rows=0, a=0), OK), (dict(dim=0, a=0), OK)])
def test_combine_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_combine(*{**COMBINE, **kw}.values()) == status


COMBINEG = dict(rows=10, top=4, n=40, dim=256, dout=P, lddo=256, do_type=BF16, a=P, lda=256, a_type=BF16,
                slot=P, weight=P, da=P, ldda=256, da_type=F32, dweight=P)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(dout=0), INVALID), (dict(lddo=255), INVALID),
    (dict(do_type=2), INVALID), (dict(a=0), INVALID), (dict(lda=2), INVALID), (dict(a_type=-1), INVALID),
    (dict(slot=0), INVALID), (dict(weight=0), INVALID), (dict(ldda=255), INVALID),
    (dict(da_type=9), INVALID), (dict(da=P + 2), INVALID), (dict(dweight=P + 2), INVALID),
    (dict(top=33), UNSUPPORTED), (dict(da=0, dweight=0), OK), (dict(rows=0), OK), (dict(top=0), OK)])
def test_combine_backward_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_expert_combine_backward(*{**COMBINEG, **kw}.values()) == status


@needs_no_device
def test_no_device_no_fallback(gemm_lib):
    g = gemm_lib
    assert g.gemm_expert_route(*ROUTE.values()) == UNSUPPORTED
    assert g.gemm_expert_route_backward(*ROUTEG.values()) == UNSUPPORTED
    assert g.gemm_expert_sort(*SORT.values()) == UNSUPPORTED
    assert g.gemm_expert_sort(0, 8, 0, 0, P, 0) == UNSUPPORTED   # offsets are written
    assert g.gemm_expert_dispatch(*DISPATCH.values()) == UNSUPPORTED
    assert g.gemm_expert_combine(*COMBINE.values()) == UNSUPPORTED
    assert g.gemm_expert_combine(*{**COMBINE, "top": 0, "a": 0}.values()) == UNSUPPORTED
    assert g.gemm_expert_combine_backward(*COMBINEG.values()) == UNSUPPORTED


def test_tensor_helpers_refuse_host_tensors(gemm_lib):
    g = gemm_lib
    i32 = torch.int32
    x, e, w, off = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2), torch.zeros(9, dtype=i32)
    a = torch.zeros(8, 8)
    for call in (lambda: g.expert_route(x, e, w), lambda: g.expert_route_backward(x, e, w, x),
                 lambda: g.expert_sort(e, e, off), lambda: g.expert_dispatch(x, e, a),
                 lambda: g.expert_combine(a, e, x), lambda: g.expert_combine_backward(x, a, e, w, a, w)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_tensor_helpers_refuse_wrong_tensors(gemm_lib, cuda_device):
    g = gemm_lib
    i32 = torch.int32

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    x, e, w, a, off = z(4, 8), z(4, 2, dtype=i32), z(4, 2), z(8, 8), z(9, dtype=i32)
    bad = [
        (TypeError, lambda: g.expert_route(x.half(), e, w)),
        (TypeError, lambda: g.expert_route(x, e.long(), w)),
        (ValueError, lambda: g.expert_route(x, e, z(4, 3))),
        (ValueError, lambda: g.expert_route(z(5, 8), e, w)),
        (ValueError, lambda: g.expert_route(x, z(2, 4, dtype=i32).t(), w)),
        (ValueError, lambda: g.expert_route_backward(x, e, w, z(4, 7))),
        (g.GemmError, lambda: g.expert_route(z(4, 1), e, w)),
        (TypeError, lambda: g.expert_sort(e, w, off)),
        (ValueError, lambda: g.expert_sort(e, z(4, 3, dtype=i32), off)),
        (ValueError, lambda: g.expert_sort(e, e, z(0, dtype=i32))),
        (ValueError, lambda: g.expert_sort(e, e, off, source=z(7, dtype=i32))),
        (TypeError, lambda: g.expert_dispatch(x, e, a.bfloat16())),
        (TypeError, lambda: g.expert_dispatch(x.double(), e, a.double())),
        (ValueError, lambda: g.expert_dispatch(x, e, z(8, 7))),
        (ValueError, lambda: g.expert_dispatch(x, e, a, x_scales=z(1, 4))),
        (ValueError, lambda: g.expert_dispatch(x, e, a, x_scales=z(1, 4), a_scales=z(1, 4))),
        (ValueError, lambda: g.expert_combine(a, e, z(5, 8))),
        (ValueError, lambda: g.expert_combine(a, e, x, weight=z(2, 4).t())),
        (TypeError, lambda: g.expert_combine(a, e, x, residual=x.half())),
        (ValueError, lambda: g.expert_combine_backward(x, a, e, w, z(7, 8), w)),
        (TypeError, lambda: g.expert_combine_backward(x, a, e, w.double(), a, w)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
