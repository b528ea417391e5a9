"""Arguments that layer norm and its gradient refuse (no GPU: every check comes before the first device
call)."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 3
P = 1 << 20
F32, BF16, E4M3, S8 = 0, 1, 2, 3

needs_no_device = pytest.mark.skipif(torch.cuda.is_available(),
                                     reason="calls that pass the checks would launch")


def args(g, **kw):
    a = g.LayernormArgs()
    a.x, a.ldx, a.x_type, a.weight, a.bias, a.eps = P, 256, BF16, P, P, 1e-5
    a.y, a.ldy, a.y_type = P, 256, BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(ldx=255), dict(ldy=200), dict(x_type=E4M3), dict(y_type=7), dict(x=P + 1),
    dict(weight=P + 2), dict(bias=P + 1), dict(y=P + 1), dict(residual=P, ldr=255),
    dict(residual=P, ldr=256, residual_type=3), dict(h=P, ldh=10), dict(h=P + 2, ldh=256),
    dict(q=P, ldq=256, q_type=S8), dict(scales=P, ld_scales=8), dict(q=P, ldq=255, q_type=S8, scales=P),
    dict(q=P, ldq=256, q_type=F32, scales=P, ld_scales=8), dict(q=P, ldq=256, q_type=BF16, scales=P, ld_scales=8),
    dict(q=P, ldq=256, q_type=E4M3, scales=P, ld_scales=7), dict(q=P, ldq=256, q_type=S8, scales=P + 2),
    dict(mean=P + 2), dict(rstd=P + 1)])
def test_layernorm_refuses(gemm_lib, kw):
    assert gemm_lib.gemm_layernorm(8, 256, args(gemm_lib, **kw)) == INVALID


def test_layernorm_sizes(gemm_lib):
    g = gemm_lib
    a = args(g)
    assert g.gemm_layernorm(-1, 256, a) == INVALID and g.gemm_layernorm(8, -1, a) == INVALID
    assert g.gemm_layernorm(8, (1 << 30) + 1, a) == INVALID
    assert g.gemm_layernorm(0, 256, a) == OK and g.gemm_layernorm(8, 0, a) == OK
    assert g.load_library().gemm_layernorm(8, 256, None, 0) == INVALID
    assert g.gemm_layernorm(8, 256, args(g, y=None)) == OK  # no output asked for


def grad_args(g, **kw):
    a = g.LayernormGradArgs()
    a.dy, a.lddy, a.dy_type, a.h, a.ldh, a.h_type = P, 256, BF16, P, 256, F32
    a.weight, a.mean, a.rstd, a.dh, a.lddh, a.dh_type, a.dweight, a.dbias = P, P, P, P, 256, F32, P, P
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None), dict(dh=None), dict(lddy=255),
    dict(ldh=1), dict(lddh=255), dict(dy_type=2), dict(h_type=-1), dict(dh_type=3), dict(dh=P + 2),
    dict(weight=P + 1), dict(mean=P + 2), dict(rstd=P + 1), dict(dweight=P + 2), dict(dbias=P + 2),
    dict(residual_grad=P, ldrg=255), dict(residual_grad=P, ldrg=256, residual_grad_type=9)])
def test_layernorm_backward_refuses(gemm_lib, kw):
    assert gemm_lib.gemm_layernorm_backward(8, 256, grad_args(gemm_lib, **kw)) == INVALID


@needs_no_device
def test_no_device_no_fallback(gemm_lib):
    g = gemm_lib
    assert g.gemm_layernorm(8, 256, args(g, weight=None, bias=None)) == UNSUPPORTED
    assert g.gemm_layernorm(8, 256, args(g, q=P, ldq=256, q_type=S8, scales=P)) == UNSUPPORTED
    assert g.gemm_layernorm_backward(8, 256, grad_args(g, weight=None)) == UNSUPPORTED


def test_tensor_helpers_refuse_host_tensors(gemm_lib):
    g = gemm_lib
    x, v = torch.zeros(4, 8), torch.ones(4)
    for call in (lambda: g.layernorm(x, torch.ones(8), y=x), lambda: g.layernorm_backward(x, x, None, v, v, x)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_tensor_helpers_refuse_wrong_tensors(gemm_lib, cuda_device):
    g = gemm_lib

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    x, w, v, s8, f8 = z(4, 8), z(8), z(4), z(4, 8, dtype=torch.int8), z(4, 8, dtype=torch.float8_e4m3fn)
    bad = [
        (TypeError, lambda: g.layernorm(x.half(), w, y=x)),
        (TypeError, lambda: g.layernorm(x, w.bfloat16(), y=x)),
        (ValueError, lambda: g.layernorm(x, w, z(7), y=x)),
        (ValueError, lambda: g.layernorm(x.t(), z(4), y=z(8, 4))),
        (ValueError, lambda: g.layernorm(x, w, q=s8)),
        (ValueError, lambda: g.layernorm(x, w, q=s8, scales=z(1, 4))),
        (ValueError, lambda: g.layernorm(x, w, q=f8, scales=z(4))),
        (TypeError, lambda: g.layernorm(x, w, q=x, scales=v)),
        (ValueError, lambda: g.layernorm(x, w, y=x, mean=z(5))),
        (TypeError, lambda: g.layernorm(x, w, y=torch.zeros(4, 8))),
        (ValueError, lambda: g.layernorm_backward(x, z(4, 9), w, v, v, x)),
        (ValueError, lambda: g.layernorm_backward(x, x, w, z(5), v, x)),
        (ValueError, lambda: g.layernorm_backward(x, x, w, v, v, x, dbias=z(4))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


def test_packed_arguments_are_the_mirrors(gemm_lib):
    g = gemm_lib
    for mirror, pack in ((g.LayernormArgs, g._pack_layernorm), (g.LayernormGradArgs, g._pack_layernorm_grad)):
        values = [0.5 if name == "eps" else 1000 + i for i, (name, _) in enumerate(mirror._fields_)]
        a = mirror.from_buffer_copy(pack(*values))
        assert [getattr(a, name) for name, _ in mirror._fields_] == values
