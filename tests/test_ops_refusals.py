"""Arguments that the operators around the GEMMs refuse (no GPU: every check
comes before the first device call)."""
import ctypes

import pytest
import torch

OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
P = 1 << 20  # an address that is only ever looked at
F32, BF16, E4M3 = 0, 1, 2


needs_no_device = pytest.mark.skipif(torch.cuda.is_available(),
                                     reason="calls that pass the checks would launch")


def norm_args(g, **kw):
    a = g.RmsnormArgs()
    a.x, a.ldx, a.x_type, a.weight, a.eps = P, 256, BF16, P, 1e-6
    a.y, a.ldy, a.y_type = P, 256, BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(weight=None), dict(ldx=255), dict(ldy=200), dict(x_type=E4M3), dict(y_type=7),
    dict(x=P + 1), dict(weight=P + 2), dict(y=P + 1),
    dict(residual=P, ldr=255), dict(residual=P, ldr=256, residual_type=3),
    dict(h=P, ldh=10, h_type=F32), dict(h=P + 2, ldh=256, h_type=F32),
    dict(q=P, ldq=256), dict(scales=P, ld_scales=8), dict(q=P, ldq=255, scales=P, ld_scales=8),
    dict(q=P, ldq=256, scales=P, ld_scales=7), dict(q=P, ldq=256, scales=P + 2, ld_scales=8),
    dict(rstd=P + 2)])
def test_rmsnorm_refuses(gemm_lib, kw):
    g = gemm_lib
    assert g.gemm_rmsnorm(8, 256, norm_args(g, **kw)) == INVALID


def test_rmsnorm_sizes(gemm_lib):
    g = gemm_lib
    a = norm_args(g)
    assert g.gemm_rmsnorm(-1, 256, a) == INVALID
    assert g.gemm_rmsnorm(8, -1, a) == INVALID
    assert g.gemm_rmsnorm(8, (1 << 30) + 1, a) == INVALID
    assert g.gemm_rmsnorm(0, 256, a) == OK and g.gemm_rmsnorm(8, 0, a) == OK
    assert g.load_library().gemm_rmsnorm(8, 256, None, 0) == INVALID
    assert g.gemm_rmsnorm(8, 256, norm_args(g, y=None)) == OK  # no output asked for


def grad_args(g, **kw):
    a = g.RmsnormGradArgs()
    a.dy, a.lddy, a.dy_type, a.h, a.ldh, a.h_type = P, 256, BF16, P, 256, F32
    a.weight, a.rstd, a.dh, a.lddh, a.dh_type, a.dweight = P, P, P, 256, F32, P
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(h=None), dict(weight=None), dict(rstd=None), dict(dh=None), dict(lddy=255),
    dict(ldh=1), dict(lddh=255), dict(dy_type=2), dict(h_type=-1), dict(dh_type=3), dict(dh=P + 2),
    dict(rstd=P + 1), dict(dweight=P + 2), dict(residual_grad=P, ldrg=255),
    dict(residual_grad=P, ldrg=256, residual_grad_type=9)])
def test_rmsnorm_backward_refuses(gemm_lib, kw):
    g = gemm_lib
    assert g.gemm_rmsnorm_backward(8, 256, grad_args(g, **kw)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(x=0), dict(q=0), dict(scales=0), dict(ldx=199), dict(ldq=199),
    dict(lds=99), dict(x_type=2), dict(block=2), dict(block=-1), dict(x=P + 1), dict(scales=P + 2),
    dict(transpose=1, ldq=99), dict(transpose=1, ldq=100, lds=199), dict(block=1, lds=0)])
def test_quantize_refuses(gemm_lib, kw):
    a = dict(rows=100, cols=200, x=P, ldx=200, x_type=BF16, block=0, transpose=0, q=P, ldq=200,
             scales=P, lds=100)
    a.update(kw)
    assert gemm_lib.gemm_fp8_quantize(*a.values()) == INVALID


FP8 = dict(M=100, N=300, K=256, alpha=1.0, A=P, lda=256, sa=P, ldsa=100, B=P, ldb=256, sb=P, ldsb=3,
           block=1, beta=0.0, D=P, ldd=300, d_type=F32)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(A=0), dict(B=0), dict(sa=0), dict(sb=0),
    dict(D=0), dict(lda=255), dict(ldb=255), dict(ldsa=99), dict(ldsb=2), dict(block=0, ldsb=299),
    dict(block=5), dict(ldd=299), dict(d_type=E4M3), dict(D=P + 2), dict(sa=P + 2), dict(sb=P + 1)])
def test_fp8gemm_refuses(gemm_lib, kw):
    assert gemm_lib.gemm_fp8gemm(*{**FP8, **kw}.values()) == INVALID


def test_fp8gemm_empty_and_unread(gemm_lib):
    g = gemm_lib
    assert g.gemm_fp8gemm(*{**FP8, "M": 0}.values()) == OK
    assert g.gemm_fp8gemm(*{**FP8, "N": 0}.values()) == OK
    # alpha == 0: the operands are not looked at
    if not torch.cuda.is_available():
        assert g.gemm_fp8gemm(*{**FP8, "alpha": 0.0, "A": 0, "sa": 0}.values()) == UNSUPPORTED


FP8G = dict(G=4, off=P, M=100, N=300, K=256, alpha=1.0, A=P, lda=256, sa=P, ldsa=100, B=P, ldb=256,
            stride=76800, sb=P, ldsb=3, sstride=6, block=1, beta=0.0, D=P, ldd=300, d_type=F32)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INVALID), (dict(off=0), INVALID), (dict(off=P + 2), INVALID),
    (dict(stride=76799), INVALID), (dict(sstride=5), INVALID), (dict(lda=100), INVALID),
    (dict(D=0), INVALID), (dict(G=1025), UNSUPPORTED), (dict(G=0), OK)])
def test_fp8gemm_grouped_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_fp8gemm_grouped(*{**FP8G, **kw}.values()) == status


GROUPED = dict(G=4, off=P, rows=100, N=300, K=256, alpha=1.0, A=P, lda=256, B=P, ldb=300,
               stride=76800, transpose=0, beta=0.0, D=P, ldd=300, d_type=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INVALID), (dict(rows=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(off=0), INVALID), (dict(off=P + 1), INVALID), (dict(A=0), INVALID), (dict(B=0), INVALID),
    (dict(D=0), INVALID), (dict(lda=255), INVALID), (dict(ldb=299), INVALID),
    (dict(stride=76799), INVALID), (dict(transpose=1, ldb=255), INVALID), (dict(ldd=299), INVALID),
    (dict(d_type=2), INVALID), (dict(D=P + 1), INVALID), (dict(A=P + 1), MISALIGNED),
    (dict(B=P + 1), MISALIGNED), (dict(G=1025), UNSUPPORTED), (dict(G=0), OK), (dict(rows=0), OK)])
def test_bf16gemm_grouped_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_bf16gemm_grouped(*{**GROUPED, **kw}.values()) == status


WGRAD = dict(G=4, off=P, rows=100, N=300, K=256, alpha=1.0, A=P, lda=256, dD=P, lddd=300, beta=0.0,
             dB=P, ldb=300, stride=76800, d_type=F32)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INVALID), (dict(rows=-1), INVALID), (dict(off=0), INVALID), (dict(A=0), INVALID),
    (dict(dD=0), INVALID), (dict(dB=0), INVALID), (dict(lda=255), INVALID), (dict(lddd=299), INVALID),
    (dict(ldb=299), INVALID), (dict(stride=76799), INVALID), (dict(d_type=3), INVALID),
    (dict(dB=P + 2), INVALID), (dict(A=P + 1), MISALIGNED), (dict(dD=P + 1), MISALIGNED),
    (dict(G=1025), UNSUPPORTED), (dict(G=0), OK), (dict(N=0), OK), (dict(K=0), OK)])
def test_bf16gemm_grouped_wgrad_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_bf16gemm_grouped_wgrad(*{**WGRAD, **kw}.values()) == status


@needs_no_device
def test_no_device_no_fallback(gemm_lib):
    g = gemm_lib
    assert g.gemm_rmsnorm(8, 256, norm_args(g)) == UNSUPPORTED
    assert g.gemm_rmsnorm_backward(8, 256, grad_args(g)) == UNSUPPORTED
    assert g.gemm_fp8_quantize(100, 200, P, 200, BF16, 0, 0, P, 200, P, 100) == UNSUPPORTED
    assert g.gemm_fp8gemm(*FP8.values()) == UNSUPPORTED
    assert g.gemm_fp8gemm_grouped(*FP8G.values()) == UNSUPPORTED
    assert g.gemm_bf16gemm_grouped(*GROUPED.values()) == UNSUPPORTED
    assert g.gemm_bf16gemm_grouped_wgrad(*WGRAD.values()) == UNSUPPORTED


def test_tensor_helpers_refuse_host_tensors(gemm_lib):
    g = gemm_lib
    x, w = torch.zeros(4, 8), torch.ones(8)
    q, s = torch.zeros(4, 8).to(torch.float8_e4m3fn), torch.zeros(1, 4)
    off = torch.zeros(2, dtype=torch.int32)
    b = x.to(torch.bfloat16)
    for call in (lambda: g.rmsnorm(x, w, y=x), lambda: g.rmsnorm_backward(x, x, w, torch.ones(4), x),
                 lambda: g.fp8_quantize(x, q, s), lambda: g.fp8gemm(q, s, q, s, torch.zeros(4, 4)),
                 lambda: g.fp8gemm_grouped(q, s, q[None], s[None], off, torch.zeros(4, 4)),
                 lambda: g.bf16gemm_grouped(b, torch.zeros(1, 8, 3).to(torch.bfloat16), off,
                                            torch.zeros(4, 3)),
                 lambda: g.bf16gemm_grouped_wgrad(b, b, off, torch.zeros(1, 8, 8))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_tensor_helpers_refuse_wrong_tensors(gemm_lib, cuda_device):
    g = gemm_lib
    f8, bf, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    w, x, q, s = z(8), z(4, 8), z(4, 8, dtype=f8), z(1, 4)
    bad = [
        (TypeError, lambda: g.rmsnorm(x.half(), w, y=x)),
        (TypeError, lambda: g.rmsnorm(x, w.to(bf), y=x)),
        (ValueError, lambda: g.rmsnorm(x, z(7), y=x)),
        (ValueError, lambda: g.rmsnorm(x.t(), z(4), y=z(8, 4))),
        (ValueError, lambda: g.rmsnorm(x, w, q=q)),
        (ValueError, lambda: g.rmsnorm(x, w, q=q, scales=z(4, 1))),
        (TypeError, lambda: g.rmsnorm(x, w, y=torch.zeros(4, 8))),
        (TypeError, lambda: g.rmsnorm(torch.zeros(4, 8), w, y=x)),
        (ValueError, lambda: g.rmsnorm_backward(x, z(4, 9), w, z(4), x)),
        (ValueError, lambda: g.rmsnorm_backward(x, x, w, z(5), x)),
        (KeyError, lambda: g.fp8_quantize(x, q, s, block="columns")),
        (ValueError, lambda: g.fp8_quantize(x, q, s, transpose=True)),
        (TypeError, lambda: g.fp8_quantize(x, x, s)),
        (ValueError, lambda: g.fp8gemm(q, s, z(3, 7, dtype=f8), z(1, 3), z(4, 3))),
        (ValueError, lambda: g.fp8gemm(q, s, z(3, 8, dtype=f8), z(1, 2), z(4, 3))),
        (ValueError, lambda: g.fp8gemm(q, z(2, 4), z(3, 8, dtype=f8), z(1, 3), z(4, 3))),
        (TypeError, lambda: g.fp8gemm(q, s, z(3, 8, dtype=f8), z(1, 3), z(4, 3).half())),
        (ValueError, lambda: g.fp8gemm_grouped(q, s, z(2, 3, 8, dtype=f8), z(2, 1, 3), z(2, dtype=i32),
                                               z(4, 3))),
        (TypeError, lambda: g.fp8gemm_grouped(q, s, z(2, 3, 8, dtype=f8), z(2, 1, 3),
                                              z(3, dtype=torch.int64), z(4, 3))),
        (ValueError, lambda: g.bf16gemm_grouped(x.to(bf), z(2, 7, 3, dtype=bf), z(3, dtype=i32), z(4, 3))),
        (ValueError, lambda: g.bf16gemm_grouped_wgrad(x.to(bf), z(5, 3, dtype=bf), z(3, dtype=i32),
                                                      z(2, 8, 3))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    st = g.load_library().gemm_fp8gemm(4, 3, 8, 1.0, None, 8, None, 4, None, 8, None, 3, 0, 0.0,
                                       ctypes.c_void_p(x.data_ptr()), 3, 0, 0)
    assert st == INVALID
