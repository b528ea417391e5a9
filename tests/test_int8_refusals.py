"""Arguments that the int8 quantiser and product refuse (no GPU: every check comes before the first
device call)."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 3
P = 1 << 20
F32, BF16, E4M3, S8 = 0, 1, 2, 3
BIG = 1 << 31

needs_no_device = pytest.mark.skipif(torch.cuda.is_available(),
                                     reason="calls that pass the checks would launch")

QUANT = dict(rows=100, cols=200, x=P, ldx=200, x_type=BF16, transpose=0, q=P, ldq=200, scales=P)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(rows=BIG), INVALID), (dict(x=0), INVALID),
    (dict(q=0), INVALID), (dict(scales=0), INVALID), (dict(ldx=199), INVALID), (dict(ldq=199), INVALID),
    (dict(x_type=E4M3), INVALID), (dict(x=P + 1), INVALID), (dict(scales=P + 2), INVALID),
    (dict(transpose=1, ldq=99), INVALID), (dict(cols=(1 << 30) + 1, ldx=BIG - 1, ldq=BIG - 1), INVALID),
    (dict(rows=0, x=0), OK), (dict(cols=0, q=0), OK)])
def test_quantize_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_int8_quantize(*{**QUANT, **kw}.values()) == status


GEMM = dict(M=100, N=300, K=256, alpha=1.0, A=P, lda=256, sa=P, B=P, ldb=256, sb=P, bias=P, beta=0.0, D=P,
            ldd=300, d_type=F32)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(M=BIG - 255), INVALID),
    (dict(N=BIG - 255), INVALID), (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(sa=0), INVALID),
    (dict(sb=0), INVALID), (dict(D=0), INVALID), (dict(lda=255), INVALID), (dict(ldb=255), INVALID),
    (dict(ldd=299), INVALID), (dict(d_type=E4M3), INVALID), (dict(d_type=S8), INVALID),
    (dict(D=P + 2), INVALID), (dict(sa=P + 2), INVALID), (dict(sb=P + 1), INVALID), (dict(bias=P + 2), INVALID),
    (dict(K=1 << 17, lda=1 << 17, ldb=1 << 17), UNSUPPORTED), (dict(M=0), OK), (dict(N=0), OK)])
def test_int8gemm_refuses(gemm_lib, kw, status):
    assert gemm_lib.gemm_int8gemm(*{**GEMM, **kw}.values()) == status


@needs_no_device
def test_no_device_no_fallback(gemm_lib):
    g = gemm_lib
    assert g.gemm_int8_quantize(*QUANT.values()) == UNSUPPORTED
    assert g.gemm_int8gemm(*GEMM.values()) == UNSUPPORTED
    # alpha == 0: the operands are not looked at
    assert g.gemm_int8gemm(*{**GEMM, "alpha": 0.0, "A": 0, "sa": 0, "bias": 0}.values()) == UNSUPPORTED


def test_tensor_helpers_refuse_host_tensors(gemm_lib):
    g = gemm_lib
    x, q, v = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: g.int8_quantize(x, q, v), lambda: g.int8gemm(q, v, q, v, torch.zeros(4, 4))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_tensor_helpers_refuse_wrong_tensors(gemm_lib, cuda_device):
    g = gemm_lib

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    s8 = torch.int8
    x, q, v, b, d = z(4, 8), z(4, 8, dtype=s8), z(4), z(3, 8, dtype=s8), z(4, 3)
    bad = [
        (TypeError, lambda: g.int8_quantize(x.half(), q, v)),
        (TypeError, lambda: g.int8_quantize(x, x, v)),
        (ValueError, lambda: g.int8_quantize(x, q, v, transpose=True)),
        (ValueError, lambda: g.int8_quantize(x, q, z(8))),
        (TypeError, lambda: g.int8gemm(x, v, b, z(3), d)),
        (ValueError, lambda: g.int8gemm(q, z(3), b, z(3), d)),
        (ValueError, lambda: g.int8gemm(q, v, z(3, 7, dtype=s8), z(3), d)),
        (ValueError, lambda: g.int8gemm(q, v, b, z(4), d)),
        (ValueError, lambda: g.int8gemm(q, v, b, z(3), d, bias=z(4))),
        (TypeError, lambda: g.int8gemm(q, v, b, z(3), d.half())),
        (ValueError, lambda: g.int8gemm(q, v, z(8, 3, dtype=s8).t(), z(3), d)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
