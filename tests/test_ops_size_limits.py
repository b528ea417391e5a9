"""Sizes next to 2^31 (no GPU: the checks come before the first device call).

The product kernels round up to tiles of at most 256 in 32 bits, so 2^31 - 256
is the largest size they are right for; one more is refused, before it could
wrap to a negative number of tiles and leave the output unwritten."""
import pytest
import torch

INVALID, UNSUPPORTED = 1, 3
P = 1 << 20  # an address that is only ever looked at
F32 = 0
MOST = (1 << 31) - 256
LD = (1 << 31) - 1

needs_no_device = pytest.mark.skipif(torch.cuda.is_available(),
                                     reason="calls that pass the checks would launch")


def fp8(g, M=16, N=16, K=16):
    return g.gemm_fp8gemm(M, N, K, 1.0, P, LD, P, LD, P, LD, P, LD, 1, 0.0, P, LD, F32)


def fp8_grouped(g, M=16, N=16, K=16):
    return g.gemm_fp8gemm_grouped(1, P, M, N, K, 1.0, P, LD, P, LD, P, LD, 0, P, LD, 0, 1, 0.0, P, LD, F32)


def grouped(g, M=16, N=16, K=16):
    return g.gemm_bf16gemm_grouped(1, P, M, N, K, 1.0, P, LD, P, LD, 0, 0, 0.0, P, LD, F32)


def grouped_t(g, M=16, N=16, K=16):
    return g.gemm_bf16gemm_grouped(1, P, M, N, K, 1.0, P, LD, P, LD, 0, 1, 0.0, P, LD, F32)


def wgrad(g, M=16, N=16, K=16):
    return g.gemm_bf16gemm_grouped_wgrad(1, P, M, N, K, 1.0, P, LD, P, LD, 0.0, P, LD, 0, F32)


CASES = [(call, dim) for call in (fp8, fp8_grouped, grouped, grouped_t, wgrad) for dim in "MNK"]


@pytest.mark.parametrize("call,dim", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_sizes_that_would_wrap_are_refused(gemm_lib, call, dim):
    most = LD if dim == "K" and call in (fp8, fp8_grouped) else MOST  # fp8: K is never rounded up in 32 bits
    for size in {most + 1, LD, 1 << 31} - {most}:
        assert call(gemm_lib, **{dim: size}) == INVALID


@needs_no_device
@pytest.mark.parametrize("call,dim", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_largest_sizes_pass_the_checks(gemm_lib, call, dim):
    assert call(gemm_lib, **{dim: MOST}) == UNSUPPORTED  # no device


def test_rounding_up_at_the_largest_size_stays_in_32_bits():
    # what the kernels add: a tile's rows or columns less one, or a position plus a tile's rest
    for tile in (16, 32, 64, 128, 256):
        assert MOST + tile - 1 < 1 << 31
    assert MOST // 256 * 256 + 255 < 1 << 31            # the last column of the last tile
    assert (MOST - 1) + 128 + 96 < 1 << 31              # a group's last row, in a pair's second half
    assert MOST + 256 >= 1 << 31                        # and one tile more would wrap
