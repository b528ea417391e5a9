"""gemm_int8gemm where a sum passes 2^24 on its way and comes back.

Values of 110 to 127 in both operands, the second half of k with the other sign in B: after 2048 of k a sum
is above 2^24 (2048 * 110^2 = 2.5e7), where fp32 holds every other whole number at best, and the whole sum
is below 2^24, which an fp32 output holds exactly.  Sums carried on in integers give it; sums kept in
fp32 lose odd numbers on the way, and a sum that stops or starts anew on the way misses by millions."""
import pytest
import torch

import dense_gemm_12_gb300 as g

K = 4096


def operands(M, N, device="cpu"):
    gen = torch.Generator().manual_seed(M + N)
    a, b = (torch.randint(110, 128, (n, K), generator=gen).to(torch.int8) for n in (M, N))
    b[:, K // 2:] *= -1
    return a.to(device), b.to(device)


def test_sums_kept_in_fp32_would_differ():
    a, b = (v.double() for v in operands(16, 300))
    want = a @ b.t()
    assert float(want.abs().max()) < 2.0 ** 24
    total = torch.zeros(16, 300)
    for k in range(0, K, 16):   # an MMA's 16 products, then the accumulator's rounding
        total = (total.double() + a[:, k:k + 16] @ b[:, k:k + 16].t()).float()
    assert float((total.double() != want).double().mean()) > 0.5


# 16, 32, 64 and 128 tokens to a tile, its k split over a cluster's CTAs (few tiles) or not; more tokens; widened
# beforehand
@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(2, 2), (16, 300), (16, 38912), (20, 300), (32, 38912), (50, 300), (64, 38912),
                                 (100, 300), (120, 12200), (127, 24001), (200, 30000), (513, 1000), (2304, 2304),
                                 (3000, 4096)])
def test_sums_beyond_two_to_the_24(gemm_lib, cuda_device, M, N):
    A, B = operands(M, N, "cuda")
    one, D = torch.ones(max(M, N), device="cuda"), torch.empty(M, N, device="cuda")
    g.int8gemm(A, one[:M], B, one[:N], D)
    assert g.gemm_check_device_error(0) == 0
    assert torch.equal(D.double(), A.double() @ B.double().t())
