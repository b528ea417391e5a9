"""Plain 64-bit forms of the operators around the GEMMs, and input helpers for
their tests.  They share no code with the library.

Error units used below: fp32 rounds by at most 2^-24 of the value (U32), bf16
by 2^-8 (UBF), E4M3 by 2^-4 of the value or 2^-10 where that is larger.
"""
from __future__ import annotations

import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8
FILL = 0x5A  # byte pattern planted around outputs
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def up(n, m=128):
    return -(-n // m)


def e4m3_round(v):
    """Nearest E4M3 value of fp64 v, ties to even, saturated."""
    v = v.clamp(-448.0, 448.0)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-5) - 4)
    return torch.round(v / step) * step


def block_amax(x, block):
    """Largest finite magnitude of each block, k-blocks first."""
    rows, cols = x.shape
    high = 128 if block == "tiles" else 1
    p = x.new_zeros(up(rows, high) * high, up(cols) * 128)
    p[:rows, :cols] = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs()
    return p.view(up(rows, high), high, up(cols), 128).amax(dim=(1, 3)).t()


def spread(scales, block, rows, cols):
    """One scale per value from scales[k-block][row or block of rows]."""
    i = torch.arange(rows, device=scales.device) // (128 if block == "tiles" else 1)
    j = torch.arange(cols, device=scales.device) // 128
    return scales.double().t()[i][:, j]


def check_fp8(q, scales, want, block, err):
    """q * scales must be `want` (fp64, known to within `err`) rounded to E4M3 under scales that
    are the blocks' largest magnitude / 448.  err: elementwise bound on the value quantised."""
    rows, cols = want.shape
    fine = torch.isfinite(want)
    amax = block_amax(want, block)
    off = block_amax(torch.where(fine, err, torch.zeros_like(err)), block)
    s = (amax / 448.0).clamp_min(2.0 ** -126)
    # the kernel's largest value is off by at most the block's largest error; one quotient
    assert bool(((scales.double() - s).abs() <= off / 448.0 + 2 * U32 * s).all()), "scales"
    sv = spread(scales, block, rows, cols)
    got = q.double() * sv
    # three fp32 roundings (448 / a, the product with it, and a / 448 in the scale) and E4M3's;
    # the largest value may end a few roundings above 448 and saturate
    bound = err + 4 * U32 * want.abs() + torch.maximum(want.abs() * 2.0 ** -4 * (1 + 2.0 ** -20),
                                                       2.0 ** -10 * sv)
    bad = fine & ~((got - want).abs() <= bound)
    assert not bool(bad.any()), "%d values, first at %s" % (int(bad.sum()), bad.nonzero()[0].tolist())
    assert bool(torch.isnan(q.double()[torch.isnan(want)]).all())
    inf = torch.isinf(want)
    assert bool((q.double()[inf] == 448.0 * torch.sign(want[inf])).all())


class Guarded:
    """A matrix (or a batch of them) inside a buffer of FILL bytes, `pad` elements between rows
    and `off` elements before the first; guards are checked untouched."""

    def __init__(self, shape, dtype, pad=0, off=0, device="cuda"):
        self.shape, self.size = tuple(shape), torch.empty(0, dtype=dtype).element_size()
        lead = 1
        for n in shape[:-1]:
            lead *= n
        self.pitch = shape[-1] + pad
        count = off + lead * self.pitch + 64
        self.raw = torch.full((count * self.size,), FILL, dtype=torch.uint8, device=device)
        flat = self.raw.view(dtype)
        strides = [1]
        step = self.pitch
        for n in reversed(shape[:-1]):
            strides.insert(0, step)
            step *= n
        self.t = torch.as_strided(flat, shape, strides, off)
        self.off = off

    def set(self, value):
        self.t.copy_(value)
        return self

    def clean_outside(self):
        keep = torch.ones(self.raw.numel() // self.size, dtype=torch.bool, device=self.raw.device)
        torch.as_strided(keep, self.shape, self.t.stride(), self.off).fill_(False)
        outside = self.raw.view(-1, self.size)[keep]
        return bool((outside == FILL).all())


def randn(*shape, seed=0, scale=1.0, dtype=torch.float32, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(device)


def fp8_matrix(rows, cols, block, seed, lead=(), pad=0, off=0):
    """(values, scales): random E4M3 values of every size with random positive scales."""
    gen = torch.Generator().manual_seed(seed)
    v = torch.randn(*lead, rows, cols, generator=gen) * torch.exp(
        2.0 * torch.randn(*lead, rows, 1, generator=gen))
    q = Guarded((*lead, rows, cols), torch.float8_e4m3fn, pad, off)
    q.t.copy_(v.clamp(-448, 448).to(torch.float8_e4m3fn))
    s = torch.exp(torch.randn(*lead, up(cols), up(rows) if block == "tiles" else rows, generator=gen))
    return q.t, s.cuda()


def offsets_of(counts, start=0):
    off = torch.tensor([start, *counts]).cumsum(0)
    return off.to(torch.int32).cuda()
