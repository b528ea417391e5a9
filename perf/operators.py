"""Cases of the operators around the GEMMs of a transformer's layers.

Five operators, in the order in which a layer uses them:

* ``norm``           root-mean-square norm with the residual's addition, written in bf16 or in fp8
                     (E4M3) with one fp32 scale per row and 128 columns; scale (b, i) belongs to
                     columns 128 b to 128 b + 127 of row (or block of rows) i
* ``norm_backward``  its gradients
* ``quantize``       a matrix, or its transpose, in fp8 with a scale per 1 x 128 or 128 x 128 block
* ``fp8gemm``        the product of two such matrices
* ``grouped``        products grouped by expert with ragged row counts: bf16 forward and backward,
                     and fp8 with block scales

``run`` computes them in plain torch operations in fp32 (``own`` false) or with
dense_gemm_12_gb300 (``own`` true); ``exact`` computes them from their definitions in fp64.
"""
import math

import torch

own = False

FP8_MAX = 448.0           # largest finite E4M3 value
SCALE_MIN = 2.0 ** -126   # smallest scale: blocks of zeros keep a usable one
BLOCK = 128
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the rows of one decoding step of a small batch, before its projections in 8 bits
        {"name": "norm_token", "op": "norm", "rows": 4, "dim": 4096, "x": "bf16",
         "residual": "bf16", "out": "fp8"},
        # a prompt's rows
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "dim": 8192, "x": "bf16",
         "residual": "bf16", "out": "fp8"},
        # a training step's gradient through the norm, the skip connection's gradient added
        {"name": "norm_backward", "op": "norm_backward", "rows": 8192, "dim": 4096, "x": "bf16",
         "residual": "bf16"},
        # activations of a ragged batch, transposed for the weight gradient's product
        {"name": "quantize_ragged_t", "op": "quantize", "rows": 3000, "cols": 1999, "x": "bf16",
         "block": "rows", "transpose": True},
        # a weight matrix laid out for the forward product
        {"name": "quantize_weight", "op": "quantize", "rows": 8192, "cols": 8192, "x": "bf16",
         "block": "tiles", "transpose": True},
        # one decoding step of 16 sequences
        {"name": "fp8_decode", "op": "fp8gemm", "m": 16, "n": 12288, "k": 4096, "block": "tiles",
         "out": "bf16"},
        # a weight gradient: both operands with a scale per row, ragged in every direction
        {"name": "fp8_ragged", "op": "fp8gemm", "m": 3000, "n": 5000, "k": 1999, "block": "rows",
         "out": "bf16"},
        # a large layer over a long batch
        {"name": "fp8_large", "op": "fp8gemm", "m": 8192, "n": 8192, "k": 8192, "block": "tiles",
         "out": "bf16"},
        # experts' forward products in training, loads uneven
        {"name": "grouped_forward", "op": "grouped", "kind": "forward", "rows": 16384,
         "groups": 16, "n": 4096, "k": 2048, "skew": 0.5},
        # their gradients with respect to the rows and the weights
        {"name": "grouped_backward", "op": "grouped", "kind": "backward", "rows": 8001,
         "groups": 24, "n": 2048, "k": 1024, "skew": 0.7},
        # one decoding step: few rows over many experts, some of them without any
        {"name": "grouped_fp8_decode", "op": "grouped", "kind": "fp8", "rows": 64, "groups": 64,
         "n": 2048, "k": 4096, "skew": 0.7},
        # a prompt through the experts in 8 bits
        {"name": "grouped_fp8_prompt", "op": "grouped", "kind": "fp8", "rows": 16384,
         "groups": 32, "n": 4096, "k": 2048, "skew": 0.5},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def maybe_even(v):  # most sizes in use are multiples of 64; the others are drawn as they are
        return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.6 else v

    op = rng.choice(["norm", "norm_backward", "quantize", "fp8gemm", "fp8gemm", "grouped", "grouped"])
    if op in ("norm", "norm_backward"):
        dim = maybe_even(size(64, 16384))
        rows = size(1, min(32768, (1 << 26) // dim))
        case = {"op": op, "rows": rows, "dim": dim, "x": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.choice(["none", "bf16", "f32"])}
        if op == "norm":
            case["out"] = rng.choice(["fp8", "bf16"])
        return case
    if op == "quantize":
        return {"op": op, "rows": maybe_even(size(1, 8192)), "cols": maybe_even(size(64, 8192)),
                "x": rng.choice(["bf16", "bf16", "f32"]), "block": rng.choice(["rows", "tiles"]),
                "transpose": rng.random() < 0.5}
    if op == "fp8gemm":
        return {"op": op, "m": size(1, 8192), "n": maybe_even(size(64, 8192)),
                "k": maybe_even(size(64, 8192)), "block": rng.choice(["tiles", "tiles", "rows"]),
                "out": "bf16"}
    groups = size(2, 64)
    kind = rng.choice(["forward", "backward", "fp8"])
    n, k = maybe_even(size(64, 4096)), maybe_even(size(64, 4096))
    return {"op": op, "kind": kind, "rows": size(1, 8192), "groups": groups, "n": n, "k": k,
            "skew": round(rng.uniform(0.0, 1.0), 2)}


def group_counts(case):
    """Rows of each expert, largest first: popularity falls off as rank^-skew."""
    g, rows = case["groups"], case["rows"]
    p = [(i + 1.0) ** -case["skew"] for i in range(g)]
    share = [rows * v / sum(p) for v in p]
    counts = [int(s) for s in share]
    rest = sorted(range(g), key=lambda i: counts[i] - share[i])
    for i in rest[: rows - sum(counts)]:
        counts[i] += 1
    return counts


# -------------------------------------------------------------------- inputs
def padded(rows, cols, dtype, device="cuda", lead=()):
    """A matrix whose row pitch is a multiple of 16 elements, as its owner allocates it."""
    pitch = -(-cols // 16) * 16
    return torch.empty(*lead, rows, pitch, dtype=dtype, device=device)[..., :cols]


def blocks(n):
    return -(-n // BLOCK)


def spread(s, block, rows, cols):
    """The scales (blocks of columns first) of a matrix, one for each of its values."""
    s = s.transpose(-1, -2).repeat_interleave(BLOCK, dim=-1)[..., :cols]
    return s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :] if block == "tiles" else s


def plain_quantize(x, block):
    """fp32 values -> (E4M3 values, fp32 scales, blocks of columns first)."""
    rows, cols = x.shape[-2:]
    pad = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % BLOCK if block == "tiles" else 0))
    if block == "tiles":
        cut = pad.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
        amax = cut.abs().amax(dim=(-3, -1))
    else:
        amax = pad.unflatten(-1, (-1, BLOCK)).abs().amax(dim=-1)
    scales = (amax / FP8_MAX).clamp_min(SCALE_MIN).transpose(-1, -2).contiguous()
    v = x / spread(scales, block, rows, cols)
    return v.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    op, st = case["op"], {"case": case}
    if op in ("norm", "norm_backward"):
        rows, dim = case["rows"], case["dim"]
        xt = DTYPES[case["x"]]
        rt = DTYPES.get(case["residual"])
        st["weight"] = 1.0 + normal(dim, scale=0.1)
        if op == "norm":
            st["x"] = normal(rows, dim, dtype=xt)
            # a few channels are much larger than the others, as in trained models
            st["x"][:, :: 97] *= 20.0
            st["residual"] = None if rt is None else normal(rows, dim, dtype=rt, scale=3.0)
            st["h"] = None if rt is None else torch.empty(rows, dim, dtype=rt, device="cuda")
            if case["out"] == "fp8":
                st["q"] = padded(rows, dim, torch.float8_e4m3fn)
                st["scales"] = torch.empty(blocks(dim), rows, device="cuda")
            else:
                st["y"] = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
            return st
        st["h"] = normal(rows, dim, dtype=rt or xt, scale=3.0)
        st["dy"] = normal(rows, dim, dtype=xt, scale=0.01)
        st["residual_grad"] = None if rt is None else normal(rows, dim, dtype=rt, scale=0.01)
        st["rstd"] = (st["h"].float().square().mean(-1) + EPS).rsqrt()
        st["dh"] = torch.empty(rows, dim, dtype=rt or xt, device="cuda")
        st["dweight"] = torch.empty(dim, device="cuda")
        return st
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = normal(rows, cols)
        x[:, :: 97] *= 20.0
        st["x"] = x.to(DTYPES[case["x"]])
        if case["transpose"]:
            rows, cols = cols, rows
        st["q"] = padded(rows, cols, torch.float8_e4m3fn)
        st["scales"] = torch.empty(blocks(cols), blocks(rows) if case["block"] == "tiles" else rows,
                                   device="cuda")
        return st

    def in_fp8(block, rows, cols, lead=(), scale=1.0):
        v, s = plain_quantize(normal(*lead, rows, cols, scale=scale), block)
        q = padded(rows, cols, torch.float8_e4m3fn, lead=lead)
        q.copy_(v)
        return q, s

    if op == "fp8gemm":
        st["a"], st["a_scales"] = in_fp8("rows", case["m"], case["k"])
        st["b"], st["b_scales"] = in_fp8(case["block"], case["n"], case["k"], scale=0.02)
        st["d"] = torch.empty(case["m"], case["n"], dtype=DTYPES[case["out"]], device="cuda")
        return st

    rows, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    counts = torch.tensor(group_counts(case))
    counts = counts[torch.randperm(g, generator=torch.Generator().manual_seed(int(seed)))]
    st["offsets"] = torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32).cuda()
    st["most"] = int(counts.max())
    if case["kind"] == "fp8":
        st["a"], st["a_scales"] = in_fp8("rows", rows, k)
        st["b"], st["b_scales"] = in_fp8("tiles", n, k, lead=(g,), scale=0.02)
        st["d"] = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        return st
    st["a"] = padded(rows, k, torch.bfloat16)
    st["a"].copy_(normal(rows, k))
    st["b"] = padded(k, n, torch.bfloat16, lead=(g,))
    st["b"].copy_(normal(g, k, n, scale=0.02))
    if case["kind"] == "forward":
        st["d"] = padded(rows, n, torch.bfloat16)
        return st
    st["grad"] = padded(rows, n, torch.bfloat16)
    st["grad"].copy_(normal(rows, n, scale=0.01))
    st["da"] = padded(rows, k, torch.bfloat16)
    st["db"] = padded(k, n, torch.bfloat16, lead=(g,))
    return st


# ---------------------------------------------------------------- plain forms
def plain_norm(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["weight"]
    kept = [] if st["residual"] is None else [h.to(st["residual"].dtype)]
    if st["case"]["out"] == "fp8":
        return [*kept, *plain_quantize(y, "rows")]
    return [*kept, y.to(torch.bfloat16)]


def plain_norm_backward(st):
    h, rstd = st["h"].float(), st["rstd"][:, None]
    dy, xh = st["dy"].float(), h * rstd
    gw = dy * st["weight"]
    dh = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    if st["residual_grad"] is not None:
        dh = dh + st["residual_grad"].float()
    return [dh.to(st["dh"].dtype), (dy * xh).sum(0)]


def by_group(rows_of, offsets, most):
    """Rows gathered group by group, each group padded with zeros to `most` rows, and their places."""
    total = rows_of.shape[0]
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    real = at < offsets[1:, None]
    got = rows_of[at.clamp(max=total - 1)] * real[..., None]
    return got, torch.where(real, at, total)


def to_rows(grouped, at, total):
    out = grouped.new_zeros(total + 1, grouped.shape[-1])
    out[at] = grouped
    return out[:total]


def plain_grouped(st):
    case, off, most = st["case"], st["offsets"], st["most"]
    rows, n, k = case["rows"], case["n"], case["k"]
    if case["kind"] == "fp8":
        a = st["a"].float() * spread(st["a_scales"], "rows", rows, k)
        b = st["b"].float() * spread(st["b_scales"], "tiles", n, k)
        ag, at = by_group(a, off, most)
        return to_rows(ag @ b.transpose(1, 2), at, rows).to(torch.bfloat16)
    ag, at = by_group(st["a"].float(), off, most)
    if case["kind"] == "forward":
        return to_rows(ag @ st["b"].float(), at, rows).to(torch.bfloat16)
    gg, _ = by_group(st["grad"].float(), off, most)
    da = to_rows(gg @ st["b"].float().transpose(1, 2), at, rows)
    return [da.to(torch.bfloat16), (ag.transpose(1, 2) @ gg).to(torch.bfloat16)]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return run_own(st)
    if op == "norm":
        return plain_norm(st)
    if op == "norm_backward":
        return plain_norm_backward(st)
    if op == "quantize":
        x = st["x"].float()
        return list(plain_quantize(x.t() if case["transpose"] else x, case["block"]))
    if op == "fp8gemm":
        a = st["a"].float() * spread(st["a_scales"], "rows", case["m"], case["k"])
        b = st["b"].float() * spread(st["b_scales"], case["block"], case["n"], case["k"])
        return (a @ b.t()).to(st["d"].dtype)
    return plain_grouped(st)


def run_own(st):
    import dense_gemm_12_gb300 as g
    case = st["case"]
    op = case["op"]
    if op == "norm":
        kept = [] if st["residual"] is None else [st["h"]]
        if case["out"] == "fp8":
            g.rmsnorm(st["x"], st["weight"], eps=EPS, residual=st["residual"], h=st["h"],
                      q=st["q"], scales=st["scales"])
            return [*kept, st["q"], st["scales"]]
        g.rmsnorm(st["x"], st["weight"], eps=EPS, residual=st["residual"], h=st["h"], y=st["y"])
        return [*kept, st["y"]]
    if op == "norm_backward":
        g.rmsnorm_backward(st["dy"], st["h"], st["weight"], st["rstd"], st["dh"], st["dweight"],
                           residual_grad=st["residual_grad"])
        return [st["dh"], st["dweight"]]
    if op == "quantize":
        g.fp8_quantize(st["x"], st["q"], st["scales"], block=case["block"],
                       transpose=case["transpose"])
        return [st["q"], st["scales"]]
    if op == "fp8gemm":
        return g.fp8gemm(st["a"], st["a_scales"], st["b"], st["b_scales"], st["d"])
    if case["kind"] == "fp8":
        return g.fp8gemm_grouped(st["a"], st["a_scales"], st["b"], st["b_scales"], st["offsets"],
                                 st["d"])
    if case["kind"] == "forward":
        return g.bf16gemm_grouped(st["a"], st["b"], st["offsets"], st["d"])
    g.bf16gemm_grouped(st["grad"], st["b"], st["offsets"], st["da"], transpose_b=True)
    g.bf16gemm_grouped_wgrad(st["a"], st["grad"], st["offsets"], st["db"])
    return [st["da"], st["db"]]


# ------------------------------------------------------------------ 64 bits
def exact_e4m3(v):
    """Nearest E4M3 value (ties to even), saturated: 3 fraction bits, exponents from -6."""
    v = v.clamp(-FP8_MAX, FP8_MAX)
    _, e = torch.frexp(v)                      # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-5) - 4)
    return (v / step).round() * step


def exact_quantize(x, block):
    """From the definition, block by block, on a copy padded with zeros."""
    rows, cols = x.shape
    high = BLOCK if block == "tiles" else 1
    br, bc = -(-rows // high), blocks(cols)
    cut = x.new_zeros(br * high, bc * BLOCK)
    cut[:rows, :cols] = x
    cut = cut.view(br, high, bc, BLOCK)
    s = torch.clamp(cut.abs().amax(dim=3).amax(dim=1) / FP8_MAX, min=SCALE_MIN)
    q = exact_e4m3(cut / s[:, None, :, None]).view(br * high, bc * BLOCK)
    return q[:rows, :cols], s.t()


def exact_values(q, s, high):
    """The fp64 values of a matrix in fp8 whose blocks are `high` x 128."""
    i = torch.arange(q.shape[0], device=q.device) // high
    j = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * s.double().t()[i][:, j]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h += st["residual"].double()
        rms = torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["dim"] + EPS)
        y = h / rms * st["weight"].double()
        kept = [] if st["residual"] is None else [h]
        return [*kept, *(exact_quantize(y, "rows") if case["out"] == "fp8" else [y])]
    if op == "norm_backward":
        h, dy, w = st["h"].double(), st["dy"].double(), st["weight"].double()
        v = (h * h).sum(1, keepdim=True) / case["dim"] + EPS
        dot = (dy * w * h).sum(1, keepdim=True)
        dh = dy * w / v.sqrt() - h * dot / (case["dim"] * v * v.sqrt())
        if st["residual_grad"] is not None:
            dh += st["residual_grad"].double()
        return [dh, (dy * h / v.sqrt()).sum(0)]
    if op == "quantize":
        x = st["x"].double()
        return list(exact_quantize(x.t().contiguous() if case["transpose"] else x, case["block"]))
    if op == "fp8gemm":
        a = exact_values(st["a"], st["a_scales"], 1)
        return a @ exact_values(st["b"], st["b_scales"], BLOCK if case["block"] == "tiles" else 1).t()
    rows, n, k = case["rows"], case["n"], case["k"]
    if 2.0 * rows * n * k > 1.2e13:
        return None
    ends = st["offsets"].tolist()
    d = torch.zeros(rows, k if case["kind"] == "backward" else n, dtype=torch.float64, device="cuda")
    db = torch.zeros(case["groups"], k, n, dtype=torch.float64, device="cuda")
    for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if case["kind"] == "fp8":
            w = exact_values(st["b"][g], st["b_scales"][g], BLOCK).t()
            d[lo:hi] = exact_values(st["a"][lo:hi], st["a_scales"][:, lo:hi], 1) @ w
        elif case["kind"] == "forward":
            d[lo:hi] = st["a"][lo:hi].double() @ st["b"][g].double()
        else:
            d[lo:hi] = st["grad"][lo:hi].double() @ st["b"][g].double().t()
            db[g] = st["a"][lo:hi].double().t() @ st["grad"][lo:hi].double()
    return [d, db] if case["kind"] == "backward" else d


# -------------------------------------------------------------------- floors
def work(case):
    """Bytes read and written once, and operations, of one pass."""
    size = {"f32": 4, "bf16": 2, "none": 0}
    op = case["op"]
    if op == "norm":
        v = case["rows"] * case["dim"]
        out = v + 4 * case["rows"] * blocks(case["dim"]) if case["out"] == "fp8" else 2 * v
        return {"bytes": v * (size[case["x"]] + 2 * size[case["residual"]]) + out + 4 * case["dim"],
                "flops": 5 * v}
    if op == "norm_backward":
        v = case["rows"] * case["dim"]
        r = size[case["residual"]]
        x = size[case["x"]]
        return {"bytes": v * (x + 2 * (r or x) + r) + 4 * case["rows"] + 8 * case["dim"],
                "flops": 10 * v}
    if op == "quantize":
        v = case["rows"] * case["cols"]
        rows, cols = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        s = (blocks(rows) if case["block"] == "tiles" else rows) * blocks(cols)
        return {"bytes": v * (size[case["x"]] + 1) + 4 * s, "flops": 3 * v}
    n, k = case["n"], case["k"]
    if op == "fp8gemm":
        m = case["m"]
        s = m + (blocks(n) if case["block"] == "tiles" else n)
        return {"bytes": m * k + n * k + 4 * s * blocks(k) + m * n * size[case["out"]],
                "flops": 2.0 * m * n * k}
    rows = case["rows"]
    used = sum(c > 0 for c in group_counts(case))
    if case["kind"] == "fp8":
        return {"bytes": rows * (k + 4 * blocks(k) + 2 * n) + used * (n * k + 4 * blocks(n) * blocks(k)),
                "flops": 2.0 * rows * n * k}
    if case["kind"] == "forward":
        return {"bytes": 2 * rows * (k + n) + 2 * used * n * k, "flops": 2.0 * rows * n * k}
    # the rows and their gradients in, both gradients out (of every expert, with or without rows)
    return {"bytes": 2 * rows * (n + 2 * k) + 2 * (used + case["groups"]) * n * k,
            "flops": 4.0 * rows * n * k}
