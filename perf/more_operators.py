"""Cases of the operators around the products of a transformer's layers: experts' rows, layer norm, int8.

* ``route``      a router's softmax and top k of each token, and the pairs (token, choice) sorted by
                 expert: their places among the experts' rows, and where each expert's rows begin
* ``rows``       the tokens' rows to their experts' places (``dispatch``, bf16 or fp8 with scales),
                 the experts' rows back to the tokens with weights (``combine``), and the gradients of
                 rows, weights and logits (``backward``)
* ``layernorm``  layer norm with the residual's addition, forward and backward
* ``int8``       a linear layer in 8-bit integers with a scale for each token and channel, its input
                 quantised by itself or by the layer norm in front of it

``run`` computes them in plain torch operations in fp32 (``own`` false) or with
dense_gemm_12_gb300 (``own`` true); ``exact`` computes them from their definitions in fp64.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128               # columns of an fp8 scale
INT8_MAX = 127.0
SCALE_MIN = 2.0 ** -126   # smallest scale: rows of zeros keep a usable one
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a small batch
        {"name": "route_token", "op": "route", "rows": 16, "experts": 64, "top": 8, "logits": "f32",
         "normalize": True, "drop": 0.0},
        # a long prompt over many experts, a few tokens of it padding
        {"name": "route_prompt", "op": "route", "rows": 16384, "experts": 256, "top": 8,
         "logits": "f32", "normalize": True, "drop": 0.02},
        # the rows of a decoding step to their experts
        {"name": "dispatch_token", "op": "rows", "kind": "dispatch", "rows": 16, "dim": 4096, "top": 8,
         "experts": 64, "x": "bf16", "residual": "none", "drop": 0.0},
        # a prompt's rows in fp8, with their scales
        {"name": "dispatch_prompt", "op": "rows", "kind": "dispatch", "rows": 16384, "dim": 4096,
         "top": 4, "experts": 128, "x": "fp8", "residual": "none", "drop": 0.0},
        # the experts' rows of a ragged batch back to their tokens, onto the residual stream
        {"name": "combine_prompt", "op": "rows", "kind": "combine", "rows": 8001, "dim": 4096, "top": 8,
         "experts": 64, "x": "bf16", "residual": "bf16", "drop": 0.0},
        # a training step: from the layer's output to the experts' rows and the router's logits
        {"name": "rows_backward", "op": "rows", "kind": "backward", "rows": 8192, "dim": 2048, "top": 4,
         "experts": 64, "x": "bf16", "residual": "none", "drop": 0.02},
        # the rows of one decoding step
        {"name": "layernorm_token", "op": "layernorm", "kind": "forward", "rows": 4, "dim": 4096,
         "x": "bf16", "residual": "bf16"},
        # a prompt's rows
        {"name": "layernorm_prompt", "op": "layernorm", "kind": "forward", "rows": 8192, "dim": 8192,
         "x": "bf16", "residual": "bf16"},
        # a training step's gradients through the norm, the skip connection's gradient added
        {"name": "layernorm_backward", "op": "layernorm", "kind": "backward", "rows": 8192, "dim": 4096,
         "x": "bf16", "residual": "bf16"},
        # one decoding step of 16 sequences: the norm writes the product's 8-bit rows
        {"name": "int8_decode", "op": "int8", "m": 16, "n": 12288, "k": 4096, "norm": True,
         "bias": True, "out": "bf16"},
        # ragged in every direction
        {"name": "int8_ragged", "op": "int8", "m": 3000, "n": 5000, "k": 1999, "norm": False,
         "bias": False, "out": "bf16"},
        # a large layer over a long batch
        {"name": "int8_large", "op": "int8", "m": 8192, "n": 8192, "k": 8192, "norm": False,
         "bias": True, "out": "bf16"},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def maybe_even(v):  # most sizes in use are multiples of 64; the others are drawn as they are
        return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.6 else v

    op = rng.choice(["route", "rows", "rows", "layernorm", "layernorm", "int8", "int8"])
    experts = rng.choice([size(2, 256), 2 ** rng.randint(2, 8)])
    top = min(rng.randint(1, 8), experts)
    drop = rng.choice([0.0, 0.0, 0.1])
    if op == "route":
        return {"op": op, "rows": size(1, 16384), "experts": experts, "top": top,
                "logits": rng.choice(["f32", "f32", "bf16"]), "normalize": rng.random() < 0.5,
                "drop": drop}
    if op == "rows":
        kind = rng.choice(["dispatch", "combine", "backward"])
        dim = maybe_even(size(64, 8192))
        x = rng.choice(["bf16", "bf16", "fp8" if kind == "dispatch" else "f32"])
        rows = size(1, min(32768, (1 << 29) // (dim * (2 * top + 2) * (4 if x == "f32" else 2))))
        return {"op": op, "kind": kind, "rows": rows, "dim": dim, "top": top, "experts": experts,
                "x": x, "residual": rng.choice(["none", "bf16"]) if kind == "combine" else "none",
                "drop": drop}
    if op == "layernorm":
        dim = maybe_even(size(64, 16384))
        return {"op": op, "kind": rng.choice(["forward", "backward"]),
                "rows": size(1, min(32768, (1 << 25) // dim)), "dim": dim,
                "x": rng.choice(["bf16", "bf16", "f32"]),
                "residual": rng.choice(["none", "bf16", "f32"])}
    return {"op": op, "m": size(1, 8192), "n": maybe_even(size(64, 8192)),
            "k": maybe_even(size(512, 8192)), "norm": rng.random() < 0.3, "bias": rng.random() < 0.5,
            "out": "bf16"}


# -------------------------------------------------------------------- inputs
def padded(rows, cols, dtype):
    """A matrix whose row pitch is a multiple of 16 bytes, as its owner allocates it."""
    pitch = -(-cols // 16) * 16
    return torch.zeros(rows, pitch, dtype=dtype, device="cuda")[..., :cols]


def blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    def logits_of(rows, experts, dtype):
        # some experts are more popular than others; padding's rows have all of them masked
        v = normal(rows, experts, scale=1.5) + normal(experts)
        pad = torch.rand(rows, generator=gen, device="cuda") < case["drop"]
        return v.masked_fill_(pad[:, None], -math.inf).to(dtype)

    op, st = case["op"], {"case": case}
    if op == "route":
        rows, experts, top = case["rows"], case["experts"], case["top"]
        st["logits"] = logits_of(rows, experts, DTYPES[case["logits"]])
        st["expert"] = torch.empty(rows, top, dtype=torch.int32, device="cuda")
        st["weight"] = torch.empty(rows, top, device="cuda")
        st["slot"] = torch.empty_like(st["expert"])
        st["offsets"] = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        return st
    if op == "rows":
        rows, dim, top, experts = case["rows"], case["dim"], case["top"], case["experts"]
        st["logits"] = logits_of(rows, experts, torch.float32)
        st["expert"], st["weight"] = plain_route(st["logits"], top, False)
        st["slot"], _ = plain_sort(st["expert"], experts)
        if case["kind"] == "dispatch":
            if case["x"] == "fp8":
                st["x"] = padded(rows, dim, torch.float8_e4m3fn)
                st["x"].copy_(normal(rows, dim, scale=100.0).clamp_(-448, 448))
                st["x_scales"] = normal(blocks(dim), rows).abs_()
                st["a_scales"] = torch.zeros(blocks(dim), rows * top, device="cuda")
                st["a"] = padded(rows * top, dim, torch.float8_e4m3fn)
            else:
                st["x"] = normal(rows, dim, dtype=DTYPES[case["x"]])
                st["a"] = torch.zeros(rows * top, dim, dtype=DTYPES[case["x"]], device="cuda")
            return st
        xt = DTYPES[case["x"]]
        st["a"] = normal(rows * top, dim, dtype=xt)
        if case["kind"] == "combine":
            st["residual"] = None if case["residual"] == "none" else normal(
                rows, dim, dtype=DTYPES[case["residual"]], scale=3.0)
            st["out"] = torch.empty(rows, dim, dtype=xt, device="cuda")
            return st
        st["dout"] = normal(rows, dim, dtype=xt, scale=0.01)
        st["da"] = torch.zeros(rows * top, dim, dtype=xt, device="cuda")
        st["dweight"] = torch.empty(rows, top, device="cuda")
        st["dlogits"] = torch.empty(rows, experts, device="cuda")
        return st
    if op == "layernorm":
        rows, dim = case["rows"], case["dim"]
        xt, rt = DTYPES[case["x"]], DTYPES.get(case["residual"])
        st["gain"], st["bias"] = 1.0 + normal(dim, scale=0.1), normal(dim, scale=0.1)
        # a few channels are much larger than the others, as in trained models, and none has mean 0
        if case["kind"] == "forward":
            st["x"] = normal(rows, dim, dtype=xt)
            st["x"][:, :: 97] *= 20.0
            st["residual"] = None if rt is None else (normal(rows, dim, scale=3.0) + 0.5).to(rt)
            st["h"] = None if rt is None else torch.empty(rows, dim, dtype=rt, device="cuda")
            st["y"] = torch.empty(rows, dim, dtype=xt, device="cuda")
            return st
        h = normal(rows, dim, scale=3.0) + 0.5
        st["h"] = h.to(rt or xt)
        st["dy"] = normal(rows, dim, dtype=xt, scale=0.01)
        st["residual_grad"] = None if rt is None else normal(rows, dim, dtype=rt, scale=0.01)
        h = st["h"].float()
        st["mean"] = h.mean(-1)
        st["rstd"] = ((h - st["mean"][:, None]).square().mean(-1) + EPS).rsqrt()
        st["dh"] = torch.empty_like(st["h"])
        st["dgain"], st["dbias"] = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
        return st

    m, n, k = case["m"], case["n"], case["k"]
    st["x"] = normal(m, k, dtype=torch.bfloat16)
    st["x"][:, :: 97] *= 20.0
    if case["norm"]:
        st["gain"], st["norm_bias"] = 1.0 + normal(k, scale=0.1), normal(k, scale=0.1)
        st["residual"] = normal(m, k, dtype=torch.bfloat16, scale=3.0)
        st["h"] = torch.empty_like(st["residual"])
    w, st["w_scales"] = plain_int8(normal(n, k, scale=0.02))
    st["w"] = padded(n, k, torch.int8)
    st["w"].copy_(w)
    st["bias"] = normal(n) if case["bias"] else None
    st["q"], st["scales"] = padded(m, k, torch.int8), torch.empty(m, device="cuda")
    st["d"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device="cuda")
    return st


# ---------------------------------------------------------------- plain forms
def plain_shares(l):
    """exp of each row's logits less their largest, and its sum (1 where all are masked)."""
    top = l.amax(-1, keepdim=True)
    e = (l - torch.where(torch.isinf(top), 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total == 0, 1.0, total)


def plain_route(logits, top, normalize):
    l = logits.float()
    value, index = l.sort(dim=-1, descending=True, stable=True)
    value, index = value[:, :top], index[:, :top]
    real = value > -math.inf
    e, total = plain_shares(l)
    w = torch.where(real, e.gather(-1, index), 0.0)
    if normalize:
        total = w.sum(-1, keepdim=True)
        total = torch.where(total == 0, 1.0, total)
    return torch.where(real, index, -1).to(torch.int32), w / total


def plain_sort(expert, experts):
    flat = expert.reshape(-1).long()
    key, order = torch.where(flat < 0, experts, flat).sort(stable=True)
    place = torch.arange(flat.shape[0], device=flat.device)
    slot = torch.empty_like(flat)
    slot[order] = torch.where(key < experts, place, -1)
    ends = (key[:, None] < torch.arange(experts + 1, device=key.device)).sum(0)
    return slot.view(expert.shape).to(torch.int32), ends.to(torch.int32)


def plain_rows(st):
    case, slot = st["case"], st["slot"].long()
    n = slot.numel()
    real = slot >= 0
    at = torch.where(real, slot, n)      # pairs without a row: one row behind the last
    if case["kind"] == "dispatch":
        def moved(x, to):
            wide = torch.zeros(n + 1, x.shape[1], dtype=x.dtype, device=x.device)
            wide[at.reshape(-1)] = x.repeat_interleave(case["top"], dim=0)
            return to.copy_(wide[:n])
        if case["x"] == "fp8":
            moved(st["x"].view(torch.uint8), st["a"].view(torch.uint8))
            return [st["a"], moved(st["x_scales"].t(), st["a_scales"].t()).t()]
        return moved(st["x"], st["a"])
    a = torch.cat([st["a"], st["a"].new_zeros(1, case["dim"])])[at].float()   # (rows, top, dim)
    if case["kind"] == "combine":
        out = (a * torch.where(real, st["weight"], 0.0)[..., None]).sum(1)
        if st["residual"] is not None:
            out = out + st["residual"].float()
        return out.to(st["out"].dtype)
    dout = st["dout"].float()
    da = torch.zeros(n + 1, case["dim"], device="cuda")
    da[at] = dout[:, None] * st["weight"][..., None]
    dw = (a * dout[:, None]).sum(-1)
    e, total = plain_shares(st["logits"])
    p = e / total
    g = torch.zeros(case["rows"], case["experts"] + 1, device="cuda")
    g.scatter_(1, torch.where(real, st["expert"].long(), case["experts"]), dw)
    g = g[:, :case["experts"]]
    return [da[:n].to(st["da"].dtype), dw, p * (g - (g * p).sum(-1, keepdim=True))]


def plain_layernorm(h, gain, bias):
    mid = h - h.mean(-1, keepdim=True)
    return mid * (mid.square().mean(-1, keepdim=True) + EPS).rsqrt() * gain + bias


def plain_layernorm_backward(st):
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xh = (st["h"].float() - st["mean"][:, None]) * rstd
    g = dy * st["gain"]
    dh = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if st["residual_grad"] is not None:
        dh = dh + st["residual_grad"].float()
    return [dh.to(st["dh"].dtype), (dy * xh).sum(0), dy.sum(0)]


def plain_int8(v):
    amax = v.abs().amax(-1, keepdim=True)
    q = (v * (INT8_MAX / amax).clamp_max(1.0 / SCALE_MIN)).round().clamp(-INT8_MAX, INT8_MAX)
    return q, (amax / INT8_MAX).clamp_min(SCALE_MIN)[:, 0]


def plain_int8_linear(st):
    x, kept = st["x"].float(), []
    if st["case"]["norm"]:
        x = x + st["residual"].float()
        kept = [x.to(torch.bfloat16)]
        x = plain_layernorm(x, st["gain"], st["norm_bias"])
    q, s = plain_int8(x)
    d = (q @ st["w"].float().t()) * s[:, None] * st["w_scales"]
    if st["bias"] is not None:
        d = d + st["bias"]
    return [*kept, d.to(st["d"].dtype)]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return run_own(st)
    if op == "route":
        expert, weight = plain_route(st["logits"], case["top"], case["normalize"])
        return [expert, weight, *plain_sort(expert, case["experts"])]
    if op == "rows":
        return plain_rows(st)
    if op == "int8":
        return plain_int8_linear(st)
    if case["kind"] == "backward":
        return plain_layernorm_backward(st)
    h, kept = st["x"].float(), []
    if st["residual"] is not None:
        h = h + st["residual"].float()
        kept = [h.to(st["h"].dtype)]
    return [*kept, plain_layernorm(h, st["gain"], st["bias"]).to(st["y"].dtype)]


def run_own(st):
    import dense_gemm_12_gb300 as g
    case = st["case"]
    op = case["op"]
    if op == "route":
        g.expert_route(st["logits"], st["expert"], st["weight"], normalize=case["normalize"])
        g.expert_sort(st["expert"], st["slot"], st["offsets"])
        return [st["expert"], st["weight"], st["slot"], st["offsets"]]
    if op == "rows":
        if case["kind"] == "dispatch":
            if case["x"] == "fp8":
                g.expert_dispatch(st["x"], st["slot"], st["a"], x_scales=st["x_scales"],
                                  a_scales=st["a_scales"])
                return [st["a"], st["a_scales"]]
            return g.expert_dispatch(st["x"], st["slot"], st["a"])
        if case["kind"] == "combine":
            return g.expert_combine(st["a"], st["slot"], st["out"], weight=st["weight"],
                                    residual=st["residual"])
        g.expert_combine_backward(st["dout"], st["a"], st["slot"], st["weight"], st["da"],
                                  st["dweight"])
        g.expert_route_backward(st["logits"], st["expert"], st["dweight"], st["dlogits"])
        return [st["da"], st["dweight"], st["dlogits"]]
    if op == "layernorm":
        if case["kind"] == "backward":
            g.layernorm_backward(st["dy"], st["h"], st["gain"], st["mean"], st["rstd"], st["dh"],
                                 dweight=st["dgain"], dbias=st["dbias"],
                                 residual_grad=st["residual_grad"])
            return [st["dh"], st["dgain"], st["dbias"]]
        g.layernorm(st["x"], st["gain"], bias=st["bias"], eps=EPS, residual=st["residual"],
                    h=st["h"], y=st["y"])
        return [*([] if st["h"] is None else [st["h"]]), st["y"]]
    kept = []
    if case["norm"]:
        g.layernorm(st["x"], st["gain"], bias=st["norm_bias"], eps=EPS, residual=st["residual"],
                    h=st["h"], q=st["q"], scales=st["scales"])
        kept = [st["h"]]
    else:
        g.int8_quantize(st["x"], st["q"], st["scales"])
    g.int8gemm(st["q"], st["scales"], st["w"], st["w_scales"], st["d"], bias=st["bias"])
    return [*kept, st["d"]]


# ------------------------------------------------------------------ 64 bits
def exact_softmax(l):
    """Rows without any unmasked logit have shares of 0."""
    live = (l > -math.inf).any(1)
    p = torch.zeros_like(l)
    p[live] = torch.softmax(l[live], dim=1)
    return p


def exact_route(l, top):
    """The `top` largest logits, one after the other; the first of equal ones."""
    left, chosen = l.clone(), []
    for _ in range(top):
        best = left.amax(1, keepdim=True)
        index = (left == best).to(torch.uint8).argmax(1, keepdim=True)
        chosen.append(torch.where(best > -math.inf, index, -1))
        left.scatter_(1, index, -math.inf)
    return torch.cat(chosen, 1)


def exact_layernorm(h, gain, bias):
    n = h.shape[1]
    mu = h.sum(1, keepdim=True) / n
    var = ((h - mu) ** 2).sum(1, keepdim=True) / n
    return (h - mu) / torch.sqrt(var + EPS) * gain.double() + bias.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = st["logits"].double()
        expert = exact_route(l, case["top"])
        real = expert >= 0
        w = torch.where(real, exact_softmax(l).gather(1, expert.clamp_min(0)), 0.0)
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        flat = expert.reshape(-1)
        counts = torch.bincount(flat[flat >= 0], minlength=case["experts"])
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        slot = torch.full_like(flat, -1)
        for g in range(case["experts"]):
            mine = (flat == g).nonzero()[:, 0]
            slot[mine] = offsets[g] + torch.arange(mine.shape[0], device=flat.device)
        i32 = torch.int32
        return [expert.to(i32), w, slot.view(expert.shape).to(i32), offsets.to(i32)]
    if op == "rows":
        slot, top = st["slot"].long(), case["top"]
        real = slot >= 0
        if case["kind"] == "dispatch":
            a = torch.zeros(slot.numel(), case["dim"], dtype=torch.float64, device="cuda")
            s = None
            if case["x"] == "fp8":
                s = torch.zeros(blocks(case["dim"]), slot.numel(), dtype=torch.float64, device="cuda")
            for j in range(top):
                a[slot[:, j][real[:, j]]] = st["x"].double()[real[:, j]]
                if s is not None:
                    s[:, slot[:, j][real[:, j]]] = st["x_scales"].double()[:, real[:, j]]
            return a if s is None else [a, s]
        if case["kind"] == "combine":
            out = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
            if st["residual"] is not None:
                out += st["residual"].double()
            for j in range(top):
                r = real[:, j]
                out[r] += st["weight"][r, j, None].double() * st["a"][slot[r, j]].double()
            return out
        dout = st["dout"].double()
        da = torch.zeros(slot.numel(), case["dim"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["rows"], top, dtype=torch.float64, device="cuda")
        g = torch.zeros(case["rows"], case["experts"], dtype=torch.float64, device="cuda")
        for j in range(top):
            r = real[:, j].nonzero()[:, 0]
            da[slot[r, j]] = st["weight"][r, j, None].double() * dout[r]
            dw[r, j] = torch.einsum("rd,rd->r", dout[r], st["a"][slot[r, j]].double())
            g[r, st["expert"][r, j].long()] += dw[r, j]
        p = exact_softmax(st["logits"].double())
        return [da, dw, p * g - p * (p * g).sum(1, keepdim=True)]
    if op == "layernorm":
        if case["kind"] == "forward":
            h = st["x"].double()
            if st["residual"] is not None:
                h = h + st["residual"].double()
            kept = [] if st["residual"] is None else [h]
            return [*kept, exact_layernorm(h, st["gain"], st["bias"])]
        h, dy, w = st["h"].double(), st["dy"].double(), st["gain"].double()
        n = case["dim"]
        mid = h - h.sum(1, keepdim=True) / n
        var = (mid * mid).sum(1, keepdim=True) / n + EPS
        dxh = dy * w / var.sqrt()
        dh = dxh - dxh.sum(1, keepdim=True) / n - mid * (dxh * mid).sum(1, keepdim=True) / (n * var)
        if st["residual_grad"] is not None:
            dh += st["residual_grad"].double()
        return [dh, (dy * mid / var.sqrt()).sum(0), dy.sum(0)]
    x, kept = st["x"].double(), []
    if case["norm"]:
        x = x + st["residual"].double()
        kept = [x]
        x = exact_layernorm(x, st["gain"], st["norm_bias"])
    s = torch.clamp(x.abs().amax(1, keepdim=True) / INT8_MAX, min=SCALE_MIN)
    d = (torch.round(x / s) * s) @ (st["w"].double() * st["w_scales"].double()[:, None]).t()
    return [*kept, d if st["bias"] is None else d + st["bias"].double()]


# -------------------------------------------------------------------- floors
def work(case):
    """Bytes read and written once, and operations, of one pass."""
    size = {"f32": 4, "bf16": 2, "fp8": 1, "none": 0}
    op = case["op"]
    if op == "route":
        rows, n = case["rows"], case["rows"] * case["top"]
        # logits in; expert, weight, place of each pair and the experts' first rows out
        return {"bytes": rows * case["experts"] * size[case["logits"]] + 12 * n + 4 * case["experts"],
                "flops": 4 * rows * case["experts"]}
    if op == "rows":
        rows, dim = case["rows"], case["dim"]
        n = rows * case["top"]
        live = round(n * (1.0 - case["drop"]))
        x = size[case["x"]]
        if case["kind"] == "dispatch":
            row = dim * x + (4 * blocks(dim) if case["x"] == "fp8" else 0)
            return {"bytes": (rows + live) * row + 4 * n, "flops": 0}
        if case["kind"] == "combine":
            return {"bytes": (rows + live) * dim * x + rows * dim * size[case["residual"]] + 8 * n,
                    "flops": 2 * live * dim}
        return {"bytes": (rows + 2 * live) * dim * x + 16 * n + 8 * rows * case["experts"],
                "flops": 3 * live * dim + 6 * rows * case["experts"]}
    if op == "layernorm":
        v = case["rows"] * case["dim"]
        x, r = size[case["x"]], size[case["residual"]]
        if case["kind"] == "forward":
            return {"bytes": v * (2 * x + 2 * r) + 8 * case["dim"], "flops": 8 * v}
        return {"bytes": v * (x + 2 * (r or x) + r) + 8 * case["rows"] + 12 * case["dim"],
                "flops": 14 * v}
    m, n, k = case["m"], case["n"], case["k"]
    extra = 4 * m * k + 8 * k if case["norm"] else 0     # the residual in, its sum out
    return {"bytes": 2 * m * k + extra + n * k + 4 * n * (2 if case["bias"] else 1)
            + m * n * size[case["out"]], "flops": 2.0 * m * n * k}
