"""A layer of experts, served in fp8 and trained in bf16, on the library's operators.

    python examples/expert_layer.py

Serving (``forward``): h = x + residual and its norm in fp8 (``rmsnorm``), router logits
(``bf16gemm``), each token's experts and their weights (``expert_route``), the rows gathered expert
by expert (``expert_sort``, ``expert_dispatch``), both of the experts' products in fp8
(``fp8gemm_grouped``, weights quantised once with ``fp8_quantize``, the hidden values quantised in
between), the rows added up again (``expert_combine``) and an output projection (``fp8gemm``).

Training (``gradients``): the experts' products in bf16 (``bf16gemm_grouped``), their gradients
with respect to rows and weights (the transposed product and ``bf16gemm_grouped_wgrad``), those of
the weights of a token's experts and of the router (``expert_combine_backward``,
``expert_route_backward``) and the norm's (``rmsnorm_backward``).

No call waits for the GPU: which rows an expert has is only ever known there.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_12_gb300 as g  # noqa: E402


def blocks(n):
    return -(-n // 128)


def empty_fp8(*shape):
    """fp8 rows with a pitch of whole 16-byte pieces, which TMA can read without a copy."""
    pitch = -(-shape[-1] // 16) * 16
    return torch.empty(*shape[:-1], pitch, dtype=torch.float8_e4m3fn, device="cuda")[..., :shape[-1]]


def quantized_weights(w):
    """Weights (G, K, N) as the fp8 products want them: (G, N, K) with a scale per 128 x 128."""
    G, K, N = w.shape
    q, s = empty_fp8(G, N, K), torch.empty(G, blocks(K), blocks(N), device="cuda")
    for i in range(G):
        g.fp8_quantize(w[i], q[i], s[i], block="tiles", transpose=True)
    return q, s


class ExpertLayer:
    def __init__(self, dim, hidden, experts, top=2, eps=1e-6, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def draw(*shape, fan_in):
            w = torch.randn(*shape, generator=gen, device="cuda") * fan_in ** -0.5
            return w.to(torch.bfloat16)

        self.dim, self.hidden, self.experts, self.top, self.eps = dim, hidden, experts, top, eps
        self.norm = torch.ones(dim, device="cuda")
        self.router = draw(dim, experts, fan_in=dim)
        self.up = draw(experts, dim, hidden, fan_in=dim)
        self.down = draw(experts, hidden, dim, fan_in=hidden)
        self.out = draw(dim, dim, fan_in=dim)
        self.up_q, self.down_q = quantized_weights(self.up), quantized_weights(self.down)
        out_q, out_s = quantized_weights(self.out[None])
        self.out_q = out_q[0], out_s[0]

    def route(self, y):
        """y (rows, dim) -> the router's logits, each token's experts and their weights (rows, top), the
        rows of its pairs among the gathered ones (rows, top) and the experts' offsets."""
        rows = y.shape[0]
        logits = torch.empty(rows, self.experts, device="cuda")
        g.bf16gemm(y, self.router, logits)
        expert = torch.empty(rows, self.top, dtype=torch.int32, device="cuda")
        slot, weight = torch.empty_like(expert), torch.empty(rows, self.top, device="cuda")
        offsets = torch.empty(self.experts + 1, dtype=torch.int32, device="cuda")
        g.expert_route(logits, expert, weight)
        g.expert_sort(expert, slot, offsets)
        return logits, expert, weight, slot, offsets

    def forward(self, x, residual):
        """x, residual (rows, dim) bf16 -> (the layer's output, the new residual h)."""
        rows = x.shape[0]
        n = rows * self.top
        h, y = torch.empty_like(residual), torch.empty_like(x)
        q, s = empty_fp8(rows, self.dim), torch.empty(blocks(self.dim), rows, device="cuda")
        g.rmsnorm(x, self.norm, eps=self.eps, residual=residual, h=h, y=y, q=q, scales=s)
        _, _, weight, slot, offsets = self.route(y)
        a, a_s = empty_fp8(n, self.dim), torch.empty(blocks(self.dim), n, device="cuda")
        g.expert_dispatch(q, slot, a, x_scales=s, a_scales=a_s)
        hid = torch.empty(n, self.hidden, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm_grouped(a, a_s, *self.up_q, offsets, hid)
        hid = torch.nn.functional.gelu(hid)
        hq, hs = empty_fp8(n, self.hidden), torch.empty(blocks(self.hidden), n, device="cuda")
        g.fp8_quantize(hid, hq, hs)
        back = torch.empty(n, self.dim, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm_grouped(hq, hs, *self.down_q, offsets, back)
        both = torch.empty(rows, self.dim, device="cuda")
        g.expert_combine(back, slot, both, weight)
        g.fp8_quantize(both, q, s)
        out = torch.empty(rows, self.dim, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm(q, s, *self.out_q, out)
        return out, h

    def gradients(self, x, residual, grad):
        """Loss sum(grad * experts(norm(x + residual))): the experts' output and the gradients of h,
        the norm's weight, the router and both of the experts' weights (which experts a token has is
        fixed, how much each counts is not)."""
        rows = x.shape[0]
        n = rows * self.top
        h, y, rstd = torch.empty_like(residual), torch.empty_like(x), torch.empty(rows, device="cuda")
        g.rmsnorm(x, self.norm, eps=self.eps, residual=residual, h=h, y=y, rstd=rstd)
        logits, expert, weight, slot, offsets = self.route(y)
        a = torch.zeros(n, self.dim, dtype=torch.bfloat16, device="cuda")
        g.expert_dispatch(y, slot, a)
        pre = torch.empty(n, self.hidden, dtype=torch.bfloat16, device="cuda")
        g.bf16gemm_grouped(a, self.up, offsets, pre)
        with torch.enable_grad():
            leaf = pre.float().requires_grad_()
            act = torch.nn.functional.gelu(leaf)
        mid = act.detach().to(torch.bfloat16)
        back = torch.empty(n, self.dim, dtype=torch.bfloat16, device="cuda")
        g.bf16gemm_grouped(mid, self.down, offsets, back)
        out = torch.empty(rows, self.dim, device="cuda")
        g.expert_combine(back, slot, out, weight)

        d_back, d_weight = torch.empty_like(back), torch.empty_like(weight)
        g.expert_combine_backward(grad, back, slot, weight, da=d_back, dweight=d_weight)
        d_down = torch.empty(self.down.shape, device="cuda")
        g.bf16gemm_grouped_wgrad(mid, d_back, offsets, d_down)
        d_mid = torch.empty_like(mid)
        g.bf16gemm_grouped(d_back, self.down, offsets, d_mid, transpose_b=True)
        act.backward(d_mid.float())
        d_pre = leaf.grad.to(torch.bfloat16)
        d_up = torch.empty(self.up.shape, device="cuda")
        g.bf16gemm_grouped_wgrad(a, d_pre, offsets, d_up)
        d_a = torch.empty_like(a)
        g.bf16gemm_grouped(d_pre, self.up, offsets, d_a, transpose_b=True)
        d_y = torch.empty(rows, self.dim, device="cuda")
        g.expert_combine(d_a, slot, d_y)
        # the router: one group of all the rows
        d_logits = torch.empty(rows, self.experts, dtype=torch.bfloat16, device="cuda")
        g.expert_route_backward(logits, expert, d_weight, d_logits)
        all_rows = torch.arange(2, dtype=torch.int32, device="cuda") * rows
        d_router = torch.empty(1, self.dim, self.experts, device="cuda")
        g.bf16gemm_grouped_wgrad(y, d_logits, all_rows, d_router)
        g.bf16gemm_grouped(d_logits, self.router[None], all_rows, d_y, beta=1.0, transpose_b=True)
        d_h, d_norm = torch.empty_like(h), torch.empty_like(self.norm)
        g.rmsnorm_backward(d_y, h, self.norm, rstd, d_h, d_norm)
        return out, {"h": d_h, "norm": d_norm, "router": d_router[0], "up": d_up, "down": d_down}

    def plain(self, x, residual, project=True):
        """The same layer in fp32 torch operations on the bf16 weights (differentiable)."""
        h = x.float() + residual.float()
        y = h * (h.square().mean(-1, keepdim=True) + self.eps).rsqrt() * self.norm
        expert = self.route(y.detach().to(torch.bfloat16))[1].long()
        weight = (y @ self.router.float()).softmax(-1).gather(1, expert)
        a, expert = y.repeat_interleave(self.top, 0), expert.reshape(-1)
        mid = torch.nn.functional.gelu(torch.einsum("nk,nkf->nf", a, self.up.float()[expert]))
        back = torch.einsum("nf,nfk->nk", mid, self.down.float()[expert])
        out = (back.unflatten(0, weight.shape) * weight[..., None]).sum(1)
        return out @ self.out.float() if project else out


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(rows=96, dim=512, hidden=384, experts=8):
    layer = ExpertLayer(dim, hidden, experts)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, residual, grad = (torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
                         for _ in range(3))
    with torch.no_grad():
        out, _ = layer.forward(x, residual)
        served = relative(out, layer.plain(x, residual))
        got, grads = layer.gradients(x, residual, grad)
    up, down, norm, router = layer.up, layer.down, layer.norm, layer.router
    h = (x.float() + residual.float()).requires_grad_()
    layer.up, layer.down = (w.float().requires_grad_() for w in (up, down))
    layer.norm, layer.router = norm.clone().requires_grad_(), router.clone().requires_grad_()
    want = layer.plain(h, torch.zeros_like(h), project=False)
    (want * grad.float()).sum().backward()
    errors = {"output": relative(got, want.detach()), "h": relative(grads["h"], h.grad),
              "norm": relative(grads["norm"], layer.norm.grad),
              "router": relative(grads["router"], layer.router.grad),
              "up": relative(grads["up"], layer.up.grad), "down": relative(grads["down"], layer.down.grad)}
    layer.up, layer.down, layer.norm, layer.router = up, down, norm, router
    status = g.gemm_check_device_error(torch.cuda.current_stream().cuda_stream)
    if status != 0:
        raise g.GemmError(status, "expert_layer")
    print("fp8 output, relative error %.4f" % served)
    print("bf16 training step, relative errors:", {k: round(v, 5) for k, v in errors.items()})
    return served, errors


if __name__ == "__main__":
    g.load_library(build_if_missing=True)
    main()
