"""A layer of experts, served in fp8 and trained in bf16, on the library's operators.

    python examples/expert_layer.py

Serving (``forward``): h = x + residual and its norm in fp8 (``rmsnorm``), router logits
(``bf16gemm``), the rows gathered expert by expert, both of the experts' products in fp8
(``fp8gemm_grouped``, weights quantised once with ``fp8_quantize``, the hidden values quantised in
between), and an output projection of the combined rows (``fp8gemm``).

Training (``gradients``): the experts' products in bf16 (``bf16gemm_grouped``), their gradients
with respect to rows and weights (the transposed product and ``bf16gemm_grouped_wgrad``) and the
norm's (``rmsnorm_backward``).

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
        """(place of each gathered row's token, its weight, the experts' offsets)."""
        rows = y.shape[0]
        logits = torch.empty(rows, self.experts, device="cuda")
        g.bf16gemm(y, self.router, logits)
        weight, expert = logits.softmax(-1).topk(self.top, dim=-1)
        expert, order = expert.reshape(-1).sort(stable=True)
        counts = (expert[:, None] == torch.arange(self.experts, device="cuda")).sum(0)
        offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        return order // self.top, weight.reshape(-1)[order], offsets

    def combine(self, rows, token, weight, n):
        return torch.zeros(n, self.dim, device="cuda").index_add_(0, token, rows.float() * weight[:, None])

    def forward(self, x, residual):
        """x, residual (rows, dim) bf16 -> (the layer's output, the new residual h)."""
        rows = x.shape[0]
        h, y = torch.empty_like(residual), torch.empty_like(x)
        q, s = empty_fp8(rows, self.dim), torch.empty(blocks(self.dim), rows, device="cuda")
        g.rmsnorm(x, self.norm, eps=self.eps, residual=residual, h=h, y=y, q=q, scales=s)
        token, weight, offsets = self.route(y)
        n = token.shape[0]
        a = empty_fp8(n, self.dim)
        # (rows of fp8 are gathered as bytes)
        a.view(torch.uint8).copy_(q.view(torch.uint8)[token])
        hid = torch.empty(n, self.hidden, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm_grouped(a, s[:, token].contiguous(), *self.up_q, offsets, hid)
        hid = torch.nn.functional.gelu(hid)
        hq, hs = empty_fp8(n, self.hidden), torch.empty(blocks(self.hidden), n, device="cuda")
        g.fp8_quantize(hid, hq, hs)
        back = torch.empty(n, self.dim, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm_grouped(hq, hs, *self.down_q, offsets, back)
        both = self.combine(back, token, weight, rows)
        g.fp8_quantize(both, q, s)
        out = torch.empty(rows, self.dim, dtype=torch.bfloat16, device="cuda")
        g.fp8gemm(q, s, *self.out_q, out)
        return out, h

    def gradients(self, x, residual, grad):
        """Loss sum(grad * experts(norm(x + residual))) for a fixed routing: the experts' output
        and the gradients of h, the norm's weight, and both weights."""
        rows = x.shape[0]
        h, y, rstd = torch.empty_like(residual), torch.empty_like(x), torch.empty(rows, device="cuda")
        g.rmsnorm(x, self.norm, eps=self.eps, residual=residual, h=h, y=y, rstd=rstd)
        token, weight, offsets = self.route(y)
        n = token.shape[0]
        a = y[token]
        pre = torch.empty(n, self.hidden, dtype=torch.bfloat16, device="cuda")
        g.bf16gemm_grouped(a, self.up, offsets, pre)
        with torch.enable_grad():
            leaf = pre.float().requires_grad_()
            act = torch.nn.functional.gelu(leaf)
        mid = act.detach().to(torch.bfloat16)
        back = torch.empty(n, self.dim, dtype=torch.bfloat16, device="cuda")
        g.bf16gemm_grouped(mid, self.down, offsets, back)
        out = self.combine(back, token, weight, rows)

        d_back = (grad.float()[token] * weight[:, None]).to(torch.bfloat16)
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
        d_y = torch.zeros(rows, self.dim, device="cuda").index_add_(0, token, d_a.float())
        d_h, d_norm = torch.empty_like(h), torch.empty_like(self.norm)
        g.rmsnorm_backward(d_y, h, self.norm, rstd, d_h, d_norm)
        return out, {"h": d_h, "norm": d_norm, "up": d_up, "down": d_down}

    def plain(self, x, residual, project=True):
        """The same layer in fp32 torch operations on the bf16 weights (differentiable)."""
        h = x.float() + residual.float()
        y = h * (h.square().mean(-1, keepdim=True) + self.eps).rsqrt() * self.norm
        token, weight, offsets = self.route(y.detach().to(torch.bfloat16))
        expert = torch.bucketize(torch.arange(token.shape[0], device="cuda"), offsets[1:], right=True)
        a = y[token]
        mid = torch.nn.functional.gelu(torch.einsum("nk,nkf->nf", a, self.up.float()[expert]))
        back = torch.einsum("nf,nfk->nk", mid, self.down.float()[expert])
        out = torch.zeros_like(y).index_add(0, token, back * weight[:, None])
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
    up, down, norm = layer.up, layer.down, layer.norm
    h = (x.float() + residual.float()).requires_grad_()
    layer.up, layer.down = (w.float().requires_grad_() for w in (up, down))
    layer.norm = norm.clone().requires_grad_()
    want = layer.plain(h, torch.zeros_like(h), project=False)
    (want * grad.float()).sum().backward()
    errors = {"output": relative(got, want.detach()), "h": relative(grads["h"], h.grad),
              "norm": relative(grads["norm"], layer.norm.grad),
              "up": relative(grads["up"], layer.up.grad), "down": relative(grads["down"], layer.down.grad)}
    layer.up, layer.down, layer.norm = up, down, norm
    status = g.gemm_check_device_error(torch.cuda.current_stream().cuda_stream)
    if status != 0:
        raise g.GemmError(status, "expert_layer")
    print("fp8 output, relative error %.4f" % served)
    print("bf16 training step, relative errors:", {k: round(v, 5) for k, v in errors.items()})
    return served, errors


if __name__ == "__main__":
    g.load_library(build_if_missing=True)
    main()
