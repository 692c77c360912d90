"""One mixture-of-experts layer from the normed hidden state to the next layer's input, on one GPU.

    python examples/moe_layer.py [--tokens T] [--experts E] [--topk K] [--hidden H] [--width F] [--shards R]

The router's logits choose each token's experts (``route``), the token slots are grouped by expert
(``plan``), the grouped rows go to 4-bit floating point (``quantize_fp4``) and through each shard's
slice of the experts' two projections (``expert_product``), and ``finalize_reduce_norm`` weighs, sums
and norms what comes back.  ``router_step`` is the training side: the gradient of the routing weights
(``route_backward``) as an update of the router.  Weights and inputs are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tp_reduce_residual_gb300 import beamnorm as bn  # noqa: E402
from tp_reduce_residual_gb300 import experts  # noqa: E402

ROUTING = dict(score="sigmoid", renormalize=True, scale=2.5)


class MoELayer:
    """E experts of hidden size H and width F, cut along F into R shards, weights in 4 bits."""

    def __init__(self, H, F, E, k, R, format="nvfp4", seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.k, self.R, self.E, self.format = k, R, E, format
        self.groups = dict(groups=4, top_groups=2, group_top=2) if E % 4 == 0 and E // 2 >= k else {}
        self.router = torch.randn(E, H, generator=g, device=device) / H ** 0.5
        self.balance = torch.zeros(E, device=device)
        n = F // R
        self.up, self.down = [], []
        for _ in range(R):  # gate and up projection side by side, then the down projection
            up = torch.randn(E, 2 * n, H, generator=g, device=device) / H ** 0.5
            down = torch.randn(E, H, n, generator=g, device=device) / F ** 0.5
            self.up.append(experts.quantize_fp4(up.bfloat16(), format, tensor_scale=2.0 ** -6))
            self.down.append(experts.quantize_fp4(down.bfloat16(), format, tensor_scale=2.0 ** -6))
        self.gamma_post = 1 + 0.1 * torch.randn(H, generator=g, device=device)
        self.gamma_pre = 1 + 0.1 * torch.randn(H, generator=g, device=device)

    def route(self, logits):
        return experts.route(logits, self.k, bias=self.balance, shards=self.R, **ROUTING, **self.groups)

    def __call__(self, h, residual, eps=1e-6):
        """h [T,H] BF16 -> the next layer's input [T,H] BF16; the residual is updated in place."""
        ids, w = self.route(h.float() @ self.router.T)
        plan = experts.plan(ids, self.E, shards=self.R)
        x = experts.quantize_fp4(h, self.format, rows=plan.rows, offsets=plan.offsets)
        y = torch.empty(self.R, plan.rows.numel(), h.shape[1], dtype=torch.bfloat16, device=h.device)
        for r in range(self.R):
            gate, up = experts.expert_product(x, self.up[r]).float().chunk(2, dim=-1)
            act = (torch.nn.functional.silu(gate) * up).bfloat16()
            act = experts.quantize_fp4(act, self.format, offsets=plan.offsets)
            experts.expert_product(act, self.down[r], out=y[r])
        return bn.finalize_reduce_norm(y, plan.perm, w, None, residual, self.gamma_post, self.gamma_pre, eps)

    def router_step(self, h, dw, rate=1e-3):
        """One gradient step of the router: dw [R,T,k] is the loss's gradient with respect to the
        routing weights.  Returns the gradient with respect to h."""
        logits = h.float() @ self.router.T
        ids, _ = self.route(logits)
        dlogits = experts.route_backward(logits, ids, dw, **ROUTING)
        dh = dlogits @ self.router
        self.router -= rate * (dlogits.T @ h.float())
        return dh

    def reference(self, h, residual, eps=1e-6):
        """The layer's output in 32 bits, with the 4-bit weights but activations as they are."""
        logits = h.float() @ self.router.T
        ids, w = self.route(logits)
        total = torch.zeros(h.shape, device=h.device)
        for r in range(self.R):
            up, down = experts.dequantize_fp4(self.up[r]).float(), experts.dequantize_fp4(self.down[r]).float()
            for j in range(self.k):
                e = ids[:, j].long()
                gate, lift = torch.einsum("tnh,th->tn", up[e], h.float()).chunk(2, dim=-1)
                act = torch.nn.functional.silu(gate) * lift
                total += w[r, :, j, None] * torch.einsum("thn,tn->th", down[e], act)

        def norm(v, gamma):
            return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * gamma

        return norm(residual.float() + norm(total, self.gamma_post), self.gamma_pre)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 64), ("experts", 16), ("topk", 4), ("hidden", 2048), ("width", 1024), ("shards", 2)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--format", choices=tuple(experts.FORMATS), default="nvfp4")
    a = ap.parse_args(argv)
    layer = MoELayer(a.hidden, a.width, a.experts, a.topk, a.shards, a.format)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    residual = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    want = layer.reference(h, residual)
    out = layer(h, residual.clone())
    bn.check_device_error()
    off = float((out.float() - want).norm() / want.norm())
    dw = torch.randn(a.shards, a.tokens, a.topk, generator=g, device="cuda")
    dh = layer.router_step(h, dw)
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
    begin.record()
    for _ in range(20):
        layer(h, residual)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.experts} experts, top {a.topk}, {a.shards} shards, {a.format}: output off by {off:.3f} of "
          f"32-bit activations, |dh| {float(dh.norm()):.3f}, {begin.elapsed_time(end) / 20 * 1e3:.0f} us a layer")
    return off


if __name__ == "__main__":
    main()
