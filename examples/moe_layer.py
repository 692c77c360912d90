"""One mixture-of-experts layer from the normed hidden state to the next layer's input, on one GPU.

    python examples/moe_layer.py [--tokens T] [--experts E] [--topk K] [--hidden H] [--width F] [--shards R]
                                 [--format nvfp4|mxfp4|int8|bf16] [--timed N]

The router's logits choose each token's experts (``route``), the token slots are grouped by expert
(``plan``), the grouped rows go through each shard's slice of the experts' two projections with the
gated activation between them (``swiglu``), and ``finalize_reduce_norm`` weighs, sums and norms what
comes back.  The projections' operands are 4-bit floating point (``quantize_fp4``), 8-bit integers
(``quantize_int8``; both ``expert_product``) or BF16 (``expert_linear``).  The training side:
``gradients`` of the BF16 experts, their rows and the routing weights, and ``router_step``, the
gradient of the routing weights (``route_backward``) as an update of the router.  Weights and inputs
are random.
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

FORMATS = (*experts.FORMATS, "int8", "bf16")
ROUTING = dict(score="sigmoid", renormalize=True, scale=2.5)


class MoELayer:
    """E experts of hidden size H and width F, cut along F into R shards, weights in ``format``."""

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
            self.up.append(self.weights(up.bfloat16()))
            self.down.append(self.weights(down.bfloat16()))
        self.gamma_post = 1 + 0.1 * torch.randn(H, generator=g, device=device)
        self.gamma_pre = 1 + 0.1 * torch.randn(H, generator=g, device=device)

    def weights(self, w):
        if self.format == "bf16":
            return w
        return experts.quantize_int8(w) if self.format == "int8" else experts.quantize_fp4(w, self.format, tensor_scale=2.0 ** -6)

    def values(self, w):
        """The weights' values in 32 bits."""
        if self.format == "bf16":
            return w.float()
        return experts.dequantize_int8(w, torch.float32) if self.format == "int8" else experts.dequantize_fp4(w).float()

    def project(self, x, w, plan, rows=None, out=None):
        """Grouped rows (or rows of x by index) through one projection."""
        if self.format == "bf16":
            return experts.expert_linear(x, w, plan.offsets, rows=rows, out=out)
        if isinstance(x, torch.Tensor):
            x = self.rows(x, plan, rows)
        return experts.expert_product(x, w, out=out)

    def rows(self, x, plan, rows=None):
        """Rows as the projections take them; quantised once for every shard."""
        if self.format == "bf16":
            return x
        if self.format == "int8":
            return experts.quantize_int8(x, rows=rows, offsets=plan.offsets)
        return experts.quantize_fp4(x, self.format, rows=rows, offsets=plan.offsets)

    def route(self, logits):
        return experts.route(logits, self.k, bias=self.balance, shards=self.R, **ROUTING, **self.groups)

    def __call__(self, h, residual, eps=1e-6):
        """h [T,H] BF16 -> the next layer's input [T,H] BF16; the residual is updated in place."""
        ids, w = self.route(h.float() @ self.router.T)
        plan = experts.plan(ids, self.E, shards=self.R)
        x = self.rows(h, plan, plan.rows)
        y = torch.empty(self.R, plan.rows.numel(), h.shape[1], dtype=torch.bfloat16, device=h.device)
        for r in range(self.R):
            act = experts.swiglu(self.project(x, self.up[r], plan, rows=plan.rows))
            self.project(act, self.down[r], plan, out=y[r])
        return bn.finalize_reduce_norm(y, plan.perm, w, None, residual, self.gamma_post, self.gamma_pre, eps)

    def gradients(self, h, dz):
        """Gradients of sum(dz * z), z [T,H] the weighted sum of the experts' outputs over slots and
        shards, of a BF16 layer: ``up`` and ``down`` (FP32, a shard each), ``h`` [T,H] FP32 through the
        experts, and ``w`` [R,T,k] of the routing weights (what ``router_step`` takes)."""
        ids, w = self.route(h.float() @ self.router.T)
        plan = experts.plan(ids, self.E, shards=self.R)
        T, k = ids.shape
        place = plan.perm[0].view(-1).long()
        dz_rows = dz.float()[plan.rows.long()]
        grads = dict(up=[], down=[], w=torch.empty_like(w))
        dx = torch.empty(self.R, T * k, h.shape[1], dtype=torch.bfloat16, device=h.device)
        for r in range(self.R):
            hidden = experts.expert_linear(h, self.up[r], plan.offsets, rows=plan.rows)
            act = experts.swiglu(hidden)
            y = experts.expert_linear(act, self.down[r], plan.offsets)
            grads["w"][r] = (y.float() * dz_rows).sum(-1)[place].view(T, k)
            weight = torch.empty(T * k, device=h.device)
            weight[place] = w[r].view(-1)
            dy = (weight[:, None] * dz_rows).bfloat16()
            grads["down"].append(experts.expert_linear_dw(dy, act, plan.offsets, dtype=torch.float32))
            dhidden = experts.swiglu_backward(hidden, experts.expert_linear_dx(dy, self.down[r], plan.offsets))
            grads["up"].append(experts.expert_linear_dw(dhidden, h, plan.offsets, rows=plan.rows, dtype=torch.float32))
            experts.expert_linear_dx(dhidden, self.up[r], plan.offsets, dx=dx[r])
        # a token's gradient is the sum over its slots and the shards
        grads["h"] = bn.finalize_reduce_only(dx, plan.perm, torch.ones_like(w), None)
        return grads

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
        """The layer's output in 32 bits, with the weights' values but activations as they are."""
        ids, w = self.route(h.float() @ self.router.T)
        total = self.mixture(h.float(), [self.values(u) for u in self.up], [self.values(d) for d in self.down], ids, w)

        def norm(v, gamma):
            return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * gamma

        return norm(residual.float() + norm(total, self.gamma_post), self.gamma_pre)

    def mixture(self, h, up, down, ids, w):
        """The weighted sum of the experts' outputs over slots and shards, in elementary operations."""
        total = torch.zeros_like(h)
        for r in range(self.R):
            for j in range(self.k):
                e = ids[:, j].long()
                gate, lift = torch.einsum("tnh,th->tn", up[r][e], h).chunk(2, dim=-1)
                act = torch.nn.functional.silu(gate) * lift
                total = total + w[r, :, j, None] * torch.einsum("thn,tn->th", down[r][e], act)
        return total


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 64), ("experts", 16), ("topk", 4), ("hidden", 2048), ("width", 1024), ("shards", 2)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--format", choices=FORMATS, default="nvfp4")
    ap.add_argument("--timed", type=int, default=20, help="layers to time; 0: none")
    a = ap.parse_args(argv)
    layer = MoELayer(a.hidden, a.width, a.experts, a.topk, a.shards, a.format)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    residual = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    want = layer.reference(h, residual)
    out = layer(h, residual.clone())
    bn.check_device_error()
    off = float((out.float() - want).norm() / want.norm())
    if a.format == "bf16":
        dw = layer.gradients(h, torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16())["w"]
    else:
        dw = torch.randn(a.shards, a.tokens, a.topk, generator=g, device="cuda")
    dh = layer.router_step(h, dw)
    line = (f"{a.tokens} tokens, {a.experts} experts, top {a.topk}, {a.shards} shards, {a.format}: output off by {off:.3f} of "
            f"32-bit activations, |dh| {float(dh.norm()):.3f}")
    if a.timed > 0:
        begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
        begin.record()
        for _ in range(a.timed):
            layer(h, residual)
        end.record()
        torch.cuda.synchronize()
        line += f", {begin.elapsed_time(end) / a.timed * 1e3:.0f} us a layer"
    print(line)
    return off


if __name__ == "__main__":
    main()
