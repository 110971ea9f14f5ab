"""One mixture-of-experts layer over a rebuilt bucket: forward, gradients into a
bucket of the same layout, and a serving form over 8-bit weights.

The layer of sharded MoE training whose weights the exponent-reuse Allgather
delivers (``SimulatedAllgather.step``), run on the operators of ``experts``
without copying a weight: norm with the residual, router, experts, combination.
The router's own small products are plain matrix products (torch).

    python -m lossless_exponent_reuse_gb300.moe_layer

runs two training steps of a cut OLMoE layer, its weights rebuilt by an
Allgather before each, and one serving step, and prints what they cost.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import experts, workloads


class Kept(NamedTuple):
    """What the gradient needs of a forward pass."""
    norm: experts.Norm
    logits: torch.Tensor
    routing: experts.Routing
    pre: torch.Tensor
    h: torch.Tensor
    rows: torch.Tensor


class MoELayer:
    """Views of a flat bucket (bf16 or uint16 bits) with the tensors of
    ``workload`` in order: ``router`` [experts, dim], ``post_attn_norm`` [dim],
    and each expert's gate, up and down."""

    def __init__(self, bucket: torch.Tensor, workload: workloads.Workload, topk: int,
                 eps: float = 1e-6):
        at = {name: (off, n) for name, off, n in workloads.layer_offsets(workload)}
        shape = {t.name: t.shape for t in workload.tensors}
        self.n_experts, self.dim = shape["router"]
        self.ff = shape["expert0.gate"][0]
        self.topk, self.eps = topk, eps
        flat = bucket.view(torch.bfloat16)
        one = lambda name: flat[at[name][0]:at[name][0] + at[name][1]].view(shape[name])
        self.router, self.norm = one("router"), one("post_attn_norm")
        self.gate_up, self.down = experts.bucket_views(flat, self.n_experts, self.dim, self.ff,
                                                       at["expert0.gate"][0])
        self.quantized = None

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                token_mask: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor, Kept]:
        """(y, h, kept): the layer's output, the next residual x + residual, and
        what ``backward`` needs."""
        norm = experts.rmsnorm(x, self.norm, residual=residual, eps=self.eps)
        logits = norm.y @ self.router.T
        r = experts.route(logits, self.topk, token_mask=token_mask)
        h, pre = experts.mm_gated(norm.y, self.gate_up, r.offsets, tokens=r.tokens, keep=True)
        rows = experts.mm(h, self.down, r.offsets)
        y = experts.combine(rows, r.slots, r.weights)
        return y, norm.h, Kept(norm, logits, r, pre, h, rows)

    def backward(self, dy: torch.Tensor, kept: Kept, grads: "MoELayer",
                 dh: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The gradient of x (and of the residual); the weights' gradients are
        written to ``grads``, a layer over a gradient bucket.  ``dh`` is the
        gradient that reaches the next residual."""
        norm, r = kept.norm, kept.routing
        drows, dweights = experts.combine_backward(dy, kept.rows, r.slots, r.weights, r.offsets)
        experts.mm_dw(drows, kept.h, r.offsets, out=grads.down)
        dpre = experts.mm_dx(drows, self.down, r.offsets, gated=kept.pre)
        experts.mm_dw(dpre, norm.y, r.offsets, tokens=r.tokens, out=grads.gate_up)
        dnormed = experts.combine(experts.mm_dx(dpre, self.gate_up, r.offsets), r.slots)
        dlogits = experts.route_backward(dweights, r.weights, r.experts, kept.logits)
        torch.mm(dlogits.T, norm.y, out=grads.router)
        dnormed.addmm_(dlogits, self.router)
        dx, dweight = experts.rmsnorm_backward(dnormed, norm.h, norm.rstd, self.norm, dh=dh)
        grads.norm.copy_(dweight)
        return dx

    def quantize(self) -> None:
        """Lays out the experts' weights in 8 bits, once for many ``serve`` calls."""
        self.quantized = (*experts.quantize_rows(self.gate_up.contiguous()),
                          *experts.quantize_rows(self.down.contiguous()))

    def serve(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor]:
        """(y, h) through the 8-bit weights of ``quantize``."""
        gate_up, gate_up_scale, down, down_scale = self.quantized
        norm = experts.rmsnorm(x, self.norm, residual=residual, eps=self.eps, quantize=True)
        logits = (norm.y.to(torch.bfloat16) @ self.router.T).float() * norm.scale[:, None]
        r = experts.route(logits, self.topk)
        h = experts.mm_gated(norm.y, gate_up, r.offsets, tokens=r.tokens, x_scale=norm.scale,
                             w_scale=gate_up_scale)
        h8, h_scale = experts.quantize_rows(h)
        rows = experts.mm(h8, down, r.offsets, x_scale=h_scale, w_scale=down_scale)
        return experts.combine(rows, r.slots, r.weights), norm.h


def layer_workload(n_experts: int, dim: int, ff: int, ranks: int, block: int,
                   name: str = "moe_layer") -> workloads.Workload:
    """A layer's router, norm and experts as one bucket."""
    tensors = [workloads.Tensor("router", (n_experts, dim)),
               workloads.Tensor("post_attn_norm", (dim,), mean=1.0, sigma=0.01)]
    for e in range(n_experts):
        tensors += [workloads.Tensor(f"expert{e}.gate", (ff, dim)),
                    workloads.Tensor(f"expert{e}.up", (ff, dim)),
                    workloads.Tensor(f"expert{e}.down", (dim, ff))]
    return workloads.Workload(name, tuple(tensors), 1, ranks, block, 4, (1e-5,))


def main() -> None:
    from .allgather import SimulatedAllgather
    wl = layer_workload(16, 2048, 1024, ranks=16, block=4096)
    tokens, topk = 2048, 8
    ag = SimulatedAllgather(wl.numel, wl.block, wl.ranks)
    gradient = torch.zeros(wl.numel, dtype=torch.bfloat16, device="cuda")
    grads = MoELayer(gradient, wl, topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda scale: (torch.randn(tokens, 2048, generator=g, device="cuda")
                            * scale).to(torch.bfloat16)
    x, residual, dy = normal(1.0), normal(1.0), normal(0.01)
    mark = lambda: torch.cuda.Event(enable_timing=True)
    for step, w in enumerate(workloads.sequence(wl, 2, device="cuda")):
        a, b, c, d = mark(), mark(), mark(), mark()
        a.record()
        layer = MoELayer(ag.step(w)[:wl.numel], wl, topk)
        b.record()
        y, h, kept = layer.forward(x, residual)
        c.record()
        layer.backward(dy, kept, grads, dh=dy)
        d.record()
        torch.cuda.synchronize()
        ok = ag.status() == 0 and experts.status() == 0
        print(f"step {step}: rebuilt {2 * wl.numel / 1e6:.0f} MB in {a.elapsed_time(b):.3f} ms, "
              f"forward {b.elapsed_time(c):.3f} ms, gradients {c.elapsed_time(d):.3f} ms, "
              f"{'ok' if ok else 'FAILED'}")
    layer.quantize()
    served, _ = layer.serve(x, residual)
    off = (served.float() - y.float()).norm() / y.float().norm()
    print(f"8-bit serving step: {float(off):.3f} off the bf16 one")


if __name__ == "__main__":
    main()
