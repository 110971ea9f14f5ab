"""A mixture-of-experts layer over a bucket that the Allgather rebuilt: output
and every gradient against the whole layer differentiated in 64 bits."""
import pytest
import torch

from lossless_exponent_reuse_gb300 import ciera, experts, moe_layer, workloads
from lossless_exponent_reuse_gb300.allgather import SimulatedAllgather

pytestmark = pytest.mark.gpu


def reference(layer, x, residual, chosen, slots_used):
    """The layer in 64 bits for the experts that the router chose, with leaves
    that take gradients."""
    p = {n: getattr(layer, n).double().detach().requires_grad_()
         for n in ("router", "norm", "gate_up", "down")}
    xd = x.double().requires_grad_()
    h = xd + residual.double()
    y = h * ((h * h).mean(1, keepdim=True) + layer.eps) ** -0.5 * p["norm"]
    w = torch.softmax(y @ p["router"].T, 1)
    out = torch.zeros_like(y)
    for e in range(layer.n_experts):
        on = (chosen == e) & slots_used
        t = on.any(1).nonzero()[:, 0]
        if t.numel() == 0:
            continue
        gate, up = (y[t] @ p["gate_up"][e].T).chunk(2, 1)
        rows = (gate / (1 + torch.exp(-gate)) * up) @ p["down"][e].T
        out = out.index_add(0, t, rows * w[t, e][:, None])
    return out, h, xd, p


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("E,dim,ff,k,T", [(8, 256, 128, 2, 200), (16, 136, 72, 4, 33),
                                          (4, 64, 40, 1, 1), (12, 512, 256, 3, 1500)])
def test_layer_over_a_rebuilt_bucket(E, dim, ff, k, T):
    wl = moe_layer.layer_workload(E, dim, ff, ranks=4, block=256, name=f"layer{E}")
    ag = SimulatedAllgather(wl.numel, wl.block, wl.ranks)
    for w in workloads.sequence(wl, 2):
        rebuilt = ag.step(w.cuda())
    assert ag.status() == ciera.OK
    assert torch.equal(rebuilt[:wl.numel].view(torch.int16), w.cuda().view(torch.int16))
    layer = moe_layer.MoELayer(rebuilt[:wl.numel], wl, k)
    gradient = torch.full((wl.numel,), float("nan"), dtype=torch.bfloat16, device="cuda")
    grads = moe_layer.MoELayer(gradient, wl, k)
    g = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda s: (torch.randn(T, dim, generator=g, device="cuda") * s).to(torch.bfloat16)
    x, residual, dy, dh = normal(1.0), normal(2.0), normal(1.0), normal(1.0)
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    mask[0] = True
    y, h, kept = layer.forward(x, residual, token_mask=mask)
    dx = layer.backward(dy, kept, grads, dh=dh)
    assert experts.status() == ciera.OK
    assert torch.isfinite(gradient).all()

    want, wh, xd, p = reference(layer, x, residual, kept.routing.experts,
                                kept.routing.slots >= 0)
    ((want * dy.double()).sum() + (wh * dh.double()).sum()).backward()
    # each quantity passes at most ten roundings to bf16, 2^-9 on average each;
    # they add up as squares, with as much again for those that the router's
    # logits carry into the weights
    tol = 20 ** 0.5 * 2.0 ** -8
    assert off(y, want.detach()) < tol and off(h, wh.detach()) < 2.0 ** -8
    assert off(dx, xd.grad) < tol
    for name in ("norm", "gate_up", "down"):
        assert off(getattr(grads, name), p[name].grad) < tol, name
    # the router's gradient is a difference of softmax terms: judged by their size
    assert off(grads.router, p["router"].grad) < 4 * tol

    layer.quantize()
    served, _ = layer.serve(x[mask], residual[mask])
    again, _, _ = layer.forward(x[mask], residual[mask])
    # three roundings to e4m3 (2^-5 on average), and tokens whose last choice
    # flips between nearly equal experts
    assert off(served, again.double()) < 0.25


def test_example_runs(capsys):
    moe_layer.main()
    out = capsys.readouterr().out
    assert out.count("ok") == 2 and "8-bit serving step" in out
