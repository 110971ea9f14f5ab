"""Forms of the grouped products that a call takes by its sizes and layout
alone, each against the formula in 64 bits."""
import pytest
import torch

import moe_reference as ref
from lossless_exponent_reuse_gb300 import ciera, experts
from test_moe_experts_gpu import GROUPS, make, sums, weights
from test_moe_rows_gpu import rand, strided

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gated_slack(a, e):
    """Of silu(gate) * up where the products `a` are within e: |silu'| <= 1.1, exp
    and the division within 16 ulp."""
    g, u = a.chunk(2, 1)
    eg, eu = e.chunk(2, 1)
    return (1.1 * eg * (u.abs() + eu) + ref.silu(g).abs() * eu
            + ref.gated(a).abs() * 16 * ref.U_F32)


@pytest.mark.parametrize("kind", ["plain", "wide", "odd"])
@pytest.mark.parametrize("groups,unused,K,N", GROUPS)
def test_rows_gathered_inside_products_of_any_size(groups, unused, K, N, kind, monkeypatch):
    """Rows picked by the product itself, however many an expert has, with
    indexes outside x among them."""
    monkeypatch.setattr(experts, "_GATHER_ROWS", 1 << 40)
    T = 50
    offsets, R, tokens = make(groups, unused, T=T)
    if R > 2:
        tokens[R // 2] = T
        tokens[R // 3] = -5
    x = rand(T, K, seed=2)
    w = weights(len(groups), 2 * N, K, kind, scale=1.0 / K ** 0.5)
    rows = ref.gather(x, tokens, R)
    a, size = ref.product(rows, w, offsets)
    e = sums(size, K)
    h, pre = experts.mm_gated(strided(x, kind), w, offsets, tokens=tokens, keep=True)
    ref.within(pre, a, e, "pre")
    ref.within(h, ref.gated(a), gated_slack(a, e), "h")
    ref.within(experts.mm(strided(x, kind), w, offsets, tokens=tokens), a, e, "y")
    assert (h[int(offsets[-1]):] == 0).all() and (pre[int(offsets[-1]):] == 0).all()

    x8, xs = experts.quantize_rows(x)
    w8, ws = experts.quantize_rows(w.contiguous())
    a, size = ref.product(ref.gather(x8.double() * xs.double()[:, None], tokens, R),
                          w8.double() * ws.double()[..., None], offsets)
    e = sums(size, K + 4)
    h, pre = experts.mm_gated(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws, keep=True)
    ref.within(pre, a, e, "pre, 8 bits")
    ref.within(h, ref.gated(a), gated_slack(a, e), "h, 8 bits")
    y = experts.mm(x8, w8, offsets, tokens=tokens, x_scale=xs, w_scale=ws)
    ref.within(y, a, e, "y, 8 bits")
    assert experts.status() == ciera.OK
