"""GPU tests of drafted tokens that have no place, since their sequence has fewer cached tokens than new ones: they see nothing,
whatever their masks name, and the others see what theirs name of those that have one (extend_case.py has the bounds)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, WEIGHT, ExtendCase

pytestmark = pytest.mark.gpu


# (few rows a head: an item a block, and the line; tiles)
@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,other", [(8, 2, (20, 3)), (8, 2, (9000, 3)), (64, 8, (30, 60))])
@pytest.mark.parametrize("window", [0, 7])
def test_tokens_without_a_place(Hq, heads, other, window, fmt):
    m, n = 40, 25
    c = ExtendCase([(0, m), other], Hq, heads, 64, 32, fmt, seed=3)
    masks = c.trees(1, "any")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(masks, window=window, sinks=2 * (window > 0), lens=[n, c.lens[1]], dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    none = m - n
    assert (out[:none] == 0).all() and (lse[:none] == -torch.inf).all()
    got, gl, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), ref.bf16_value(c.q_bits)
    for i in range(none, m):
        see = c.kin[0][i][none:]  # new token j lies at place j - none
        for h in range(0, Hq, 3):
            g = h // (Hq // heads)
            want, wl, ab, S = ref.attn(q[i, h], c.k[:n, g][see], c.v[:n, g][see], float(np.float32(64 ** -0.5)))
            if wl == -np.inf:
                assert (got[i, h] == 0).all() and gl[i, h] == -np.inf
                continue
            e = (64 + 7) * 2.0 ** -23 * S + 2.0 ** -21
            d = ab * (WEIGHT + 2 * e + 2 * (n + 64) * 2.0 ** -24)
            assert (np.abs(got[i, h] - want) <= d + ref.bf16_half_step(np.abs(want) + d)).all(), (i, h)
            assert abs(gl[i, h] - wl) <= e + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(wl), (i, h)
    c.check(out, lse, tree=True, window=window, sinks=2 * (window > 0), rows=lambda b, i: b == 1 and i % 7 == 0)
