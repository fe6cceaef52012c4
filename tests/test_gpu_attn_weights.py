"""GPU tests of the softmax weights' precision in k3moe_attn_decode over a bf16 cache: a
weight enters the product with V as two bf16 numbers, the rounded weight and what the
rounding left.  Each rounding leaves at most 2^-8 of what it rounds, so that 2^-16 of a weight is
lost; with the other terms of the bound as in test_gpu_attn_decode.py (ab = sum p |V| / l, S the largest scale *
sum |q K|), e = (D + 7) 2^-23 S + 2^-21 of a weight, fp32 sums of n terms 2 (n + 64) 2^-24:
|out - ref| <= d + half a bf16 step at |out| + d, d = ab (2^-16 + 2 e + 2 (n + 64) 2^-24)."""
import numpy as np
import pytest

import decoder_ref as ref
from test_gpu_attn_decode import BF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,Hq,heads,dim,page,window", [
    ([300, 17, 0, 1], 8, 2, 128, 64, 0), ([900, 40], 16, 1, 64, 16, 0), ([700], 12, 1, 256, 32, 0),
    ([3000], 4, 1, 128, 64, 1700), ([30000], 9, 1, 128, 64, 0), ([1500] * 90, 16, 2, 64, 32, 0), ([60] * 200, 16, 4, 128, 16, 0)])
def test_weights_keep_sixteen_bits(lens, Hq, heads, dim, page, window):
    c = Case(lens, Hq, heads, dim, page, BF, seed=dim + Hq)
    out, _ = c.run(window=window)
    got, q, scale, at = out.double().cpu().numpy(), ref.bf16_value(c.q_bits), float(np.float32(dim ** -0.5)), 0
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        for h in range(Hq):
            g = h // (Hq // heads)
            want, _, ab, S = ref.attn(q[b, h], c.k[at + lo:at + n, g], c.v[at + lo:at + n, g], scale)
            m = n - lo
            d = ab * (2.0 ** -16 + 2 * ((dim + 7) * 2.0 ** -23 * S + 2.0 ** -21) + 2 * (m + 64) * 2.0 ** -24)
            assert (np.abs(got[b, h] - want) <= d + ref.bf16_half_step(np.abs(want) + d)).all(), (b, h)
        at += n
