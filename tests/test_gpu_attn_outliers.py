"""GPU tests of query rows with one large channel over an E4M3 cache, where the kernels of tiles hold a row in two E4M3 numbers a
value: of a row scaled to a largest value in [128, 256) the second number's step is 2^-9 at least, so that a value is off by
2^-10 at most, 2^-17 of the row's largest, and not at all from 2^-2 on.  Scores are off by scale * 2^-17 max|q| sum|K| of the
channels below that: a term of its own beside extend_case.py's."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
from extend_case import E4, WEIGHT, ExtendCase, dev

pytestmark = pytest.mark.gpu
PLAN, HQ, HEADS = [(300, 40), (0, 25)], 64, 8


def _check(c, q_bits, scale):
    out, lse = c.run(q=dev(q_bits))
    got, gl, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), ref.bf16_value(q_bits)
    at = 0
    for b, (ctx, m) in enumerate(c.plan):
        for i in range(0, m, 6):
            r, see = int(c.offsets[b]) + i, slice(at, at + ctx + i + 1)
            for h in range(0, HQ, 5):
                k, v = c.k[see, h // 8], c.v[see, h // 8]
                want, wl, ab, S = ref.attn(q[r, h], k, v, scale)
                top = np.abs(q[r, h]).max()
                low = np.abs(q[r, h]) < 2.0 ** -9 * top
                lost = scale * 2.0 ** -17 * top * np.abs(k[:, low]).sum(-1).max()
                e = (c.dim + 7) * 2.0 ** -23 * S + 2.0 ** -21 + lost
                d = ab * (WEIGHT + 2 * np.expm1(e) + 2 * (len(k) + 64) * 2.0 ** -24)
                assert (np.abs(got[r, h] - want) <= d + ref.bf16_half_step(np.abs(want) + d)).all(), (b, i, h)
                assert abs(gl[r, h] - wl) <= e + (len(k) + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(wl), (b, i, h, gl[r, h] - wl, e)
        at += ctx + m


def _case(dim, k_of):
    def kv(rng, n):
        return ref.bf16_bits(k_of(rng, n)), ref.bf16_bits(rng.standard_normal((n, HEADS, dim)))
    return ExtendCase(PLAN, HQ, HEADS, dim, 32, E4, seed=dim, kv=kv)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [9, 11, 14])
def test_a_large_channel_whose_keys_are_zero(dim, power):
    def keys(rng, n):
        k = rng.standard_normal((n, HEADS, dim))
        k[:, :, 3] = 0
        return k
    c = _case(dim, keys)
    q = c.rng.standard_normal((c.rows, HQ, dim))
    q[:, :, 3] = 2.0 ** power * np.abs(q).max() * (1 + 0.9 * c.rng.random((c.rows, HQ)))
    _check(c, ref.bf16_bits(q), float(np.float32(dim ** -0.5)))


@pytest.mark.parametrize("dim", [64, 128])
def test_the_largest_error(dim):
    """All other channels at the value that loses most, with keys of one sign: the bound is met, and a fourth of it is not."""
    c = _case(dim, lambda rng, n: np.broadcast_to(2.0 ** rng.integers(-3, 2, (n, HEADS, 1)), (n, HEADS, dim)) * (np.arange(dim) > 0))
    q = np.full((c.rows, HQ, dim), 2.0 ** -3 + 2.0 ** -10)
    q[:, :, 0] = 128
    scale = float(np.float32(dim ** -0.5))
    _check(c, ref.bf16_bits(q), scale)
    _, lse = c.run(q=dev(ref.bf16_bits(q)))
    _, wl, _, _ = ref.attn(q[0, 0], c.k[:301, 0], c.v[:301, 0], scale)
    assert abs(lse[0, 0].item() - wl) > scale * 2.0 ** -19 * 128 * (dim - 1) * 0.5
