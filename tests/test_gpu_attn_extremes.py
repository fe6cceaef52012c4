"""GPU tests of k3moe_attn_decode on E4M3 values at the ends of their range, where the
weights' running maximum (score and scale of V) lies far from the scores' own."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
from test_gpu_attn_decode import BF, E4, Case

pytestmark = pytest.mark.gpu
LENGTHS = [[1], [20], [300, 5], [3000], [45000]]  # one step, one block, blocks joined in a cluster, and on the line


def _keys(n, dim, score):
    """Keys whose score is `score` for q = (1, 0, ..) and a scale of 1 (a power of two: exact), spread by up to 1."""
    k = np.zeros((n, 1, dim))
    k[:, 0, 0] = score
    k[:, 0, 1] = np.random.default_rng(n).standard_normal(n) * 0.25
    return k


def _query(c, dim):
    q = np.zeros((len(c.lens), c.Hq, dim))
    q[..., 0], q[..., 1] = 1.0, 0.5
    c.q_bits = ref.bf16_bits(q)


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("score", [0.0, 128.0, 512.0, -512.0])
def test_rows_whose_values_are_all_nan_are_nan(lens, score):
    """Whatever the scores are: lse is a number, the output is not."""
    n, dim = sum(lens), 128
    v = np.full((n, 1, dim), np.nan)
    c = Case(lens, 2, 1, dim, 64, E4, seed=1, kv=(ref.bf16_bits(_keys(n, dim, score)), ref.bf16_bits(v)))
    _query(c, dim)
    out, lse = c.run(scale=1.0)
    assert torch.isnan(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("lens", LENGTHS)
def test_rows_without_weight_stay_zeros(lens):
    """Scores of -inf only: zeros."""
    n, dim = sum(lens), 64
    c = Case(lens, 2, 1, dim, 64, BF, seed=1, kv=(ref.bf16_bits(_keys(n, dim, -np.inf)), ref.bf16_bits(np.full((n, 1, dim), 2.0))))
    _query(c, dim)
    out, lse = c.run(scale=1.0)
    assert not out.float().any() and (lse == -np.inf).all()


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("power", [-100, -118, -124, 100, 117])
def test_tiny_and_huge_values(lens, power):
    """Values of 2^power: within the bound that holds for ordinary ones (it is relative to sum p |V|, plus half a step of
    the bf16 output, 2^-134 at its smallest).  At 2^-124 a vector's scale is at its least, 2^-127."""
    n, dim = sum(lens), 128
    v = np.random.default_rng(2).standard_normal((n, 1, dim)) * 2.0 ** power
    c = Case(lens, 2, 1, dim, 64, E4, seed=3, kv=(ref.bf16_bits(_keys(n, dim, 3.0)), ref.bf16_bits(v)))
    _query(c, dim)
    out, lse = c.run(scale=1.0)
    c.check(out, lse, scale=1.0)


@pytest.mark.parametrize("lens", [[300], [3000], [45000]])
def test_a_sink_of_tiny_values(lens):
    """One token far above the rest whose values are near 2^-124, the others' ordinary: the output is the sum of both."""
    n, dim = sum(lens), 128
    v = np.random.default_rng(4).standard_normal((n, 1, dim))
    v[n // 3] *= 2.0 ** -124
    k = _keys(n, dim, 0.0)
    k[n // 3, 0, 0] = 90.0
    c = Case(lens, 2, 1, dim, 64, E4, seed=5, kv=(ref.bf16_bits(k), ref.bf16_bits(v)))
    _query(c, dim)
    out, lse = c.run(scale=1.0)
    c.check(out, lse, scale=1.0)
