"""GPU tests of scores so small that the factor of a raw score leaves fp32's numbers: all places weigh the same."""
import pytest

from extend_case import BF, E4, ExtendCase
from test_gpu_attn_tiles import CUT, LINE, ONE, PARTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shape", [ONE, PARTS, LINE, CUT, ([(300, 2), (5, 1)], 8, 4)])
@pytest.mark.parametrize("q_scale,scale", [(2.0 ** -120, 2.0 ** -40), (2.0 ** -125, 2.0 ** -125), (1.0, 2.0 ** -140), (2.0 ** -120, None)])
def test_tiny_scores(q_scale, scale, shape, dim, fmt):
    plan, Hq, heads = shape
    c = ExtendCase(plan, Hq, heads, dim, 64, fmt, seed=dim, q_scale=q_scale)
    c.check(*c.run(scale=scale), scale=scale, rows=lambda b, i: i in (0, 1, 17, 39))
