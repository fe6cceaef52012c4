"""GPU tests of k3moe_rmsnorm against the float64 reference, within bounds derived
from the kernel's arithmetic:
  * residual_out is the bf16 rounding of the fp32 sum x + residual, bit for bit;
  * y before its rounding is within REL of the exact value, relatively: one rounding
    of the sum, a sum of squares whose longest chain is under 80 roundings (halved by the
    root), the root's 2 ulp and two products: (1 + 40 + 2 + 2 + 4) 2^-24 < 3e-6;
  * the bf16 y is within that and half a bf16 step of it;
  * a scale is the exact group's, except where the group's maximum is within REL of a
    scale's limit; a code is within half an E4M3 step and REL of the exact value."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3

pytestmark = pytest.mark.gpu
REL = 3e-6
EPS = 1e-6


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _inputs(T, H, seed, residual=True):
    rng = np.random.default_rng(seed)
    x = ref.bf16_bits(rng.standard_normal((T, H)))
    r = ref.bf16_bits(rng.standard_normal((T, H)) * np.exp(rng.standard_normal(H))) if residual else None
    w = ref.bf16_bits(1 + 0.2 * rng.standard_normal(H))
    return x, r, w


def _dev(bits):
    return None if bits is None else torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def _run(x, r, w, eps=EPS, res_out=True, y=True, q=True):
    T, H = x.shape
    new = lambda *s, dt=torch.bfloat16: torch.full(s, 7, dtype=dt, device="cuda")  # noqa: E731
    o = dict(residual_out=new(T, H) if res_out else None, y=new(T, H) if y else None,
             codes=new(T, H, dt=torch.uint8) if q else None, scales=new(T, H // 32, dt=torch.uint8) if q else None)
    k3.k3moe_rmsnorm(_dev(x), _dev(w), eps, residual=_dev(r), **o)
    torch.cuda.synchronize()
    return o


def _check(x, r, w, o, eps=EPS):
    a, y = ref.rmsnorm(ref.bf16_value(x), None if r is None else ref.bf16_value(r), ref.bf16_value(w), eps)
    if o["residual_out"] is not None:
        np.testing.assert_array_equal(_bits(o["residual_out"]), ref.bf16_bits(a.astype(np.float32)))
    if o["y"] is not None:
        got = ref.bf16_value(_bits(o["y"]))
        assert (np.abs(got - y) <= ref.bf16_half_step(np.abs(y) * (1 + REL)) + REL * np.abs(y)).all()
    if o["codes"] is not None:
        T, H = x.shape
        g = y.reshape(T, -1, 32)
        b = o["scales"].cpu().numpy()
        amax = np.abs(g).max(-1)
        lo, hi = ref.mx8(g * (1 - REL))[1], ref.mx8(g * (1 + REL))[1]
        assert ((b == lo) | (b == hi)).all()
        X = ref.e8m0_value(b)[..., None]
        v = ref.e4m3_value(o["codes"].cpu().numpy()).reshape(g.shape) * X
        step = X * 2.0 ** (np.clip(np.floor(np.log2(np.maximum(np.abs(g / X), 1e-300))), -6, 8) - 3)
        assert (np.abs(v - g) <= step / 2 + REL * np.abs(g) + 1e-300).all()
        assert amax.shape == b.shape


@pytest.mark.parametrize("T,H", [(1, 32), (1, 7168), (3, 64), (2, 160), (37, 7168), (300, 4128), (5, 4096), (4, 8224),
                                 (3, 16384), (1000, 256), (13, 224), (2, 16352), (700, 2048)])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm(T, H, residual):
    x, r, w = _inputs(T, H, T + H, residual)
    _check(x, r, w, _run(x, r, w))


@pytest.mark.parametrize("outs", [(True, False, False), (False, True, False), (False, False, True), (True, False, True),
                                  (False, True, True)])
def test_rmsnorm_each_output_alone(outs):
    x, r, w = _inputs(19, 1056, 5)
    some, every = _run(x, r, w, res_out=outs[0], y=outs[1], q=outs[2]), _run(x, r, w)
    _check(x, r, w, some)
    for name, t in some.items():
        if t is not None:
            assert torch.equal(t.view(torch.uint8), every[name].view(torch.uint8)), name


def test_rmsnorm_special_rows():
    """A zero row (zeros out, scale byte 0), tiny and huge rows, a row with an infinity and one with a NaN."""
    T, H = 6, 512
    x, _, w = _inputs(T, H, 9)
    v = ref.bf16_value(x)
    v[1] = 0
    v[2] *= 2.0 ** -120
    v[3] *= 2.0 ** 55
    x = ref.bf16_bits(v)
    x[4, 100] = 0x7F80
    x[5, 200] = 0x7FC1
    o = _run(x, None, w, eps=0.0)
    keep = [0, 3]
    _check(x[keep], None, w, {n: t[keep] for n, t in o.items()}, eps=0.0)
    y, codes, scales = o["y"].float().cpu().numpy(), o["codes"].cpu().numpy(), o["scales"].cpu().numpy()
    # 0 * rsqrt(0) is NaN without eps; with one the row is zeros
    z = _run(x[1:2], None, w)
    assert not z["y"].float().any() and not z["codes"].any() and not z["scales"].any()
    # row 4: finite / inf = 0, inf * 0 = NaN in the one place and its group; row 5: NaN throughout
    assert np.isnan(y[4, 100]) and (np.delete(y[4], 100) == 0).all()
    assert scales[4, 3] == 255 and (np.delete(scales[4], 3) == 0).all() and (codes[4, 96:128] == 0x7F).all()
    assert np.isnan(y[5]).all() and (scales[5] == 255).all() and (codes[5] == 0x7F).all()


def test_rmsnorm_in_place():
    """residual_out over residual and y over x."""
    x, r, w = _inputs(33, 7168, 11)
    want = _run(x, r, w, q=False)
    xd, rd = _dev(x), _dev(r)
    k3.k3moe_rmsnorm(xd, _dev(w), EPS, residual=rd, residual_out=rd, y=xd)
    torch.cuda.synchronize()
    assert torch.equal(xd, want["y"]) and torch.equal(rd, want["residual_out"])


def test_rmsnorm_on_its_stream_and_repeatable():
    x, r, w = _inputs(500, 7168, 12)
    first = _run(x, r, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = _run(x, r, w)
    for n in first:
        assert torch.equal(first[n].view(torch.uint8), again[n].view(torch.uint8)), n
    third = torch.empty_like(first["y"])
    k3.k3moe_rmsnorm(_dev(x), _dev(w), EPS, residual=_dev(r), y=third, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(third, first["y"])
