"""GPU tests of k3moe_kv_append against the rotation in float64.

A rotated value x cos a - y sin a is off by at most e = 2^-21 (|x| + |y|) scale: cos and sin are within 2 units in
the last place (2^-22) of their angle's, whose own error (64-bit turns) is below 2^-30, and two products and a
sum round by 2^-24 each.  q and an unquantised cache add half a bf16 step.  A code of the quantised cache is
off by e and half an E4M3 step of the scale X that the kernel chose, which is one of those that amax - e and
amax + e have."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, dev, i32

pytestmark = pytest.mark.gpu


def turned(x, positions, inv_freq, neighbours, scale):
    """x [n, heads, dim] rotated in float64, and |x| + |y| of each value's pair."""
    rot = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i = np.arange(len(inv_freq))
    p, r = (2 * i, 2 * i + 1) if neighbours else (i, i + len(inv_freq))
    out, size = x.copy(), np.zeros_like(x)
    out[..., p] = (x[..., p] * c - x[..., r] * s) * scale
    out[..., r] = (x[..., r] * c + x[..., p] * s) * scale
    size[..., p] = size[..., r] = np.abs(x[..., p]) + np.abs(x[..., r])
    assert rot <= x.shape[-1]
    return out, size * abs(scale)


class AppendCase:
    def __init__(self, n, Hq, heads, dim, page, fmt, rot, neighbours=False, scale=1.0, seed=0, far=0, pad=0, inv_freq=None):
        rng = np.random.default_rng(seed)
        pages = -(-n // page) + 3
        self.cache = k3.KVCache.empty(pages, heads, page, dim, fmt)
        for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales):
            if t is not None:
                t.fill_(0x55 if t.dtype == torch.uint8 else 7.0)
        self.slots = rng.permutation(pages * page)[:n].astype(np.int32)
        self.slots[rng.permutation(n)[:pad]] = -1
        self.positions = rng.integers(far - far // 3, far + 300, n).astype(np.int32)
        self.x = [ref.bf16_bits(rng.standard_normal((n, h, dim)) * 2.0 ** rng.integers(-6, 7, (n, h, 1)))
                  for h in (Hq, heads, heads)]
        self.inv_freq = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)] if inv_freq is None else inv_freq
        self.rotation = k3.Rotation(rot, inv_freq=self.inv_freq, neighbours=neighbours, scale=scale)
        self.n, self.Hq, self.fmt, self.page, self.neighbours, self.scale = n, Hq, fmt, page, neighbours, scale

    def run(self, q=None, q_out=None, **kw):
        q = dev(self.x[0]) if q is None else q
        q_out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
        k3.k3moe_kv_append(self.cache, dev(self.x[1]), dev(self.x[2]), i32(self.slots), i32(self.positions), self.rotation,
                           q=q, q_out=q_out, **kw)
        return q_out

    def check(self, q_out, left=9.0):
        live = self.slots >= 0
        args = (self.positions, self.inv_freq, self.neighbours, float(np.float32(self.scale)))
        q, qs = turned(ref.bf16_value(self.x[0]), *args)
        got = q_out.double().cpu().numpy()
        e = 2.0 ** -21 * qs
        assert (np.abs(got - q) <= e + ref.bf16_half_step(np.abs(q) + e))[live].all()
        if left is not None:
            assert (got[~live] == left).all()
        k, ks = turned(ref.bf16_value(self.x[1]), *args)
        v = ref.bf16_value(self.x[2])
        pg, pl = np.divmod(self.slots[live], self.page)
        rest = np.ones((self.cache.pages, self.page), bool)
        rest[pg, pl] = False
        for t, s, want, size in ((self.cache.k, self.cache.k_scales, k[live], ks[live]),
                                 (self.cache.v, self.cache.v_scales, v[live], 0 * v[live])):
            e = 2.0 ** -21 * size
            if self.fmt == BF:
                all_ = t.double().cpu().numpy().transpose(0, 2, 1, 3)
                assert (np.abs(all_[pg, pl] - want) <= e + np.where(e > 0, ref.bf16_half_step(np.abs(want) + e), 0)).all()
                assert (all_[rest] == 7).all()
                continue
            codes, bytes_ = t.cpu().numpy().transpose(0, 2, 1, 3), s.cpu().numpy().transpose(0, 2, 1)
            assert (codes[rest] == 0x55).all() and (bytes_[rest] == 0x55).all()
            X = ref.e8m0_value(bytes_[pg, pl])[..., None]
            lo = ref.e8m0_value(ref.mx8(np.maximum(np.abs(want) - e, 0))[1])
            hi = ref.e8m0_value(ref.mx8(np.abs(want) + e)[1])
            assert ((X[..., 0] >= lo) & (X[..., 0] <= hi)).all()
            got = ref.e4m3_value(codes[pg, pl])
            a = (np.abs(want) + e) / X
            step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
            assert (np.abs(got - want / X) <= e / X + step / 2).all()


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("n,Hq,heads,dim,page,rot", [(1, 1, 1, 64, 16, 64), (5, 8, 2, 128, 64, 128), (37, 3, 3, 256, 32, 256),
                                                     (13, 6, 1, 128, 16, 32), (700, 4, 2, 64, 64, 48), (610, 5, 5, 128, 128, 16),
                                                     (3, 96, 96, 128, 64, 128), (9, 7, 1, 256, 1024, 80)])
def test_appends(n, Hq, heads, dim, page, rot, neighbours, fmt):
    c = AppendCase(n, Hq, heads, dim, page, fmt, rot, neighbours, seed=n, far=1000, pad=n // 5)
    c.check(c.run())


@pytest.mark.parametrize("far", [0, 131072, 2 ** 24 + 1, 2 ** 31 - 400])
def test_far_positions(far):
    """Float64 itself holds the angle to 2^-22 at position 2^31."""
    c = AppendCase(50, 2, 2, 128, 64, BF, 128, seed=3, far=far)
    c.check(c.run())


def test_negative_positions_scale_and_odd_frequencies():
    c = AppendCase(30, 2, 2, 64, 16, E4, 32, True, scale=1.3, seed=3, far=100,
                   inv_freq=[0.0, 7.5, -0.3, 1e-9, 3.2, 1e-3] + [0.1] * 10)
    c.positions = -c.positions
    c.check(c.run())


def test_the_same_as_writing_where_nothing_turns():
    """At position 0 the cache holds what k3moe_kv_write leaves, bit for bit."""
    for fmt in (E4, BF):
        c = AppendCase(300, 2, 4, 128, 32, fmt, 128, seed=4, pad=20)
        c.positions[:] = 0
        q = c.run()
        live = c.slots >= 0
        assert torch.equal(q[torch.from_numpy(live)], dev(c.x[0])[torch.from_numpy(live)])
        d = AppendCase(300, 2, 4, 128, 32, fmt, 128, seed=4, pad=20)
        k3.k3moe_kv_write(d.cache, dev(c.x[1]), dev(c.x[2]), i32(c.slots))
        for a, b in ((c.cache.k, d.cache.k), (c.cache.v, d.cache.v), (c.cache.k_scales, d.cache.k_scales),
                     (c.cache.v_scales, d.cache.v_scales)):
            assert a is None or torch.equal(a, b)


def test_in_place_strided_and_without_queries():
    for n in (40, 700):
        c = AppendCase(n, 4, 2, 128, 64, E4, 64, seed=6, pad=3)
        fused = torch.full((n, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        fused[:, :4] = dev(c.x[0])
        want = c.run()
        got = c.run(q=fused[:, :4], q_out=fused[:, :4])
        live = torch.from_numpy(c.slots >= 0).cuda()
        assert torch.equal(got[live], want[live]) and torch.equal(got[~live], dev(c.x[0])[~live])
        assert torch.isnan(fused[:, 4:]).all()
        c.check(want)
        d = AppendCase(n, 4, 2, 128, 64, E4, 64, seed=6, pad=3)
        k3.k3moe_kv_append(d.cache, dev(d.x[1]), dev(d.x[2]), i32(d.slots), i32(d.positions), d.rotation)
        assert torch.equal(c.cache.k, d.cache.k) and torch.equal(c.cache.v_scales, d.cache.v_scales)


def test_values_that_are_not_finite():
    """They stay within their token's head: a group holding one has the scale byte 255."""
    for bad in (float("nan"), float("inf")):
        for fmt in (E4, BF):
            c = AppendCase(20, 2, 2, 64, 16, fmt, 64, seed=2)
            k, v, q = dev(c.x[1]), dev(c.x[2]), dev(c.x[0])
            k[3, 1, 5] = v[4, 0, 7] = q[6, 1, 0] = bad
            q_out = torch.empty_like(q)
            k3.k3moe_kv_append(c.cache, k, v, i32(c.slots), i32(c.positions), c.rotation, q=q, q_out=q_out)
            ok = torch.isfinite(q_out.float())
            assert not ok[6, 1, 0] and int((~ok).sum()) <= 2
            for t, s, where in ((c.cache.k, c.cache.k_scales, (3, 1)), (c.cache.v, c.cache.v_scales, (4, 0))):
                pg, pl = divmod(int(c.slots[where[0]]), 16)
                if fmt == E4:
                    assert s[pg, where[1], pl] == 255 and (t[pg, where[1], pl] == 0x7F).all()
                    assert int((s == 255).sum()) == 1
                else:
                    assert 1 <= int((~torch.isfinite(t.float())).sum()) <= 2


def test_slots_past_the_end():
    c = AppendCase(20, 2, 2, 64, 16, E4, 64, seed=2)
    ok = c.slots.copy()
    c.slots[[3, 9]] = [c.cache.pages * 16, 2 ** 31 - 1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.run(dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.slots[[3, 9]] = -1
    c.check(q)
    c.slots, status = ok, status.zero_()
    c.check(c.run(dev_status=status))
    assert status.item() == 0


def test_captured_and_on_another_stream():
    c = AppendCase(50, 4, 2, 128, 64, E4, 128, seed=7)
    q, k, v = (dev(x) for x in c.x)
    slots, pos, out = i32(c.slots), i32(c.positions), torch.full((50, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    k3.k3moe_kv_append(c.cache, k, v, slots, pos, c.rotation, q=q, q_out=out, stream=st)
    st.synchronize()
    c.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k3.k3moe_kv_append(c.cache, k, v, slots, pos, c.rotation, q=q, q_out=out)
    c.positions = c.positions + 5
    pos.copy_(i32(c.positions))
    graph.replay()
    c.check(out)


def test_refusals():
    c = AppendCase(8, 4, 2, 128, 16, E4, 64)
    q, k, v = (dev(x) for x in c.x)
    slots, pos, out = i32(c.slots), i32(c.positions), torch.empty_like(q)

    def fails(code, **kw):
        a = dict(k=k, v=v, slots=slots, positions=pos, rotation=c.rotation, q=q, q_out=out) | kw
        with pytest.raises((k3.K3moeError, ValueError, TypeError)) as e:
            k3.k3moe_kv_append(c.cache, **a)
        if code is not None:
            assert e.value.code == code
    fails(None, q_out=None)
    fails(None, q=None)
    fails(None, positions=pos.long())
    fails(None, positions=pos[:4])
    fails(None, k=k[:, :1])
    fails(None, v=v.float())
    fails(None, q_out=out[:, :, :64])
    fails(k3.K3MOE_ERR_SHAPE, rotation=k3.Rotation(24))
    fails(k3.K3MOE_ERR_SHAPE, rotation=k3.Rotation(256))
    fails(k3.K3MOE_ERR_ARG, rotation=k3.Rotation(64, scale=float("nan")))
    wide = torch.zeros(8, 4 * 128 + 4, dtype=torch.bfloat16, device="cuda")[:, :512].view(8, 4, 128)
    fails(k3.K3MOE_ERR_ALIGN, q=wide)
    fails(k3.K3MOE_ERR_ALIGN, q_out=wide)
    with pytest.raises(ValueError):
        k3.Rotation(64, inv_freq=[1.0] * 31)
    with pytest.raises(ValueError):
        k3.Rotation(64, inv_freq=[float("inf")] * 32)
    none = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    k3.k3moe_kv_append(c.cache, none, none, slots[:0], pos[:0], c.rotation)
