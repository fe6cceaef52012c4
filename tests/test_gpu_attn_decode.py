"""GPU tests of k3moe_attn_decode against the float64 reference on the cache's own
values, row by row, within a bound derived from the kernel's arithmetic.  With ab =
sum p |V| / l of the row and S the largest scale * sum |q K|:
  * a score is a fp32 sum of D exact products and two scalings: off by at most ds =
    (D + 4) 2^-23 S; exp2's argument adds 3 2^-23 max|s| (|s| <= S) and its result 2^-21;
  * weights are rounded before the product with V: half a step of bf16 (2^-8) or f16
    (2^-11, below 2^-28 of the largest product an absolute 2^-38 of it);
  * sums over n tokens in fp32: at most (n + 64) 2^-24 relative to the sum of
    magnitudes, and l the same;
  * the output's own rounding to bf16: half a step.
So |out - ref| <= d + half a step at |out| + d, d = ab (u_p + 2 e + 2 (n + 64) 2^-24), and |lse - ref| <= e +
(n + 64) 2^-24 + 2^-22 |lse| with e = ds + 3 2^-23 S + 2^-21."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3

pytestmark = pytest.mark.gpu
E4, BF = k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _stale(c, bits):
    """Fill a cache with what stale places may hold: NaN, or infinities."""
    if c.format == E4:
        for t in (c.k, c.v):
            t.fill_(0x7F if bits == "nan" else 0x7E)
        for t in (c.k_scales, c.v_scales):
            t.fill_(255 if bits == "nan" else 254)
    else:
        for t in (c.k, c.v):
            t.fill_(float(bits))


class Case:
    """A cache with the sequences' tokens written through the library into shuffled pages."""

    def __init__(self, lens, Hq, heads, dim, page, fmt, seed=0, spread=0, stale="nan", extra_pages=3, kv=None):
        rng = np.random.default_rng(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        pages = sum(need) + extra_pages
        self.cache = k3.KVCache.empty(pages, heads, page, dim, fmt)
        _stale(self.cache, stale)
        order = rng.permutation(pages)
        table = np.full((len(lens), max(1, max(need)) + 1), -1, np.int32)
        at, slots = 0, []
        for b, n in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            t = np.arange(max(n, 0))
            slots.append(mine[t // page] * page + t % page if n > 0 else t)
        slots = np.concatenate(slots).astype(np.int32)
        N = len(slots)
        if kv is None:
            size = 2.0 ** rng.integers(-spread, spread + 1, (2, N, heads, 1))
            k = ref.bf16_bits(rng.standard_normal((N, heads, dim)) * np.minimum(size[0], 1.0))
            v = ref.bf16_bits(rng.standard_normal((N, heads, dim)) * size[1])
        else:
            k, v = kv
        self.slots = torch.from_numpy(slots).cuda()
        k3.k3moe_kv_write(self.cache, _dev(k), _dev(v), self.slots)
        ko, vo = (torch.empty((N, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k3.k3moe_kv_read(self.cache, self.slots, ko, vo)
        self.k, self.v = (t.double().cpu().numpy() for t in (ko, vo))  # the values that the cache holds
        self.q_bits = ref.bf16_bits(rng.standard_normal((len(lens), Hq, dim)) * 1.5)
        self.table, self.lens, self.heads, self.Hq, self.dim, self.fmt = table, list(lens), heads, Hq, dim, fmt

    def run(self, window=0, scale=None, q=None, lse=True, status=None, table=None, lens=None, stream=None):
        B = len(self.lens)
        out = torch.full((B, self.Hq, self.dim), 9.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((B, self.Hq), 9.0, dtype=torch.float32, device="cuda") if lse else None
        ws = torch.full((max(1, k3.k3moe_attn_decode_workspace_bytes(self.cache, B, self.Hq)),), 255, dtype=torch.uint8,
                        device="cuda")
        k3.k3moe_attn_decode(self.cache, _dev(self.q_bits) if q is None else q,
                             torch.from_numpy(self.table if table is None else table).cuda(),
                             torch.tensor(self.lens if lens is None else lens, dtype=torch.int32, device="cuda"), out,
                             lse=l, scale=scale, window=window, ws=ws, dev_status=status, stream=stream)
        return out, l

    def check(self, out, lse, window=0, scale=None, skip=()):
        scale = self.dim ** -0.5 if scale is None else scale
        scale = float(np.float32(scale))
        got, gl = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        q = ref.bf16_value(self.q_bits)
        at = 0
        for b, n in enumerate(self.lens):
            n = max(n, 0)
            lo = max(0, n - window) if window else 0
            for h in range(self.Hq):
                g = h // (self.Hq // self.heads)
                k, v = self.k[at + lo:at + n, g], self.v[at + lo:at + n, g]
                want, wl, ab, S = ref.attn(q[b, h], k, v, scale)
                if (b, h) in skip:
                    continue
                if wl == -np.inf:
                    assert (got[b, h] == 0).all() and (gl is None or gl[b, h] == -np.inf), (b, h)
                    continue
                m = len(k)
                e = (self.dim + 7) * 2.0 ** -23 * S + 2.0 ** -21
                up = (2.0 ** -8 if self.fmt == BF else 2.0 ** -11) + m * 2.0 ** -38
                d = ab * (up + 2 * e + 2 * (m + 64) * 2.0 ** -24)
                bound = d + ref.bf16_half_step(np.abs(want) + d)
                assert (np.abs(got[b, h] - want) <= bound).all(), (b, h, np.abs(got[b, h] - want).max(), bound.min())
                if gl is not None:
                    assert abs(gl[b, h] - wl) <= e + (m + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(wl), (b, h, gl[b, h], wl)
            at += n


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 257, 1000, 0, 48]


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim,page", [(8, 8, 128, 64), (8, 1, 128, 16), (12, 4, 64, 32), (10, 2, 256, 64),
                                               (16, 1, 64, 128), (9, 1, 128, 1024), (40, 2, 128, 32), (5, 5, 256, 16),
                                               (16, 1, 256, 16), (33, 1, 64, 64)])
def test_lengths_and_head_layouts(fmt, Hq, heads, dim, page):
    c = Case(LENS, Hq, heads, dim, page, fmt, seed=Hq + dim)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("window", [1, 16, 33, 64, 500, 5000])
def test_window(fmt, window):
    c = Case([1, 700, 0, 64, 500, 33], 6, 2, 128, 32, fmt, seed=window, stale="inf")
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("lens,Hq,heads,dim,page", [([40000], 8, 1, 128, 64), ([9000, 3, 20011], 4, 2, 64, 16),
                                                    ([5000] * 3 + [17] * 60, 16, 2, 128, 128), ([30000], 2, 2, 256, 32)])
def test_long_caches_are_split_and_joined(fmt, lens, Hq, heads, dim, page):
    c = Case(lens, Hq, heads, dim, page, fmt, seed=3)
    out, lse = c.run()
    c.check(out, lse)
    again, lse2 = c.run()  # a split does not change from run to run, whatever the workspace held
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 200, 700).tolist()
    c = Case(lens, 4, 2, 64, 16, E4, seed=6)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("B,most,Hq,heads,dim,page,window", [
    (70, 100, 8, 8, 128, 16, 0), (160, 200, 24, 2, 128, 32, 0), (150, 220, 12, 4, 64, 32, 0), (600, 1, 8, 1, 128, 16, 0),
    (120, 300, 20, 4, 256, 16, 33), (80, 110, 40, 4, 256, 16, 0), (170, 60, 17, 1, 64, 64, 0), (300, 60, 16, 1, 128, 16, 0),
    (300, 60, 16, 1, 256, 16, 0), (250, 60, 17, 1, 64, 64, 0), (250, 100, 24, 2, 128, 16, 0), (240, 100, 12, 4, 64, 16, 50)])
def test_many_short_sequences(fmt, B, most, Hq, heads, dim, page, window):
    """More short items than the GPU holds at once: each is one warp's."""
    lens = np.random.default_rng(B).integers(0, most + 1, B)
    lens[:2] = most, 0
    c = Case(lens.tolist(), Hq, heads, dim, page, fmt, seed=dim + Hq)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("B,most,Hq,heads,dim,page,window", [
    (30, 3000, 16, 1, 64, 32, 0), (30, 1500, 11, 1, 256, 16, 0), (4, 1800, 18, 2, 256, 64, 0), (25, 200, 130, 10, 64, 16, 0),
    (20, 700, 40, 4, 128, 32, 300), (3, 3900, 6, 2, 256, 32, 0), (19, 240, 128, 8, 64, 128, 0), (2, 40, 27, 3, 256, 16, 0)])
def test_few_sequences_of_shared_heads(fmt, B, most, Hq, heads, dim, page, window):
    """Up to one item an SM or little more, with more than 8 query heads a key: split by 8 or shared by 16."""
    lens = np.random.default_rng(B + most).integers(0, most + 1, B)
    lens[:2] = most, 0
    c = Case(lens.tolist(), Hq, heads, dim, page, fmt, seed=dim + Hq)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("fmt", [E4, BF])
def test_many_short_sequences_with_bad_pages(fmt):
    c = Case([70, 100, 90] + [40] * 120, 8, 4, 128, 16, fmt, seed=21)
    good, good_lse = c.run()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1, c.cache.pages, 2 ** 31 - 1):
        table = c.table.copy()
        table[2, 5] = bad  # its last page: places 80 to 89
        st.zero_()
        out, lse = c.run(table=table, status=st)
        assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
        short, short_lse = c.run(lens=[70, 100, 80] + [40] * 120)
        torch.testing.assert_close(out[2].float(), short[2].float(), rtol=2.0 ** -7, atol=1e-3)
        torch.testing.assert_close(lse[2], short_lse[2], rtol=2.0 ** -18, atol=2.0 ** -18)
        out[2], lse[2] = good[2], good_lse[2]
        assert torch.equal(out, good) and torch.equal(lse, good_lse)
    st.zero_()
    out, lse = c.run(lens=[-5, 100, 2 ** 31 - 1] + [40] * 120, status=st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS and not out[0].float().any() and torch.isinf(lse[0]).all()
    assert torch.equal(out[1], good[1]) and torch.equal(out[3:], good[3:])


@pytest.mark.parametrize("fmt", [E4, BF])
def test_everything_empty(fmt):
    c = Case([0, 0, 0], 8, 2, 128, 16, fmt)
    c.check(*c.run())


def test_values_of_very_different_size():
    """Values whose scales span 2^80: the weights meet the scales before they are rounded."""
    c = Case([700, 40], 8, 2, 128, 64, E4, seed=8, spread=40)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [E4, BF])
def test_peaked_and_flat_scores(fmt):
    """One token far above the rest, a slow drift upwards (the running maximum rises at
    every tile), equal scores, and a sink: a score far above the rest whose value is zero."""
    n, dim = 3000, 128
    rng = np.random.default_rng(9)
    for kind in ("peak", "rise", "flat", "sink", "negative"):
        k = np.zeros((n, 1, dim))
        v = rng.standard_normal((n, 1, dim))
        k[:, 0, 1] = rng.standard_normal(n)
        if kind in ("peak", "sink"):
            k[1234, 0, 0] = 300.0 if kind == "peak" else 60.0
        if kind == "sink":
            v[1234] = 0.0
        if kind == "rise":
            k[:, 0, 0] = np.linspace(-100, 100, n)
        if kind == "flat":
            k[:] = 0.0
        if kind == "negative":
            k[:, 0, 0] = -500.0
        c = Case([n], 4, 1, dim, 64, fmt, seed=10, kv=(ref.bf16_bits(k), ref.bf16_bits(v)))
        q = np.zeros((1, 4, dim))
        q[..., 0], q[..., 1] = 1.0, 0.5
        c.q_bits = ref.bf16_bits(q)
        c.check(*c.run(scale=0.25), scale=0.25)


def test_non_finite_tokens_reach_their_heads_only():
    """A NaN or infinite key or value that is seen makes its head's rows NaN, as the
    formula does; a score of -inf drops its token; a row of such scores only is zeros."""
    n, heads, dim = 100, 6, 64
    rng = np.random.default_rng(11)
    k, v = (ref.bf16_bits(rng.standard_normal((n, heads, dim))) for _ in range(2))
    k[50, 0, 3] = 0x7FC0          # NaN key
    v[60, 1, 4] = 0x7FC0          # NaN value
    k[70, 2, 0] = 0x7F80          # infinite key, q[0] > 0: score inf, inf - inf
    k[80, 3, 0] = 0xFF80          # score -inf: no weight
    k[:, 4, 0] = 0xFF80           # nothing but -inf
    c = Case([n], heads, heads, dim, 16, BF, seed=12, kv=(k, v))
    c.q_bits[0, :, 0] = 0x3F80    # q[0] = 1
    out, lse = c.run()
    c.check(out, lse, skip={(0, 0), (0, 1), (0, 2)})
    got = out.float().cpu().numpy()[0]
    assert np.isnan(got[0]).all() and np.isnan(lse[0, 0].item())
    assert np.isnan(got[1, 4]) and np.isfinite(np.delete(got[1], 4)).all() and np.isfinite(lse[0, 1].item())
    assert np.isnan(got[2]).all()
    assert np.isfinite(got[3]).all() and (got[4] == 0).all() and np.isfinite(got[5]).all()
    e = Case([n], heads, heads, dim, 16, E4, seed=12, kv=(k, v))  # quantised: the vector is NaN as a whole
    out, lse = e.run()
    got = out.float().cpu().numpy()[0]
    for h in range(5):
        assert np.isnan(got[h]).all(), h
    assert np.isfinite(lse[0, 1].item()) and np.isnan(lse[0, 0].item())
    e.check(out, lse, skip={(0, h) for h in range(5)})


@pytest.mark.parametrize("fmt", [E4, BF])
def test_large_and_small_queries(fmt):
    """Query rows of very different size, one with an outlier, a zero row, a negative and a zero scale."""
    c = Case([300, 20], 8, 2, 128, 32, fmt, seed=13)
    q = ref.bf16_value(c.q_bits)
    q[0, 0] *= 2.0 ** -40
    q[0, 1, 7] = 300.0
    q[0, 2] = 0.0
    q[0, 3] *= 30
    q[1, 0] = 2.0 ** -130
    c.q_bits = ref.bf16_bits(q)
    c.check(*c.run())
    c.check(*c.run(scale=-0.02), scale=-0.02)
    c.check(*c.run(scale=0.0), scale=0.0)


@pytest.mark.parametrize("fmt", [E4, BF])
def test_strided_queries_streams_and_optional_outputs(fmt):
    c = Case([77, 1, 300], 8, 2, 128, 32, fmt, seed=14)
    fused = torch.full((3, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = _dev(c.q_bits)
    out, lse = c.run()
    c.check(out, lse)
    strided, _ = c.run(q=fused[:, 2:10], lse=False)
    assert torch.equal(out, strided)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other, _ = c.run()
    st.synchronize()
    assert torch.equal(out, other)


def test_lengths_and_pages_out_of_range():
    """A negative length is an empty row, one past the table is the table's, a page
    outside the cache counts as not seen: each sets K3MOE_DEV_BOUNDS."""
    page = 16
    c = Case([40, 64, 50], 4, 2, 64, page, E4, seed=15)
    good, _ = c.run()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(lens=[-5, 64, 50], status=st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS and not out[0].float().any() and torch.isinf(lse[0]).all()
    assert torch.equal(out[1:], good[1:])
    st.zero_()
    out, _ = c.run(table=np.ascontiguousarray(c.table[:, :4]), lens=[40, 2 ** 31 - 1, 50], status=st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS and torch.equal(out, good)
    for bad in (-1, c.cache.pages, 2 ** 31 - 1):
        table = c.table.copy()
        table[2, 3] = bad           # its last page: places 48 and 49
        st.zero_()
        out, lse = c.run(table=table, status=st)
        assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
        assert torch.equal(out[:2], good[:2])
        short, _ = c.run(lens=[40, 64, 48])
        # the same tokens; the split may fall elsewhere: within two roundings of bf16
        torch.testing.assert_close(out[2].float(), short[2].float(), rtol=2.0 ** -7, atol=1e-3)
    c.run(lens=[-1, 64, 50])  # without a status word
    torch.cuda.synchronize()


def test_captured_in_a_graph_follows_the_lengths():
    """A captured call reads lengths and tables at replay: nothing about them is fixed on the host."""
    c = Case([1500, 90, 700], 8, 2, 128, 64, E4, seed=16)
    B = 3
    out = torch.empty((B, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, 8), device="cuda")
    ws = torch.empty(max(1, k3.k3moe_attn_decode_workspace_bytes(c.cache, B, 8)), dtype=torch.uint8, device="cuda")
    q, table = _dev(c.q_bits), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    k3.k3moe_attn_decode(c.cache, q, table, lens, out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k3.k3moe_attn_decode(c.cache, q, table, lens, out, lse=lse, ws=ws)
    for new in ([1500, 90, 700], [1, 0, 65], [1499, 90, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(9.0)
        g.replay()
        want, wl = c.run(lens=new)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl), new


def test_a_cache_past_32_bits():
    """Pages whose byte and element offsets pass 32 bits."""
    for fmt, pages in ((BF, 20000), (E4, 40000)):
        c = Case([130, 64], 16, 16, 128, 64, fmt, seed=17, extra_pages=pages)
        c.check(*c.run())
