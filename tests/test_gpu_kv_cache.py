"""GPU tests of the paged key-value cache: written codes and scales are bit for bit
the float64 reference's (the inputs are bf16, v / X is exact, so every rounding decision
is the exact one), untouched places keep their bytes, and slots read back as the bf16
rounding of code * scale."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _cache(pages, heads, page, dim, fmt):
    c = k3.KVCache.empty(pages, heads, page, dim, fmt)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 120, b.shape, dtype=torch.uint8, device="cuda", generator=g))
    return c


def _vectors(n, heads, dim, seed):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((n, heads, dim)) * 2.0 ** rng.integers(-30, 30, (n, heads, 1))
    v[rng.random((n, heads, dim)) < 0.1] *= 2.0 ** -9   # values that land on subnormal codes
    v[rng.random((n, heads)) < 0.05] = 0.0
    return ref.bf16_bits(v)


def _slots(n, places, seed, pad=0):
    rng = np.random.default_rng(seed)
    s = rng.permutation(places)[:n].astype(np.int32)
    s[rng.permutation(n)[:pad]] = -1
    return s


def _host(c):
    return {n: (None if t is None else t.view(torch.uint8).cpu().numpy().copy())
            for n, t in (("k", c.k), ("v", c.v), ("k_scales", c.k_scales), ("v_scales", c.v_scales))}


def _expect(before, c, slots, new):
    """The cache's bytes after a write of new = {"k": bits, "v": bits}."""
    want = {n: (None if b is None else b.copy()) for n, b in before.items()}
    live = (slots >= 0) & (slots < c.pages * c.page_size)
    pg, at = slots[live] // c.page_size, slots[live] % c.page_size
    for n in ("k", "v"):
        bits = new[n][live]
        if c.format == k3.K3MOE_KV_BF16:
            want[n].view(np.uint16)[pg, :, at] = bits
        else:
            want[n][pg, :, at], want[n + "_scales"][pg, :, at] = ref.mx8(ref.bf16_value(bits))
    return want


def _same(got, want):
    for n in got:
        if got[n] is not None:
            np.testing.assert_array_equal(got[n], want[n], err_msg=n)


def _read_expect(h, c, slots):
    live = (slots >= 0) & (slots < c.pages * c.page_size)
    out = []
    for n in ("k", "v"):
        r = np.zeros((len(slots), c.heads, c.dim), np.uint16)
        pg, at = slots[live] // c.page_size, slots[live] % c.page_size
        if c.format == k3.K3MOE_KV_BF16:
            r[live] = h[n].view(np.uint16)[pg, :, at]
        else:
            v = ref.e4m3_value(h[n][pg, :, at]) * ref.e8m0_value(h[n + "_scales"][pg, :, at])[..., None]
            r[live] = ref.bf16_bits(v.astype(np.float32))
        out.append(r)
    return out


@pytest.mark.parametrize("fmt", [k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16])
@pytest.mark.parametrize("n,heads,dim,page,pad", [(1, 1, 64, 16, 0), (13, 96, 128, 64, 3), (7, 5, 256, 32, 7),
                                                   (1000, 8, 128, 64, 11), (3001, 3, 64, 128, 0), (515, 1, 256, 1024, 2),
                                                   (31, 2, 128, 16, 1)])
def test_write_and_read_back(fmt, n, heads, dim, page, pad):
    c = _cache(n // page + 2, heads, page, dim, fmt)
    before = _host(c)
    slots = _slots(n, c.pages * page, n, pad)
    new = {"k": _vectors(n, heads, dim, 1), "v": _vectors(n, heads, dim, 2)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    k3.k3moe_kv_write(c, _dev(new["k"]), _dev(new["v"]), sl, st)
    after = _host(c)
    _same(after, _expect(before, c, slots, new))
    ko, vo = (torch.full((n, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3.k3moe_kv_read(c, sl, ko, vo, st)
    for got, want in zip((ko, vo), _read_expect(after, c, slots)):
        np.testing.assert_array_equal(_bits(got), want)
    assert int(st.item()) == 0


@pytest.mark.parametrize("fmt", [k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16])
def test_write_from_slices_of_a_fused_projection(fmt):
    n, heads, dim = 77, 4, 128
    qkv = _dev(_vectors(n, 10, dim, 3))  # 2 other heads, 4 keys, 4 values
    k, v = qkv[:, 2:6], qkv[:, 6:]
    slots = _slots(n, 3 * 64, 4)
    a, b = _cache(3, heads, 64, dim, fmt), _cache(3, heads, 64, dim, fmt)
    sl = torch.from_numpy(slots).cuda()
    k3.k3moe_kv_write(a, k, v, sl)
    k3.k3moe_kv_write(b, k.contiguous(), v.contiguous(), sl)
    _same(_host(a), _host(b))
    _same(_host(a), _expect(_host(_cache(3, heads, 64, dim, fmt)), a, slots, {"k": _bits(k), "v": _bits(v)}))


def test_special_vectors():
    """Zeros, signed zeros, subnormal, the largest values, infinities and NaN."""
    heads, dim = 2, 64
    bits = _vectors(9, heads, dim, 5)
    bits[0] = 0x8000                    # -0 throughout
    bits[1] = 0x0001                    # the smallest subnormal
    bits[2] = 0x7F7F                    # the largest finite value: the exponent is at its limit
    bits[3, 0, 5], bits[3, 1, 6] = 0x7F80, 0xFF80
    bits[4, 0, 7] = 0x7FC0
    bits[5], bits[5, :, 0] = 0x0000, 0x43E0   # 448 and zeros
    bits[6], bits[6, :, 0] = 0x0000, 0x43E1   # the next value up
    bits[7] = 0x0080                    # the smallest normal
    c = _cache(1, heads, 16, dim, k3.K3MOE_KV_E4M3)
    before = _host(c)
    slots = np.arange(9, dtype=np.int32)
    sl = torch.from_numpy(slots).cuda()
    k3.k3moe_kv_write(c, _dev(bits), _dev(bits[::-1]), sl)
    after = _host(c)
    _same(after, _expect(before, c, slots, {"k": bits, "v": bits[::-1]}))
    ko, vo = (torch.empty((9, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3.k3moe_kv_read(c, sl, ko, vo)
    want = _read_expect(after, c, slots)
    for got, w in zip((_bits(ko), _bits(vo)), want):
        nan = np.isnan(ref.bf16_value(w))
        np.testing.assert_array_equal(np.isnan(ref.bf16_value(got)), nan)
        np.testing.assert_array_equal(got[~nan], w[~nan])


@pytest.mark.parametrize("fmt", [k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16])
def test_slots_past_the_end(fmt):
    c = _cache(2, 3, 16, 64, fmt)
    before = _host(c)
    slots = np.array([3, 32, -7, 31, 2 ** 31 - 1, -2 ** 31], np.int32)
    new = {"k": _vectors(6, 3, 64, 1), "v": _vectors(6, 3, 64, 2)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    k3.k3moe_kv_write(c, _dev(new["k"]), _dev(new["v"]), sl, st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
    after = _host(c)
    _same(after, _expect(before, c, slots, new))
    st.zero_()
    ko, vo = (torch.full((6, 3, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3.k3moe_kv_read(c, sl, ko, vo, st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
    for got, want in zip((ko, vo), _read_expect(after, c, slots)):
        np.testing.assert_array_equal(_bits(got), want)
    k3.k3moe_kv_write(c, _dev(new["k"]), _dev(new["v"]), sl)  # without a status word
    torch.cuda.synchronize()


def test_a_cache_past_32_bits():
    """Places whose byte offsets (5 GB) and element offsets (2.6 G) pass 32 bits."""
    heads, dim, page = 16, 128, 64
    pages = 20000
    c = k3.KVCache.empty(pages, heads, page, dim, k3.K3MOE_KV_BF16)
    q = k3.KVCache.empty(2 * pages, heads, page, dim, k3.K3MOE_KV_E4M3)
    for cache in (c, q):
        end = cache.pages * page
        slots = np.array([0, end - 1, end // 2, end - page, 17], np.int32)
        new = {"k": _vectors(5, heads, dim, 1), "v": _vectors(5, heads, dim, 2)}
        sl = torch.from_numpy(slots).cuda()
        k3.k3moe_kv_write(cache, _dev(new["k"]), _dev(new["v"]), sl)
        ko, vo = (torch.empty((5, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k3.k3moe_kv_read(cache, sl, ko, vo)
        for got, bits in ((ko, new["k"]), (vo, new["v"])):
            want = bits
            if cache is q:
                codes, b = ref.mx8(ref.bf16_value(bits))
                want = ref.bf16_bits((ref.e4m3_value(codes) * ref.e8m0_value(b)[..., None]).astype(np.float32))
            np.testing.assert_array_equal(_bits(got), want)
