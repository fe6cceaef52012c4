"""Refusals of the RMS norm, the key-value cache and the decode attention, before
any launch (no GPU needed), and pins of the float64 references that their GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3
from mxfp4_expert_ffn_router_gb300 import build as k3build

P = 4096  # any aligned non-NULL address: nothing is launched


@pytest.fixture(scope="module")
def L():
    k3build.build()
    return k3.lib()


def _cache(pages=4, page_size=64, heads=2, dim=128, fmt=k3.K3MOE_KV_E4M3, k=P, v=P, ks=P, vs=P):
    return ctypes.byref(k3._KVCacheC(pages, page_size, heads, dim, fmt, k, v, ks, vs))


BAD_SHAPES = [dict(pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=2048), dict(heads=0),
              dict(heads=1025), dict(dim=96), dict(dim=512), dict(pages=1 << 21, page_size=1024)]
BAD_ARGS = [dict(fmt=2), dict(fmt=-1), dict(k=0), dict(v=0), dict(ks=0), dict(vs=0)]


@pytest.mark.parametrize("bad,want", [(b, k3.K3MOE_ERR_SHAPE) for b in BAD_SHAPES] +
                         [(b, k3.K3MOE_ERR_ARG) for b in BAD_ARGS] + [(dict(k=P + 8), k3.K3MOE_ERR_ALIGN),
                                                                      (dict(v=P + 4), k3.K3MOE_ERR_ALIGN),
                                                                      (dict(ks=P + 8), k3.K3MOE_ERR_ALIGN),
                                                                      (dict(vs=P + 1), k3.K3MOE_ERR_ALIGN)])
def test_cache_refused_by_every_call(L, bad, want):
    c = _cache(**bad)
    assert L.k3moe_kv_write(c, 1, P, P, 1 << 20, 1 << 20, P, None, None) == want
    assert L.k3moe_kv_read(c, 1, P, P, P, None, None) == want
    assert L.k3moe_attn_decode(c, 1, 1024, P, 1 << 20, P, 4, P, 0, 0.1, P, P, P, 1 << 30, None, None) == want
    assert L.k3moe_attn_decode_workspace_bytes(c, 1, 8) == 0


def test_cache_null(L):
    assert L.k3moe_kv_write(None, 1, P, P, 256, 256, P, None, None) == k3.K3MOE_ERR_ARG
    assert L.k3moe_attn_decode_workspace_bytes(None, 1, 8) == 0


def test_kv_calls_refused(L):
    c = _cache()
    w, r = L.k3moe_kv_write, L.k3moe_kv_read
    assert w(c, -1, P, P, 256, 256, P, None, None) == k3.K3MOE_ERR_SHAPE
    assert w(c, 0, None, None, 0, 0, None, None, None) == k3.K3MOE_OK
    for k, v, slots in ((None, P, P), (P, None, P), (P, P, None)):
        assert w(c, 3, k, v, 256, 256, slots, None, None) == k3.K3MOE_ERR_ARG
        assert r(c, 3, slots, k, v, None, None) == k3.K3MOE_ERR_ARG
    assert w(c, 3, P, P, 255, 256, P, None, None) == k3.K3MOE_ERR_SHAPE
    assert w(c, 3, P, P, 256, 248, P, None, None) == k3.K3MOE_ERR_SHAPE
    assert w(c, 3, P, P, 260, 256, P, None, None) == k3.K3MOE_ERR_ALIGN
    assert w(c, 3, P + 2, P, 256, 256, P, None, None) == k3.K3MOE_ERR_ALIGN
    assert r(c, 3, P, P, P + 8, None, None) == k3.K3MOE_ERR_ALIGN
    assert r(c, -3, P, P, P, None, None) == k3.K3MOE_ERR_SHAPE
    assert r(c, 0, None, None, None, None, None) == k3.K3MOE_OK


def test_attn_refused(L):
    c = _cache()
    need = L.k3moe_attn_decode_workspace_bytes(c, 2, 8)

    def call(B=2, Hq=8, q=P, qs=1024, table=P, pages=4, lens=P, window=0, scale=0.1, out=P, lse=P, ws=P, nb=need):
        return L.k3moe_attn_decode(c, B, Hq, q, qs, table, pages, lens, window, scale, out, lse, ws, nb, None, None)

    for kw in (dict(B=-1), dict(B=65536), dict(Hq=0), dict(Hq=7), dict(Hq=16386), dict(pages=0), dict(window=-1),
               dict(qs=1016), dict(pages=1 << 25)):
        assert call(**kw) == k3.K3MOE_ERR_SHAPE, kw
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) == k3.K3MOE_ERR_ARG, kw
    for kw in (dict(q=P + 2), dict(qs=1028), dict(out=P + 4)):
        assert call(**kw) == k3.K3MOE_ERR_ALIGN, kw
    if need:
        for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=P + 16)):
            assert call(**kw) == k3.K3MOE_ERR_WORKSPACE, kw
    assert call(B=0, q=None, table=None, lens=None, out=None) == k3.K3MOE_OK


def test_rmsnorm_refused(L):
    def call(T=2, H=64, x=P, res=None, w=P, eps=1e-6, ro=None, y=P, codes=None, scales=None):
        return L.k3moe_rmsnorm(T, H, x, res, w, eps, ro, y, codes, scales, None)

    for kw in (dict(T=-1), dict(H=0), dict(H=48), dict(H=16416)):
        assert call(**kw) == k3.K3MOE_ERR_SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(codes=P), dict(scales=P), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == k3.K3MOE_ERR_ARG, kw
    for kw in (dict(x=P + 2), dict(res=P + 8), dict(w=P + 2), dict(ro=P + 8), dict(y=P + 4), dict(codes=P + 8, scales=P)):
        assert call(**kw) == k3.K3MOE_ERR_ALIGN, kw
    assert call(T=0, x=None, w=None, y=None) == k3.K3MOE_OK


def test_no_gpu_means_arch_error(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c = _cache()
    assert L.k3moe_rmsnorm(1, 64, P, None, P, 1e-6, None, P, None, None, None) == k3.K3MOE_ERR_ARCH
    assert L.k3moe_kv_write(c, 1, P, P, 256, 256, P, None, None) == k3.K3MOE_ERR_ARCH
    assert L.k3moe_kv_read(c, 1, P, P, P, None, None) == k3.K3MOE_ERR_ARCH
    assert L.k3moe_attn_decode(c, 1, 8, P, 1024, P, 4, P, 0, 0.1, P, P, P, 1 << 30, None, None) == k3.K3MOE_ERR_ARCH


def test_binding_refusals():
    bf = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        k3.KVCache(bf, bf)  # not on a GPU
    with pytest.raises(ValueError):
        k3.KVCache(bf[0], bf[0])
    with pytest.raises(ValueError):
        k3.KVCache(bf, bf[:, :1])
    u8 = bf.to(torch.uint8)
    with pytest.raises(ValueError):
        k3.KVCache(u8, u8)  # codes without scales
    with pytest.raises(ValueError):
        k3.KVCache(bf, bf, u8[..., 0], u8[..., 0])  # scales without codes
    with pytest.raises(ValueError):
        k3.KVCache(u8, u8, u8[..., 0], u8[:3, ..., 0])
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        k3.k3moe_rmsnorm(x, x[0], 1e-6, y=x)  # not on a GPU
    with pytest.raises(ValueError):
        k3.k3moe_rmsnorm(x, x[0, :32], 1e-6, y=x)
    with pytest.raises(ValueError):
        k3.k3moe_rmsnorm(x, x[0], 1e-6, y=x[:2])


# ---- the references themselves
def test_reference_e4m3_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(ref.e4m3_value(codes.numpy()), codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.02, ref.e4m3_value(np.arange(127)),
                        [(a + b) / 2 for a, b in zip(ref._POS, ref._POS[1:])]]).astype(np.float32)
    np.testing.assert_array_equal(ref.e4m3_nearest(v), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_bf16_and_e8m0_against_torch():
    v = np.random.default_rng(1).standard_normal(4096).astype(np.float32)
    t = torch.from_numpy(v).bfloat16()
    np.testing.assert_array_equal(ref.bf16_bits(v), t.view(torch.int16).numpy().view(np.uint16))
    np.testing.assert_array_equal(ref.bf16_value(ref.bf16_bits(v)), t.double().numpy())
    b = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(ref.e8m0_value(b.numpy()), b.view(torch.float8_e8m0fnu).double().numpy())


def test_reference_mx8_by_hand():
    v = np.zeros((6, 4))
    v[1, 0] = 448.0            # 448 * 2^0: byte 127, code of 448
    v[2, 0] = 449.0            # just over: X = 2, 224.5 -> 224
    v[3] = [1.75, -1.75, 0.5, 2.0 ** -20]  # X = 2^-8
    v[4, 2] = np.inf
    v[5, 1] = np.nan
    codes, b = ref.mx8(v)
    assert b.tolist() == [0, 127, 128, 119, 255, 255]
    assert codes[0].tolist() == [0, 0, 0, 0] and codes[1, 0] == 126 and ref.e4m3_value(codes[2, 0]) == 224
    assert ref.e4m3_value(codes[3]).tolist() == [448, -448, 128, 0]
    assert (codes[4:] == 0x7F).all()


def test_reference_norm_and_attention_against_torch():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 64)), rng.standard_normal(64)
    got = ref.rmsnorm(x, None, w, 1e-5)[1]
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-5)
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-13)
    q, k, v = rng.standard_normal(8), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    out, lse, _, _ = ref.attn(q, k, v, 0.3)
    s = torch.from_numpy(k @ q * 0.3)
    np.testing.assert_allclose(out, (torch.softmax(s, 0) @ torch.from_numpy(v)).numpy(), rtol=1e-13)
    assert abs(lse - float(torch.logsumexp(s, 0))) < 1e-13
    assert ref.attn(q, k[:0], v[:0], 0.3)[1] == -np.inf
