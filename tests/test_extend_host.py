"""Refusals of k3moe_kv_append, k3moe_attn_extend and k3moe_attn_tree before any launch, and the host's part of the
rotation (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from mxfp4_expert_ffn_router_gb300 import build as k3build

P = 4096  # any aligned non-NULL address: nothing is launched


@pytest.fixture(scope="module")
def L():
    k3build.build()
    return k3.lib()


def _cache(pages=4, page_size=64, heads=2, dim=128, fmt=k3.K3MOE_KV_E4M3, k=P, v=P, ks=P, vs=P):
    return ctypes.byref(k3._KVCacheC(pages, page_size, heads, dim, fmt, k, v, ks, vs))


def _rot(dim=128, neighbours=0, scale=1.0, turns=P):
    return ctypes.byref(k3._RotationC(dim, neighbours, scale, turns))


BAD = [(dict(pages=0), k3.K3MOE_ERR_SHAPE), (dict(page_size=48), k3.K3MOE_ERR_SHAPE), (dict(heads=1025), k3.K3MOE_ERR_SHAPE),
       (dict(dim=96), k3.K3MOE_ERR_SHAPE), (dict(fmt=2), k3.K3MOE_ERR_ARG), (dict(v=0), k3.K3MOE_ERR_ARG),
       (dict(ks=0), k3.K3MOE_ERR_ARG), (dict(k=P + 8), k3.K3MOE_ERR_ALIGN), (dict(vs=P + 1), k3.K3MOE_ERR_ALIGN)]


def _append(L, c=None, n=3, Hq=4, q=P, k=P, v=P, qs=512, ks=256, vs=256, slots=P, pos=P, rot=None, out=P, outs=512):
    return L.k3moe_kv_append(_cache() if c is None else c, n, Hq, q, k, v, qs, ks, vs, slots, pos,
                             _rot() if rot is None else rot, out, outs, None, None)


def _extend(L, c=None, B=2, rows=6, Hq=4, q=P, qs=512, offs=P, most=3, table=P, pages=4, lens=P, window=0, sinks=0, scale=0.1,
            out=P, lse=P, ws=P, nbytes=1 << 40):
    return L.k3moe_attn_extend(_cache() if c is None else c, B, rows, Hq, q, qs, offs, most, table, pages, lens, window, sinks,
                               scale, out, lse, ws, nbytes, None, None)


def _tree(L, c=None, B=2, rows=6, Hq=4, q=P, qs=512, offs=P, masks=P, words=1, table=P, pages=4, lens=P, window=0, sinks=0,
          scale=0.1, out=P, lse=P, ws=P, nbytes=1 << 40):
    return L.k3moe_attn_tree(_cache() if c is None else c, B, rows, Hq, q, qs, offs, masks, words, table, pages, lens, window,
                             sinks, scale, out, lse, ws, nbytes, None, None)


@pytest.mark.parametrize("bad,want", BAD)
def test_cache_refused(L, bad, want):
    assert _append(L, _cache(**bad)) == want and _extend(L, _cache(**bad)) == want and _tree(L, _cache(**bad)) == want
    assert L.k3moe_attn_extend_workspace_bytes(_cache(**bad), 1, 1, 4) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), k3.K3MOE_ERR_SHAPE), (dict(Hq=-1), k3.K3MOE_ERR_SHAPE), (dict(Hq=16385), k3.K3MOE_ERR_SHAPE),
    (dict(rot=_rot(dim=0)), k3.K3MOE_ERR_SHAPE), (dict(rot=_rot(dim=24)), k3.K3MOE_ERR_SHAPE),
    (dict(rot=_rot(dim=144)), k3.K3MOE_ERR_SHAPE), (dict(rot=_rot(neighbours=2)), k3.K3MOE_ERR_ARG),
    (dict(rot=_rot(scale=math.inf)), k3.K3MOE_ERR_ARG), (dict(rot=_rot(turns=0)), k3.K3MOE_ERR_ARG),
    (dict(rot=_rot(turns=P + 4)), k3.K3MOE_ERR_ALIGN), (dict(q=None), k3.K3MOE_ERR_ARG), (dict(out=None), k3.K3MOE_ERR_ARG),
    (dict(k=None), k3.K3MOE_ERR_ARG), (dict(v=None), k3.K3MOE_ERR_ARG), (dict(slots=None), k3.K3MOE_ERR_ARG),
    (dict(pos=None), k3.K3MOE_ERR_ARG), (dict(qs=511), k3.K3MOE_ERR_SHAPE), (dict(ks=255), k3.K3MOE_ERR_SHAPE),
    (dict(vs=248), k3.K3MOE_ERR_SHAPE), (dict(outs=504), k3.K3MOE_ERR_SHAPE), (dict(outs=520), k3.K3MOE_ERR_ARG),
    (dict(out=2 * P, outs=516), k3.K3MOE_ERR_ALIGN), (dict(qs=516, out=2 * P), k3.K3MOE_ERR_ALIGN),
    (dict(k=P + 8), k3.K3MOE_ERR_ALIGN), (dict(q=P + 8), k3.K3MOE_ERR_ALIGN)])
def test_append_refused(L, bad, want):
    assert _append(L, **bad) == want


@pytest.mark.parametrize("call", [_extend, _tree])
@pytest.mark.parametrize("bad,want", [
    (dict(B=-1), k3.K3MOE_ERR_SHAPE), (dict(B=65536), k3.K3MOE_ERR_SHAPE), (dict(rows=-1), k3.K3MOE_ERR_SHAPE),
    (dict(Hq=3), k3.K3MOE_ERR_SHAPE), (dict(Hq=0), k3.K3MOE_ERR_SHAPE), (dict(pages=0), k3.K3MOE_ERR_SHAPE),
    (dict(pages=1 << 25), k3.K3MOE_ERR_SHAPE), (dict(window=-1), k3.K3MOE_ERR_SHAPE), (dict(sinks=-1), k3.K3MOE_ERR_SHAPE),
    (dict(scale=math.nan), k3.K3MOE_ERR_ARG), (dict(q=None), k3.K3MOE_ERR_ARG), (dict(offs=None), k3.K3MOE_ERR_ARG),
    (dict(table=None), k3.K3MOE_ERR_ARG), (dict(lens=None), k3.K3MOE_ERR_ARG), (dict(out=None), k3.K3MOE_ERR_ARG),
    (dict(qs=504), k3.K3MOE_ERR_SHAPE), (dict(qs=516), k3.K3MOE_ERR_ALIGN), (dict(q=P + 2), k3.K3MOE_ERR_ALIGN),
    (dict(out=P + 8), k3.K3MOE_ERR_ALIGN), (dict(ws=None), k3.K3MOE_ERR_WORKSPACE), (dict(nbytes=100), k3.K3MOE_ERR_WORKSPACE),
    (dict(ws=P + 16), k3.K3MOE_ERR_WORKSPACE), (dict(rows=2 ** 31 - 1, Hq=16, qs=2048), k3.K3MOE_ERR_SHAPE)])
def test_attention_refused(L, call, bad, want):
    assert call(L, **bad) == want


def test_each_call_s_own(L):
    assert _extend(L, most=0) == k3.K3MOE_ERR_SHAPE
    assert _tree(L, words=0) == k3.K3MOE_ERR_SHAPE and _tree(L, words=17) == k3.K3MOE_ERR_SHAPE
    assert _tree(L, masks=None) == k3.K3MOE_ERR_ARG and _tree(L, masks=P + 4) == k3.K3MOE_ERR_ALIGN


def test_nothing_to_do(L):
    assert _append(L, n=0, q=None, k=None, v=None, slots=None, pos=None, out=None) == k3.K3MOE_OK
    for call in (_extend, _tree):
        assert call(L, B=0, q=None, out=None, ws=None) == k3.K3MOE_OK
        assert call(L, rows=0, q=None, out=None, ws=None) == k3.K3MOE_OK


def test_workspace(L):
    c = _cache()
    small, large = (L.k3moe_attn_extend_workspace_bytes(c, 2, n, 4) for n in (6, 600000))
    assert 0 < small < large
    need = L.k3moe_attn_extend_workspace_bytes(c, 2, 6, 4)
    assert _extend(L, nbytes=need - 1) == k3.K3MOE_ERR_WORKSPACE


def test_turns():
    """The rotation's numbers: inv_freq / 2 pi modulo 1 in units of 2^-64, to the precision of a double."""
    freqs = [0.0, 1.0, 1e-9, -0.25, 7.5, 2 * math.pi, 3.2, -3.2, 1e6]
    for f, t in zip(freqs, k3._turns(freqs)):
        assert -2 ** 63 <= t < 2 ** 63
        off = (t / 2.0 ** 64 - f / (2 * math.pi)) % 1.0
        assert min(off, 1 - off) <= 2.0 ** -52 * max(1.0, abs(f)), f


def test_binding_refuses_cpu_tensors(L):
    with pytest.raises(ValueError):
        k3.Rotation(64, inv_freq=np.ones(31).tolist(), device="cpu")
    with pytest.raises(ValueError):
        k3.Rotation(64, device="cpu")  # (its numbers are read on the GPU)
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        k3.KVCache(t[None], t[None])
