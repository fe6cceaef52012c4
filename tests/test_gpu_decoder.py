"""GPU test of the decoder layer (decoder.py): several steps of a batch whose sequences
start at different lengths, one of them empty, against the operators' float64 references
stage by stage on the layer's own intermediates, and the MoE half bitwise the separate
calls; a captured step gives the same as direct ones."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import gen
import mxfp4_expert_ffn_router_gb300 as k3
from layer_run import alloc_layer
from mxfp4_expert_ffn_router_gb300 import decoder

pytestmark = pytest.mark.gpu
B, H, I, E, K, HQ, HK, D, PAGE = 4, 512, 256, 8, 2, 8, 2, 64, 16


def _bf(seed, *sizes, scale=1.0):
    v = np.random.default_rng(seed).standard_normal(sizes) * scale
    return torch.from_numpy(ref.bf16_bits(v).view(np.int16)).cuda().view(torch.bfloat16)


def _val(t):
    return ref.bf16_value(t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16))


def _layer(fmt, window=0):
    experts = k3.Weights.from_stacked(*[torch.from_numpy(z).cuda() for z in gen.expert_arrays(H, I, 0, E)])
    cache = k3.KVCache.empty(40, HK, PAGE, D, fmt)
    return decoder.DecoderLayer(gen.Shape(B, H, I, E, K), cache, HQ, _bf(1, (HQ + 2 * HK) * D, H, scale=H ** -0.5),
                                _bf(2, H, HQ * D, scale=(HQ * D) ** -0.5), _bf(3, E, H, scale=H ** -0.5),
                                1 + _bf(4, H, scale=0.1), 1 + _bf(5, H, scale=0.1), experts, window=window)


@pytest.mark.parametrize("fmt,window", [(k3.K3MOE_KV_E4M3, 0), (k3.K3MOE_KV_BF16, 0), (k3.K3MOE_KV_E4M3, 20)])
def test_steps_match_the_references(fmt, window):
    layer = _layer(fmt, window)
    pages = decoder.PageTable(B, 40, PAGE, 8)
    for b, n in enumerate((37, 0, 15, 0)):  # prefixes of the sequences; the last row stays empty
        if n:
            s = pages.append([b], n)
            k3.k3moe_kv_write(layer.cache, _bf(10 + b, n, HK, D), _bf(20 + b, n, HK, D), s)
    x, a = _bf(30, B, H), None
    for t in range(4):
        slots = torch.cat([pages.append([0, 1, 2]), torch.tensor([-1], dtype=torch.int32, device="cuda")])
        x0, a0 = x.clone(), None if a is None else a.clone()
        x, a = layer.step(x0, a0, pages.table, pages.seq_lens, slots)
        torch.cuda.synchronize()
        assert int(layer.status.item()) == 0
        # the first norm's sum, and the attention on what the cache now holds
        want_a, _ = ref.rmsnorm(_val(x0), None if a0 is None else _val(a0), _val(layer.norm1), 1e-6)
        np.testing.assert_array_equal(_val(layer.a), ref.bf16_value(ref.bf16_bits(want_a.astype(np.float32))))
        q, att = _val(layer.qkv[:, :HQ]), _val(layer.att)
        for b in range(B):
            n = pages.lens[b]
            kv = [torch.empty(n, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            if n:
                k3.k3moe_kv_read(layer.cache, pages.slots_of(b), *kv)
            lo = max(0, n - window) if window else 0
            for h in range(HQ):
                k, v = (_val(z)[lo:, h // (HQ // HK)] for z in kv)
                want, lse, ab, S = ref.attn(q[b, h], k, v, D ** -0.5)
                bound = ab * (2.0 ** -8 + (D + 20) * 2.0 ** -22 * S + 2.0 ** -18)
                assert (np.abs(att[b, h] - want) <= bound + ref.bf16_half_step(np.abs(want) + bound)).all(), (t, b, h)
        # the new tokens' keys are in their slots
        newk, newv = (torch.empty(B, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k3.k3moe_kv_read(layer.cache, slots, newk, newv)
        wrote = _val(layer.qkv[:, HQ:HQ + HK])[:3]
        half = 2.0 ** -4 if fmt == k3.K3MOE_KV_E4M3 else 0.0  # half an E4M3 step, relatively; subnormal codes below
        assert (np.abs(_val(newk)[:3] - wrote) <= half * np.abs(wrote) + (2.0 ** -18 * np.abs(wrote).max() if half else 0)).all()
        assert not newk[3].any()
        # the MoE half: the same calls on the same norm output, bit for bit
        buf = alloc_layer(layer.s, mode=layer.mode, with_f32=False)
        h = torch.empty_like(layer.h)
        k3.k3moe_rmsnorm(layer.o, layer.norm2, 1e-6, residual=layer.a, y=h)
        assert torch.equal(h, layer.h)
        logits = torch.empty((B, E), device="cuda")
        k3.k3moe_router(layer.s, h, layer.w_router, logits, buf["idx"], buf["w"], buf["status"])
        k3.k3moe_bucket(layer.s, buf["idx"], buf["counts"], buf["offsets"], buf["perm"], buf["inv"], buf["ws_bucket"])
        k3.k3moe_expert_ffn(layer.s, h, layer.experts, buf["offsets"], buf["perm"], buf["Y"], layer.mode, buf["ws_ffn"])
        out = torch.empty((B, H), dtype=torch.bfloat16, device="cuda")
        k3.k3moe_combine(layer.s, buf["Y"], buf["w"], buf["inv"], out)
        assert torch.equal(out, x)
        x, a = x.clone(), a.clone()


def test_a_captured_step_is_the_direct_one():
    layer, pages = _layer(k3.K3MOE_KV_E4M3), decoder.PageTable(B, 40, PAGE, 8)
    x, a, slots = _bf(40, B, H), _bf(41, B, H), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    slots.copy_(pages.append(range(B)))
    layer.step(x, a, pages.table, pages.seq_lens, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, r = layer.step(x, a, pages.table, pages.seq_lens, slots)
    for t in range(20):  # over a page's end
        slots.copy_(pages.append(range(B)))
        x.copy_(_bf(50 + t, B, H))
        g.replay()
        got = y.clone(), r.clone()
        want = layer.step(x, a, pages.table, pages.seq_lens, slots)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), t


def test_pages_come_back():
    pages = decoder.PageTable(2, 3, PAGE, 3)
    pages.append([0], 2 * PAGE)
    pages.append([1], PAGE)
    with pytest.raises(RuntimeError):
        pages.append([1])
    pages.release(0)
    assert pages.seq_lens.tolist()[0] == 0
    s = pages.append([1], PAGE + 1)
    assert len(set(s.tolist())) == PAGE + 1 and pages.seq_lens.tolist() == [0, 2 * PAGE + 1]
