"""GPU tests of the decoder layer with several new tokens a sequence (decoder.py): prompts, a drafted tree, the path
that is kept, and single tokens after it, each attention against the float64 reference on the layer's own queries and
the cache's own values; captured calls; the two ways of the binding."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import gen
import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import WEIGHT, ExtendCase, dev, i32
from mxfp4_expert_ffn_router_gb300 import decoder

pytestmark = pytest.mark.gpu
H, I, E, K, HQ, HK, D, PAGE = 512, 256, 8, 2, 8, 2, 64, 16


def _bf(seed, *sizes, scale=1.0):
    return dev(ref.bf16_bits(np.random.default_rng(seed).standard_normal(sizes) * scale))


def _val(t):
    return ref.bf16_value(t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16))


class Model:
    def __init__(self, fmt, window, sinks, rotated):
        self.cache = k3.KVCache.empty(60, HK, PAGE, D, fmt)
        self.rotation = k3.Rotation(D, base=1000.0) if rotated else None
        self.window, self.sinks = window, sinks
        experts = k3.Weights.from_stacked(*[torch.from_numpy(z).cuda() for z in gen.expert_arrays(H, I, 0, E)])
        self.weights = (_bf(1, (HQ + 2 * HK) * D, H, scale=H ** -0.5), _bf(2, H, HQ * D, scale=(HQ * D) ** -0.5),
                        _bf(3, E, H, scale=H ** -0.5), 1 + _bf(4, H, scale=0.1), 1 + _bf(5, H, scale=0.1), experts)

    def layer(self, rows):
        return decoder.DecoderLayer(gen.Shape(rows, H, I, E, K), self.cache, HQ, *self.weights, window=self.window,
                                    rotation=self.rotation, sinks=self.sinks)

    def at(self, positions):
        return i32(positions) if self.rotation else None

    def check(self, layer, pages, plan, kin=None):
        """The layer's attention: sequence b's last m tokens are rows from `at` on, its places before them all seen but for
        the window; `kin`: a tree's, else each sees those before it."""
        q, att, scale, at = _val(layer.qkv[:, :HQ]), _val(layer.att), float(np.float32(D ** -0.5)), 0
        for b, m in plan:
            n = pages.lens[b]
            kv = [torch.empty(n, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            k3.k3moe_kv_read(self.cache, pages.slots_of(b), *kv)
            k, v = (t.double().cpu().numpy() for t in kv)
            for i in range(m):
                c = np.arange(n)
                new = np.arange(m) <= i if kin is None else kin[i]
                p = n - m + int(new.sum()) - 1
                see = (c < n - m) & ((self.window == 0) | (c > p - self.window) | (c < self.sinks))
                see[n - m:] = new if kin is not None else new & ((self.window == 0) | (c[n - m:] > p - self.window))
                if kin is None:
                    see[n - m:] |= new & (c[n - m:] < self.sinks)
                for h in range(HQ):
                    g = h // (HQ // HK)
                    want, _, ab, S = ref.attn(q[at + i, h], k[see, g], v[see, g], scale)
                    e = (D + 7) * 2.0 ** -23 * S + 2.0 ** -21
                    d = ab * (WEIGHT + 2 * e + 2 * (n + 64) * 2.0 ** -24)
                    assert (np.abs(att[at + i, h] - want) <= d + ref.bf16_half_step(np.abs(want) + d)).all(), (b, i, h)
            at += m


@pytest.mark.parametrize("fmt,window,sinks,rotated", [(k3.K3MOE_KV_E4M3, 0, 0, True), (k3.K3MOE_KV_BF16, 24, 3, True),
                                                      (k3.K3MOE_KV_E4M3, 30, 2, False), (k3.K3MOE_KV_BF16, 0, 0, False)])
def test_prompts_drafts_and_tokens(fmt, window, sinks, rotated):
    m = Model(fmt, window, sinks, rotated)
    pages = decoder.PageTable(3, 60, PAGE, 12)
    # prompts of 40, 7 and 21 tokens in one call, its last two rows of no sequence
    plan = [(0, 40), (1, 7), (2, 21)]
    layer = m.layer(70)
    slots = torch.cat([pages.append([b], n) for b, n in plan] + [i32([-1, -1])])
    pos = m.at(np.concatenate([np.arange(n) for _, n in plan] + [[0, 0]]))
    x, a = layer.extend(_bf(30, 70, H), _bf(31, 70, H), pages.table, pages.seq_lens, slots, i32([0, 40, 47, 68]), pos)
    m.check(layer, pages, plan)
    assert int(layer.status.item()) == 0 and torch.isfinite(x.float()).all()
    if rotated:  # the keys in the cache are those of the projection, turned by their positions
        from test_gpu_kv_append import turned
        h, _ = torch.empty_like(layer.h), None
        k3.k3moe_rmsnorm(_bf(30, 70, H), layer.norm1, layer.eps, residual=_bf(31, 70, H), y=h)
        qkv = torch.matmul(h, layer.wqkv.t()).view(70, -1, D)
        want, size = turned(_val(qkv[:40, HQ:HQ + HK]), np.arange(40), [1000.0 ** (-2 * i / D) for i in range(D // 2)], False, 1.0)
        got = [torch.empty(40, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        k3.k3moe_kv_read(m.cache, pages.slots_of(0), *got)
        top = np.abs(want).max(-1, keepdims=True) * (2.0 ** -4 if fmt == k3.K3MOE_KV_E4M3 else 2.0 ** -8)
        assert (np.abs(_val(got[0]) - want) <= top + 2.0 ** -20 * size).all()
    # a tree of six drafted tokens for each sequence
    tree, path = [-1, 0, 0, 1, 2, 4], [0, 2, 4]
    masks, offsets, depths = decoder.tree_masks([tree] * 3)
    before = list(pages.lens)
    verify = m.layer(18)
    slots = pages.append(range(3), 6)
    verify.extend(_bf(40, 18, H), None, pages.table, pages.seq_lens, slots, offsets,
                  m.at([before[i // 6] + d for i, d in enumerate(depths)]), masks)
    kin = np.zeros((6, 6), bool)
    for i, p in enumerate(tree):
        kin[i] = kin[p] if p >= 0 else False
        kin[i, i] = True
    m.check(verify, pages, [(b, 6) for b in range(3)], kin)
    assert int(verify.status.item()) == 0
    # one path is kept: the cache holds its vectors at the first places, and the rest as before
    kept = [torch.empty(3, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    old = [torch.empty(before[1], HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k3.k3moe_kv_read(m.cache, pages.slots_of(1)[before[1] + torch.tensor(path, device="cuda")], *kept)
    k3.k3moe_kv_read(m.cache, pages.slots_of(1)[:before[1]].contiguous(), *old)
    for b in range(3):
        decoder.accept(m.cache, pages, b, 6, path, verify.status)
    assert pages.lens == [n + 3 for n in before]
    now = [torch.empty(before[1] + 3, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k3.k3moe_kv_read(m.cache, pages.slots_of(1), *now)
    for t, o, u in zip(now, old, kept):
        assert torch.equal(t[:before[1]], o) and torch.equal(t[before[1]:], u)
    # and single tokens go on from there
    step = m.layer(3)
    x, a = _bf(50, 3, H), None
    for _ in range(2):
        slots = pages.append(range(3))
        x, a = step.step(x.clone(), a, pages.table, pages.seq_lens, slots, m.at([n - 1 for n in pages.lens]))
        m.check(step, pages, [(b, 1) for b in range(3)])
    assert int(step.status.item()) == 0


@pytest.mark.parametrize("kept,count", [([1, 0], 4), ([0, 0], 4), ([4], 4), ([-1], 4)])
def test_accept_refuses(kept, count):
    m = Model(k3.K3MOE_KV_BF16, 0, 0, False)
    pages = decoder.PageTable(1, 60, PAGE, 12)
    pages.append([0], 20)
    with pytest.raises(ValueError):
        decoder.accept(m.cache, pages, 0, count, kept)
    assert pages.lens == [20]


def test_accept_refuses_more_than_there_are():
    m = Model(k3.K3MOE_KV_BF16, 0, 0, False)
    pages = decoder.PageTable(1, 60, PAGE, 12)
    pages.append([0], 3)
    before = m.cache.k.view(torch.int16).clone()  # (bits: the memory may hold NaN)
    with pytest.raises(ValueError):
        decoder.accept(m.cache, pages, 0, 5, [1, 3])
    assert pages.lens == [3] and torch.equal(m.cache.k.view(torch.int16), before)


def test_accept_of_two_layers():
    # pages are shared by the layers: both caches keep the path, and the tokens are forgotten once
    caches = [k3.KVCache.empty(12, heads, PAGE, D, f) for heads, f in ((HK, k3.K3MOE_KV_BF16), (1, k3.K3MOE_KV_E4M3))]
    pages = decoder.PageTable(1, 12, PAGE, 12)
    slots = pages.append([0], 20)
    want = []
    for i, c in enumerate(caches):
        k3.k3moe_kv_write(c, _bf(60 + i, 20, c.heads, D), _bf(70 + i, 20, c.heads, D), slots)
        kv = [torch.empty(18, c.heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        k3.k3moe_kv_read(c, slots[torch.tensor([*range(16), 17, 19], device="cuda")], *kv)
        want.append(kv)
    decoder.accept(caches, pages, 0, 4, [1, 3])
    assert pages.lens == [18]
    for c, w in zip(caches, want):
        kv = [torch.empty(18, c.heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        k3.k3moe_kv_read(c, pages.slots_of(0), *kv)
        assert all(torch.equal(x, y) for x, y in zip(kv, w))


def test_calls_that_do_not_fit_the_layer():
    m = Model(k3.K3MOE_KV_BF16, 0, 0, True)
    pages = decoder.PageTable(1, 60, PAGE, 12)
    layer, slots = m.layer(2), pages.append([0], 2)
    with pytest.raises(ValueError):
        layer.extend(_bf(1, 2, H), None, pages.table, pages.seq_lens, slots, i32([0, 2]))  # no positions
    m.rotation = None
    layer = m.layer(2)
    with pytest.raises(ValueError):
        layer.extend(_bf(1, 2, H), None, pages.table, pages.seq_lens, slots, i32([0, 2]), i32([0, 1]))
    with pytest.raises(ValueError):
        layer.attention(_bf(1, 2, H), None, pages.table, pages.seq_lens, slots, masks=torch.ones(2, 1, dtype=torch.int64, device="cuda"))


def test_a_captured_call_gives_the_same():
    m = Model(k3.K3MOE_KV_E4M3, 40, 2, True)
    pages = decoder.PageTable(2, 60, PAGE, 12)
    layer = m.layer(32)
    slots = torch.cat([pages.append([0], 20), pages.append([1], 12)])
    pos = i32(np.concatenate([np.arange(20), np.arange(12)]))
    x, offs = _bf(30, 32, H), i32([0, 20, 32])
    out, a = (t.clone() for t in layer.extend(x, None, pages.table, pages.seq_lens, slots, offs, pos))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.extend(x, None, pages.table, pages.seq_lens, slots, offs, pos)
    layer.out.zero_()
    graph.replay()
    assert torch.equal(layer.out, out) and torch.equal(layer.a2, a)


def test_a_captured_call_after_a_larger_batch():
    m = Model(k3.K3MOE_KV_E4M3, 0, 0, False)
    layer = m.layer(32)
    few, many = decoder.PageTable(2, 30, PAGE, 12), decoder.PageTable(200, 30, PAGE, 12)
    slots, x, offs = torch.cat([few.append([0], 20), few.append([1], 12)]), _bf(30, 32, H), i32([0, 20, 32])
    out = layer.extend(x, None, few.table, few.seq_lens, slots, offs)[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.extend(x, None, few.table, few.seq_lens, slots, offs)
    held = layer.ws_extend[0]
    layer.extend(x, None, many.table, many.seq_lens, torch.full_like(slots, -1), i32([0] * 201))  # 200 sequences without a token
    assert len(layer.ws_extend) == 2 and layer.ws_extend[0] is held
    layer.out.zero_()
    graph.replay()
    assert torch.equal(layer.out, out) and int(layer.status.item()) == 0


def test_the_command_runs(capsys):
    decoder.main(tokens=2)
    assert "device status 0" in capsys.readouterr().out.splitlines()[-1]


@pytest.mark.parametrize("tree", [False, True])
def test_both_ways_of_the_binding(tree, monkeypatch):
    c = ExtendCase([(70, 9), (0, 20), (500, 3)], 8, 2, 128, 64, k3.K3MOE_KV_E4M3, seed=3)
    masks = c.trees(1) if tree else None
    want = c.run(masks, window=40, sinks=3)
    assert k3._fast is not None
    monkeypatch.setattr(k3, "_fast", None)
    got = c.run(masks, window=40, sinks=3)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
