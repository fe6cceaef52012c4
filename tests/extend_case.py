"""Cases of attention of several new tokens per sequence (k3moe_attn_extend, k3moe_attn_tree): a
cache with the sequences' tokens in shuffled pages, the rows' float64 references on the
cache's own values, and the bound that a row's outputs have to keep.

Bound: with ab = sum p |V| / l of a row, S the largest scale * sum |q K| and n the places seen:
  * a score is a fp32 sum of D exact products and a scaling: off by at most (D + 7) 2^-23 S with the
    argument of exp2 (|s| <= S), whose result is off by 2^-21 at most: e;
  * a weight is rounded to bf16 before the product with V: WEIGHT of it;
  * sums over n places in fp32, in any order, with the running maximum's corrections: 2 (n + 64) 2^-24 of the
    sum of magnitudes, and l the same;
  * the output's own rounding to bf16: half a step.
|out - ref| <= d + half a step at |out| + d, d = ab (WEIGHT + 2 e + 2 (n + 64) 2^-24), and |lse - ref| <= e +
(n + 64) 2^-24 + 2^-22 |lse|."""
import numpy as np
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3

E4, BF = k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16
WEIGHT = 2.0 ** -8


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def i32(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def tree_masks(rng, m, words):
    """Masks of a random tree of m nodes: bool [m, m] and its words."""
    kin = np.zeros((m, m), bool)
    for i in range(m):
        p = int(rng.integers(max(-1, i - 5), i))
        if p >= 0:
            kin[i] = kin[p]
        kin[i, i] = True
    return kin


def mask_words(kin, words):
    """bool [m, m] -> int64 [m, words]."""
    m = len(kin)
    full = np.zeros((m, 64 * words), bool)
    full[:, :min(kin.shape[1], 64 * words)] = kin[:, :64 * words]
    bits = full.reshape(m, words, 64).astype(np.uint64) << np.arange(64, dtype=np.uint64)
    return np.bitwise_or.reduce(bits, -1).view(np.int64)


class ExtendCase:
    """``plan``: (places before the new tokens, new tokens) of each sequence."""

    def __init__(self, plan, Hq, heads, dim, page, fmt, seed=0, pad=(0, 0), stale="nan", kv=None, spread=0, q_scale=1.5):
        rng = self.rng = np.random.default_rng(seed)
        lens = [c + m for c, m in plan]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        self.cache = c = k3.KVCache.empty(pages, heads, page, dim, fmt)
        for t in (c.k, c.v):
            t.fill_((0x7F if stale == "nan" else 0x7E) if fmt == E4 else float(stale))
        if fmt == E4:
            for t in (c.k_scales, c.v_scales):
                t.fill_(255 if stale == "nan" else 254)
        order = rng.permutation(pages)
        table = np.full((len(plan), max(1, max(need)) + 1), -1, np.int32)
        at, slots = 0, []
        for b, n in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            t = np.arange(n)
            slots.append(mine[t // page] * page + t % page if n else t)
        slots = np.concatenate(slots).astype(np.int32)
        N = len(slots)
        if kv is None:
            size = 2.0 ** rng.integers(-spread, spread + 1, (2, N, heads, 1))
            k = ref.bf16_bits(rng.standard_normal((N, heads, dim)) * np.minimum(size[0], 1.0))
            v = ref.bf16_bits(rng.standard_normal((N, heads, dim)) * size[1])
        else:
            k, v = kv(rng, N)
        self.slots = torch.from_numpy(slots).cuda()
        k3.k3moe_kv_write(c, dev(k), dev(v), self.slots)
        ko, vo = (torch.empty((N, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k3.k3moe_kv_read(c, self.slots, ko, vo)
        self.k, self.v = (t.double().cpu().numpy() for t in (ko, vo))  # the values that the cache holds
        self.plan, self.lens, self.table = list(plan), lens, table
        self.Hq, self.heads, self.dim, self.fmt, self.pad = Hq, heads, dim, fmt, pad
        self.offsets = np.concatenate([[pad[0]], pad[0] + np.cumsum([m for _, m in plan])]).astype(np.int32)
        self.rows = int(self.offsets[-1]) + pad[1]
        self.q_bits = ref.bf16_bits(rng.standard_normal((self.rows, Hq, dim)) * q_scale)

    def trees(self, words, kind="tree"):
        """Masks for all rows; ``kind``: tree, chain, or any bits at all (rows without one among them)."""
        self.kin = []
        for _, m in self.plan:
            if kind == "tree":
                self.kin.append(tree_masks(self.rng, m, words))
            elif kind == "chain":
                self.kin.append(np.tril(np.ones((m, m), bool)))
            else:
                k = self.rng.random((m, m)) < 0.3
                k[::3] = False
                self.kin.append(k)
        out = self.rng.integers(-2 ** 63, 2 ** 63 - 1, (self.rows, words))  # (rows of no sequence: anything)
        for b, (_, m) in enumerate(self.plan):
            w = mask_words(self.kin[b], words)
            if m < 64 * words:  # bits past the last new token mean nothing
                noise = mask_words(np.ones((1, 64 * words), bool) & (np.arange(64 * words) >= m), words)
                w = w | (noise & self.rng.integers(-2 ** 63, 2 ** 63 - 1, w.shape))
            out[self.offsets[b]:self.offsets[b] + m] = w
        return torch.from_numpy(out).cuda()

    def args(self):
        return i32(self.offsets), i32(self.table), i32(self.lens)

    def workspace(self, rows=None):
        n = k3.k3moe_attn_extend_workspace_bytes(self.cache, len(self.plan), self.rows if rows is None else rows, self.Hq)
        return torch.full((max(1, n),), 255, dtype=torch.uint8, device="cuda")

    def outputs(self):
        return (torch.full((self.rows, self.Hq, self.dim), 9.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.rows, self.Hq), 9.0, dtype=torch.float32, device="cuda"))

    def run(self, masks=None, window=0, sinks=0, max_new=None, q=None, lse=True, table=None, lens=None, offsets=None, **kw):
        out, l = self.outputs()
        o, t, n = self.args()
        o = o if offsets is None else i32(offsets)
        t = t if table is None else i32(table)
        n = n if lens is None else i32(lens)
        q = dev(self.q_bits) if q is None else q
        kw.setdefault("ws", self.workspace())
        if masks is None:
            k3.k3moe_attn_extend(self.cache, q, o, t, n, out, lse=l if lse else None, window=window, sinks=sinks,
                                 max_new=max_new, **kw)
        else:
            k3.k3moe_attn_tree(self.cache, q, o, masks, t, n, out, lse=l if lse else None, window=window, sinks=sinks, **kw)
        return out, l

    def seen(self, b, i, tree, window, sinks):
        """Which of sequence b's places row i sees."""
        ctx, m = self.plan[b]
        c = np.arange(ctx + m)
        if not tree:
            p = ctx + i
            return (c <= p) & ((window == 0) | (c > p - window) | (c < sinks))
        kin = self.kin[b][i]
        p = ctx + max(0, int(kin.sum()) - 1)
        s = np.concatenate([np.ones(ctx, bool), kin])
        return s & ((c >= ctx) | (window == 0) | (c > p - window) | (c < sinks))

    def check(self, out, lse, tree=False, window=0, sinks=0, scale=None, skip=(), hidden=None, rows=None):
        """``hidden``: places of a sequence that count as not seen ({b: bool array}); ``rows``: of each sequence, which to look at."""
        scale = float(np.float32(self.dim ** -0.5 if scale is None else scale))
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = ref.bf16_value(self.q_bits)
        at = 0
        for b, (ctx, m) in enumerate(self.plan):
            n = ctx + m
            for i in range(m):
                if b in skip or (rows is not None and not rows(b, i)):
                    continue
                see = self.seen(b, i, tree, window, sinks)
                if hidden and b in hidden:
                    see = see & ~hidden[b]
                r = int(self.offsets[b]) + i
                for h in range(self.Hq):
                    g = h // (self.Hq // self.heads)
                    k, v = self.k[at:at + n, g][see], self.v[at:at + n, g][see]
                    want, wl, ab, S = ref.attn(q[r, h], k, v, scale)
                    if wl == -np.inf:
                        assert (got[r, h] == 0).all() and gl[r, h] == -np.inf, (b, i, h)
                        continue
                    e = (self.dim + 7) * 2.0 ** -23 * S + 2.0 ** -21
                    d = ab * (WEIGHT + 2 * e + 2 * (len(k) + 64) * 2.0 ** -24)
                    bound = d + ref.bf16_half_step(np.abs(want) + d)
                    off = np.abs(got[r, h] - want)
                    assert (off <= bound).all(), (b, i, h, off.max(), bound.min())
                    assert abs(gl[r, h] - wl) <= e + (len(k) + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(wl), (b, i, h, gl[r, h], wl)
            at += n
        left = np.ones(self.rows, bool)
        for b, (_, m) in enumerate(self.plan):
            if b not in skip:
                left[self.offsets[b]:self.offsets[b] + m] = False
        assert (got[left] == 9).all() and (gl[left] == 9).all()
