"""One decoder layer of a routed-MoE model, decoding: the attention half over a paged
key-value cache, then the MoE half, for a batch of sequences with one new token each.

    a = x + residual;  h = norm(a)                        k3moe_rmsnorm
    q, k, v = h Wqkv                                      torch.matmul (a plain product)
    cache[slots] = k, v                                   k3moe_kv_write (quantised as it is written)
    o = attention of q over the cache                     k3moe_attn_decode
    a = a + o Wo;  h = norm(a)                            torch.matmul, k3moe_rmsnorm
    x' = sum over the routed experts of h                 k3moe_router, _bucket, _expert_ffn, _combine

``extend`` takes several new tokens of a sequence at once: a prompt's chunk, or a tree of drafted tokens to be
verified (``tree_masks``; ``accept`` keeps the ones that hold).  There, and wherever the layer has a rotation or sinks:

    cache[slots] = rotated k, v; q = rotated q            k3moe_kv_append
    o = attention of the new tokens over the cache        k3moe_attn_extend, k3moe_attn_tree

``step`` and ``extend`` return (x', a): the next layer's norm adds them.  (The pages' engine has 96 attention
heads: "kimi-k3-in-c" overview, pomoai.com; every size is an argument here.)  Nothing in a step synchronises the host or
allocates, so a step can be captured in a CUDA graph: tables, lengths and slots are read on the device.  What makes room
for the new tokens does: ``PageTable`` keeps its lists on the host and copies the whole table for every ``append`` (1.0 ms for
64 sequences of up to 256 pages, 7.0 ms for 2048).  The attention chooses its way by the table's width, so a table
much wider than the sequences costs short ones 4 us a layer.

``python -m mxfp4_expert_ffn_router_gb300.decoder`` decodes a few tokens with random weights, then verifies drafted ones.
"""
from __future__ import annotations

from collections import Counter

import torch

from . import (K3MOE_FFN_AUTO, K3MOE_KV_E4M3, K3MOE_OP_BUCKET, K3MOE_OP_EXPERT_FFN, KVCache, Rotation, Shape, Weights,
               k3moe_attn_decode, k3moe_attn_decode_workspace_bytes, k3moe_attn_extend, k3moe_attn_extend_workspace_bytes,
               k3moe_attn_tree, k3moe_bucket, k3moe_combine, k3moe_expert_ffn, k3moe_kv_append, k3moe_kv_read,
               k3moe_kv_write, k3moe_rmsnorm, k3moe_router, k3moe_workspace_bytes)


class PageTable:
    """Which pages of a cache a batch of sequences owns (kept on the host), and the
    device tensors that the calls read: table [batch, max_pages], seq_lens [batch] and the
    slots of the new tokens."""

    def __init__(self, batch: int, pages: int, page_size: int, max_pages: int, device="cuda"):
        self.page_size, self.max_pages = page_size, max_pages
        self.free = list(range(pages - 1, -1, -1))
        self.lens = [0] * batch
        self.owned = [[] for _ in range(batch)]
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def append(self, which, count: int = 1) -> torch.Tensor:
        """Make room for ``count`` new tokens of each sequence in ``which``; their slots, int32
        [len(which) * count], in order.  The lengths include them from here on.  RuntimeError where they do
        not all fit: then nothing has changed, and the call can be made again once pages have come back."""
        which = list(which)
        need = 0
        for b, times in Counter(which).items():
            pages = -(-(self.lens[b] + count * times) // self.page_size)
            if pages > self.max_pages:
                raise RuntimeError(f"sequence {b} would need {pages} pages of at most {self.max_pages}")
            need += pages - len(self.owned[b])
        if need > len(self.free):
            raise RuntimeError(f"no page left: {need} needed, {len(self.free)} free")
        slots = []
        for b in which:
            for _ in range(count):
                place = self.lens[b] % self.page_size
                if place == 0:
                    self.owned[b].append(self.free.pop())
                slots.append(self.owned[b][-1] * self.page_size + place)
                self.lens[b] += 1
        self._upload()
        return torch.tensor(slots, dtype=torch.int32, device=self.table.device)

    def release(self, b: int):
        """Give sequence b's pages back; its row of a batch is empty from here on."""
        self.free += reversed(self.owned[b])
        self.owned[b], self.lens[b] = [], 0
        self._upload()

    def truncate(self, b: int, count: int):
        """Forget the last ``count`` tokens of sequence b; pages that held only those come back."""
        if not 0 <= count <= self.lens[b]:
            raise ValueError(f"sequence {b} has {self.lens[b]} tokens, not {count} to forget")
        self.lens[b] -= count
        left = -(-self.lens[b] // self.page_size)
        self.free += reversed(self.owned[b][left:])
        del self.owned[b][left:]
        self._upload()

    def positions_of(self, which, count: int = 1) -> torch.Tensor:
        """Positions of the last ``count`` tokens of each sequence in ``which`` (int32), in the order of append's slots: of a
        sequence that is named more than once, the last tokens are its last naming's."""
        which = list(which)
        left = Counter(which)
        for b, times in left.items():
            if not 0 <= count * times <= self.lens[b]:
                raise ValueError(f"sequence {b} has {self.lens[b]} tokens, not {count * times}")
        at = []
        for b in which:
            first = self.lens[b] - count * left[b]
            left[b] -= 1
            at += range(first, first + count)
        return torch.tensor(at, dtype=torch.int32, device=self.table.device)

    def slots_of(self, b: int) -> torch.Tensor:
        """The slots of all of sequence b's tokens, for k3moe_kv_read."""
        s = [self.owned[b][i // self.page_size] * self.page_size + i % self.page_size for i in range(self.lens[b])]
        return torch.tensor(s, dtype=torch.int32, device=self.table.device)

    def _upload(self):
        rows = [pg + [-1] * (self.max_pages - len(pg)) for pg in self.owned]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))
        self.seq_lens.copy_(torch.tensor(self.lens, dtype=torch.int32))


def tree_masks(parents, device="cuda", window: int = 0, sinks: int = 0, lens=None):
    """Drafted trees as k3moe_attn_tree takes them.  ``parents``: for each sequence the parents of its drafted tokens, each
    an earlier one's index, or -1 for one that follows the sequence's last token.  Returns the masks int64 [rows, words] (a
    token sees its ancestors and itself), the q_offsets int32 [B + 1], and each row's depth (0: follows the last token),
    which is its position behind the context.

    ``window`` and ``sinks``: the layer's.  A decoded token sees no other that lies ``window`` or more positions before it, but for
    the first ``sinks``, drafted or not; the call drops cached ones alone, and a tree deeper than its window needs masks
    without the ancestors that are too far.  ``lens``: the tokens of each sequence before the drafted ones (with sinks: a
    drafted token at a position below them stays visible)."""
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks are at least 0")
    parents = list(parents)
    if window and sinks:
        if lens is None:
            raise ValueError("sinks: which drafted tokens they are goes by lens, the tokens before them")
        if len(lens := list(lens)) != len(parents):
            raise ValueError(f"lens: {len(lens)} sequences, not {len(parents)}")
    rows, depths, offsets = [], [], [0]
    for b, tree in enumerate(parents):
        first, kept = len(rows), sinks - lens[b] if window and sinks else 0  # depths below `kept` are first tokens
        line = []  # of each token its ancestors and itself, from the first on
        for i, p in enumerate(tree):
            if not -1 <= p < i:
                raise ValueError(f"the parent of drafted token {i} must be an earlier one or -1, not {p}")
            depths.append(depths[first + p] + 1 if p >= 0 else 0)
            if not window:
                rows.append((rows[first + p] if p >= 0 else 0) | 1 << i)
                continue
            line.append((line[p] if p >= 0 else []) + [i])
            rows.append(sum(1 << j for d, j in enumerate(line[i]) if d > depths[-1] - window or d < kept))
        offsets.append(len(rows))
    words = max(1, -(-max((len(t) for t in parents), default=0) // 64))
    parts = [[(r >> 64 * w) & (2 ** 64 - 1) for w in range(words)] for r in rows]
    signed = [[x - 2 ** 64 if x >> 63 else x for x in row] for row in parts]
    return (torch.tensor(signed, dtype=torch.int64, device=device).view(len(rows), words),
            torch.tensor(offsets, dtype=torch.int32, device=device), depths)


def accept(cache, pages: PageTable, b: int, count: int, kept, status=None):
    """Of sequence b's last ``count`` tokens, drafted ones, keep those at the ascending indices ``kept`` (a path of the
    tree, whose positions follow one another): their cached vectors move up to the first places, and the rest is
    forgotten.  ``cache``: the KVCache, or those of all layers that the pages are shared by (a second call would forget
    other tokens).  Reading an E4M3 vector back and writing it again gives the same values."""
    caches, kept = [cache] if isinstance(cache, KVCache) else list(cache), list(kept)
    if not 0 <= count <= pages.lens[b]:
        raise ValueError(f"sequence {b} has {pages.lens[b]} tokens, not {count} drafted ones")
    if kept != sorted(set(kept)) or (kept and not 0 <= kept[0] <= kept[-1] < count):
        raise ValueError(f"kept: ascending indices below {count}, not {kept}")
    if kept != list(range(len(kept))):
        slots = pages.slots_of(b)[pages.lens[b] - count:]
        come, go = slots[torch.tensor(kept, device=slots.device)], slots[:len(kept)].contiguous()
        for c in caches:
            kv = [torch.empty(len(kept), c.heads, c.dim, dtype=torch.bfloat16, device=slots.device) for _ in range(2)]
            k3moe_kv_read(c, come, *kv, status)
            k3moe_kv_write(c, *kv, go, status)
    pages.truncate(b, count - len(kept))


class DecoderLayer:
    """Weights (bf16 but for the MXFP4 experts): wqkv [(Hq + 2 heads) dim, H], wo [H, Hq dim],
    w_router [E, H], norm1 and norm2 [H].  ``shape``: T (the rows: a batch, or all of its
    new tokens), H, I, E, k.  ``rotation``: of the positions; ``sinks``: first tokens that stay visible beside a window."""

    def __init__(self, shape, cache: KVCache, q_heads: int, wqkv, wo, w_router, norm1, norm2, experts: Weights,
                 eps: float = 1e-6, window: int = 0, mode: int = K3MOE_FFN_AUTO, rotation: Rotation | None = None,
                 sinks: int = 0):
        s = self.s = Shape.of(shape)
        self.rotation, self.sinks = rotation, sinks
        self.cache, self.q_heads, self.eps, self.window, self.mode = cache, q_heads, eps, window, mode
        self.wqkv, self.wo, self.w_router, self.norm1, self.norm2, self.experts = wqkv, wo, w_router, norm1, norm2, experts
        dev, bf, f32, i32, u8 = wqkv.device, torch.bfloat16, torch.float32, torch.int32, torch.uint8
        A = s.T * s.k

        def new(dtype, *sizes):
            return torch.empty(sizes, dtype=dtype, device=dev)

        self.status = torch.zeros(1, dtype=i32, device=dev)
        self.h, self.a, self.a2, self.o = (new(bf, s.T, s.H) for _ in range(4))
        self.qkv = new(bf, s.T, q_heads + 2 * cache.heads, cache.dim)
        self.att, self.lse = new(bf, s.T, q_heads, cache.dim), new(f32, s.T, q_heads)
        self.ws_attn = new(u8, k3moe_attn_decode_workspace_bytes(cache, s.T, q_heads))
        self.ws_extend = []  # (the last is in use; smaller ones stay, since captured calls may hold them)
        self.one_each = torch.arange(s.T + 1, dtype=i32, device=dev)
        self.logits, self.idx, self.w = new(f32, s.T, s.E), new(i32, s.T, s.k), new(f32, s.T, s.k)
        self.counts, self.offsets, self.perm, self.inv = new(i32, s.E), new(i32, s.E + 1), new(i32, A), new(i32, A)
        self.ws_bucket = new(u8, max(1, k3moe_workspace_bytes(s, K3MOE_OP_BUCKET)))
        self.ws_ffn = new(u8, max(1, k3moe_workspace_bytes(s, K3MOE_OP_EXPERT_FFN, mode)))
        self.Y, self.out = new(f32, A, s.H), new(bf, s.T, s.H)

    def attention(self, x, residual, block_table, seq_lens, slots, positions=None, q_offsets=None, masks=None,
                  max_new=None):
        """The attention half: (o Wo, a) of the new tokens x [T, H] (residual may be None); with q_offsets several of a
        sequence, as in ``extend``."""
        hq, hk = self.q_heads, self.cache.heads
        if (self.rotation is None) != (positions is None):
            raise ValueError("positions belong to a layer with a rotation, and to each of its calls")
        if masks is not None and q_offsets is None:
            raise ValueError("masks: drafted tokens need q_offsets")
        every_row = q_offsets is None  # (is a sequence's)
        if every_row and self.sinks:
            q_offsets, max_new = self.one_each, 1
        k3moe_rmsnorm(x, self.norm1, self.eps, residual=residual, residual_out=self.a, y=self.h)
        torch.matmul(self.h, self.wqkv.t(), out=self.qkv.view(self.s.T, -1))
        q, k, v = self.qkv[:, :hq], self.qkv[:, hq:hq + hk], self.qkv[:, hq + hk:]
        if self.rotation is None:
            k3moe_kv_write(self.cache, k, v, slots, self.status)
        else:
            k3moe_kv_append(self.cache, k, v, slots, positions, self.rotation, q=q, q_out=q, dev_status=self.status)
        if q_offsets is None:
            k3moe_attn_decode(self.cache, q, block_table, seq_lens, self.att, lse=self.lse, window=self.window,
                              ws=self.ws_attn, dev_status=self.status)
        else:
            need = k3moe_attn_extend_workspace_bytes(self.cache, len(seq_lens), self.s.T, hq)
            if not self.ws_extend or self.ws_extend[-1].numel() < need:
                self.ws_extend.append(torch.empty(need, dtype=torch.uint8, device=x.device))
            if not every_row:  # rows of no sequence keep what is there, which must not be an earlier call's (8192 rows of 64
                #                heads of 128: 37 us, beside 860 for their attention)
                self.att.zero_()
            rest = dict(lse=self.lse, window=self.window, sinks=self.sinks, ws=self.ws_extend[-1], dev_status=self.status)
            if masks is None:
                k3moe_attn_extend(self.cache, q, q_offsets, block_table, seq_lens, self.att, max_new=max_new, **rest)
            else:
                k3moe_attn_tree(self.cache, q, q_offsets, masks, block_table, seq_lens, self.att, **rest)
        torch.matmul(self.att.view(self.s.T, -1), self.wo.t(), out=self.o)
        return self.o, self.a

    def moe(self, x, residual):
        """The MoE half: (the routed experts' sum, a) for x, residual [T, H]."""
        s = self.s
        k3moe_rmsnorm(x, self.norm2, self.eps, residual=residual, residual_out=self.a2, y=self.h)
        k3moe_router(s, self.h, self.w_router, self.logits, self.idx, self.w, self.status)
        k3moe_bucket(s, self.idx, self.counts, self.offsets, self.perm, self.inv, self.ws_bucket, self.status)
        k3moe_expert_ffn(s, self.h, self.experts, self.offsets, self.perm, self.Y, self.mode, self.ws_ffn, self.status)
        k3moe_combine(s, self.Y, self.w, self.inv, self.out)
        return self.out, self.a2

    def step(self, x, residual, block_table, seq_lens, slots, positions=None):
        """One new token of each sequence through the layer: (x', a).  seq_lens counts the new
        tokens; slots (int32 [T]) are theirs, negative for an empty row of the batch (its sequence has length
        0); positions (int32 [T]) where the layer has a rotation."""
        return self.moe(*self.attention(x, residual, block_table, seq_lens, slots, positions))

    def extend(self, x, residual, block_table, seq_lens, slots, q_offsets, positions=None, masks=None, max_new=None):
        """Several new tokens of each sequence through the layer: (x', a).  Rows q_offsets[b] .. q_offsets[b + 1] - 1
        (int32 [B + 1]) of x [T, H] are sequence b's, which seq_lens counts; slots (int32 [T]) are theirs, negative for
        rows of no sequence (whose attention is 0).  With masks (``tree_masks``, which takes the layer's window and sinks:
        without them a token sees ancestors beyond its window, and scores as it would not be decoded) they are a drafted
        tree's.  The workspace is made for the largest batch so far: a call that is captured comes after one like it, so that it
        allocates nothing.  max_new: no sequence has more new tokens (without it the host has to expect all rows of one)."""
        return self.moe(*self.attention(x, residual, block_table, seq_lens, slots, positions, q_offsets, masks, max_new))


def main(tokens: int = 8):
    """A batch of three sequences decodes ``tokens`` tokens through one small layer; the
    cached prefix is read back once."""
    torch.manual_seed(0)
    B, H, I, E, k, hq, hk, dim, page = 3, 1024, 512, 8, 2, 16, 4, 64, 16
    dev = torch.device("cuda")

    def bf(*sizes, scale=1.0):
        return (torch.randn(*sizes, device=dev) * scale).bfloat16()

    def codes(*sizes, lo=0, hi=256):
        return torch.randint(lo, hi, sizes, dtype=torch.uint8, device=dev)

    experts = Weights.from_stacked(codes(E, 2 * I, H // 2), codes(E, 2 * I, H // 32, lo=119, hi=124),
                                   codes(E, H, I // 2), codes(E, H, I // 32, lo=119, hi=124))
    cache = KVCache.empty(32, hk, page, dim, K3MOE_KV_E4M3, dev)
    weights = (bf((hq + 2 * hk) * dim, H, scale=H ** -0.5), bf(H, hq * dim, scale=H ** -0.5), bf(E, H, scale=H ** -0.5),
               bf(H, scale=0.1) + 1, bf(H, scale=0.1) + 1, experts)
    layer = DecoderLayer(Shape(B, H, I, E, k), cache, hq, *weights)
    pages = PageTable(B, cache.pages, page, 8, dev)
    x, a = bf(B, H), None
    for t in range(tokens):
        slots = pages.append(range(B))
        x, a = layer.step(x, a, pages.table, pages.seq_lens, slots)
        x, a = x.clone(), a.clone()
        print(f"token {t}: |x| rms {x.float().pow(2).mean().sqrt():.4f}, longest {max(pages.lens)}")
    prefix = pages.slots_of(0)
    kv = [torch.empty(len(prefix), hk, dim, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    k3moe_kv_read(cache, prefix, *kv, layer.status)
    print(f"read back {len(prefix)} tokens of sequence 0; device status {int(layer.status.item())}")
    # drafted tokens of every sequence, verified in one call; of each tree one path is kept
    tree, path = [-1, 0, 0, 1, 2], [0, 2, 4]
    masks, offsets, depths = tree_masks([tree] * B, dev)
    verify = DecoderLayer(Shape(B * len(tree), H, I, E, k), cache, hq, *weights)
    slots = pages.append(range(B), len(tree))
    x, a = verify.extend(bf(B * len(tree), H), None, pages.table, pages.seq_lens, slots, offsets, masks=masks)
    for b in range(B):
        accept(cache, pages, b, len(tree), path, verify.status)
    print(f"verified {len(tree)} drafted tokens a sequence, kept {len(path)}; longest {max(pages.lens)}, "
          f"device status {int(verify.status.item())}")


if __name__ == "__main__":
    main()
