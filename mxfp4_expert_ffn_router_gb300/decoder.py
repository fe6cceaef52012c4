"""One decoder layer of a routed-MoE model, decoding: the attention half over a paged
key-value cache, then the MoE half, for a batch of sequences with one new token each.

    a = x + residual;  h = norm(a)                        k3moe_rmsnorm
    q, k, v = h Wqkv                                      torch.matmul (a plain product)
    cache[slots] = k, v                                   k3moe_kv_write (quantised as it is written)
    o = attention of q over the cache                     k3moe_attn_decode
    a = a + o Wo;  h = norm(a)                            torch.matmul, k3moe_rmsnorm
    x' = sum over the routed experts of h                 k3moe_router, _bucket, _expert_ffn, _combine

``step`` returns (x', a): the next layer's norm adds them.  (The pages' engine has 96 attention
heads: "kimi-k3-in-c" overview, pomoai.com; every size is an argument here.)  Nothing in a step synchronises the host or
allocates, so a step can be captured in a CUDA graph: tables, lengths and slots are read on the device.  What makes room
for the new tokens does: ``PageTable`` keeps its lists on the host and copies the whole table for every ``append`` (1.0 ms for
64 sequences of up to 256 pages, 7.0 ms for 2048).  The attention chooses its way by the table's width, so a table
much wider than the sequences costs short ones 4 us a layer.

``python -m mxfp4_expert_ffn_router_gb300.decoder`` decodes a few tokens with random weights.
"""
from __future__ import annotations

from collections import Counter

import torch

from . import (K3MOE_FFN_AUTO, K3MOE_KV_E4M3, K3MOE_OP_BUCKET, K3MOE_OP_EXPERT_FFN, KVCache, Shape, Weights,
               k3moe_attn_decode, k3moe_attn_decode_workspace_bytes, k3moe_bucket, k3moe_combine, k3moe_expert_ffn,
               k3moe_kv_read, k3moe_kv_write, k3moe_rmsnorm, k3moe_router, k3moe_workspace_bytes)


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

    def slots_of(self, b: int) -> torch.Tensor:
        """The slots of all of sequence b's tokens, for k3moe_kv_read."""
        s = [self.owned[b][i // self.page_size] * self.page_size + i % self.page_size for i in range(self.lens[b])]
        return torch.tensor(s, dtype=torch.int32, device=self.table.device)

    def _upload(self):
        rows = [pg + [-1] * (self.max_pages - len(pg)) for pg in self.owned]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))
        self.seq_lens.copy_(torch.tensor(self.lens, dtype=torch.int32))


class DecoderLayer:
    """Weights (bf16 but for the MXFP4 experts): wqkv [(Hq + 2 heads) dim, H], wo [H, Hq dim],
    w_router [E, H], norm1 and norm2 [H].  ``shape``: T (the batch), H, I, E, k."""

    def __init__(self, shape, cache: KVCache, q_heads: int, wqkv, wo, w_router, norm1, norm2, experts: Weights,
                 eps: float = 1e-6, window: int = 0, mode: int = K3MOE_FFN_AUTO):
        s = self.s = Shape.of(shape)
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
        self.logits, self.idx, self.w = new(f32, s.T, s.E), new(i32, s.T, s.k), new(f32, s.T, s.k)
        self.counts, self.offsets, self.perm, self.inv = new(i32, s.E), new(i32, s.E + 1), new(i32, A), new(i32, A)
        self.ws_bucket = new(u8, max(1, k3moe_workspace_bytes(s, K3MOE_OP_BUCKET)))
        self.ws_ffn = new(u8, max(1, k3moe_workspace_bytes(s, K3MOE_OP_EXPERT_FFN, mode)))
        self.Y, self.out = new(f32, A, s.H), new(bf, s.T, s.H)

    def attention(self, x, residual, block_table, seq_lens, slots):
        """The attention half: (o Wo, a) of the new tokens x [T, H] (residual may be None)."""
        hq, hk = self.q_heads, self.cache.heads
        k3moe_rmsnorm(x, self.norm1, self.eps, residual=residual, residual_out=self.a, y=self.h)
        torch.matmul(self.h, self.wqkv.t(), out=self.qkv.view(self.s.T, -1))
        k3moe_kv_write(self.cache, self.qkv[:, hq:hq + hk], self.qkv[:, hq + hk:], slots, self.status)
        k3moe_attn_decode(self.cache, self.qkv[:, :hq], block_table, seq_lens, self.att, lse=self.lse,
                          window=self.window, ws=self.ws_attn, dev_status=self.status)
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

    def step(self, x, residual, block_table, seq_lens, slots):
        """One new token of each sequence through the layer: (x', a).  seq_lens counts the new
        tokens; slots (int32 [T]) are theirs, negative for an empty row of the batch."""
        return self.moe(*self.attention(x, residual, block_table, seq_lens, slots))


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
    layer = DecoderLayer(Shape(B, H, I, E, k), cache, hq, bf((hq + 2 * hk) * dim, H, scale=H ** -0.5),
                         bf(H, hq * dim, scale=H ** -0.5), bf(E, H, scale=H ** -0.5), bf(H, scale=0.1) + 1,
                         bf(H, scale=0.1) + 1, experts)
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


if __name__ == "__main__":
    main()
