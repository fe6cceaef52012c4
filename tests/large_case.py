"""Larger calls of k3moe_attn_extend and k3moe_attn_tree than float64 references are made for: caches filled on the device, calls
compared with one another bit for bit, and their times."""
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import E4, i32
from mxfp4_expert_ffn_router_gb300.decoder import tree_masks


class LargeCase:
    """``plan``: (places before the new tokens, new tokens) of each sequence, whose pages follow one another;
    ``width``: of the table, in pages; ``tree``: chains of drafted tokens, by masks."""

    def __init__(self, plan, Hq, heads, dim, page, fmt, width=None, tree=False, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.plan, self.page, self.fmt, self.dim = list(plan), page, fmt, dim
        lens = [c + m for c, m in plan]
        need = [-(-n // page) for n in lens]
        shape = (sum(need) + 1, heads, page, dim)
        if fmt == E4:  # (codes of at most 30; scales that bring them to about 1)
            k, v = (torch.randint(0, 0x60, shape, dtype=torch.uint8, device="cuda", generator=g) |
                    torch.randint(0, 2, shape, dtype=torch.uint8, device="cuda", generator=g) << 7 for _ in range(2))
            self.cache = k3.KVCache(k, v, *(torch.full(shape[:-1], 124, dtype=torch.uint8, device="cuda") for _ in range(2)))
        else:
            self.cache = k3.KVCache(*(torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=g) for _ in range(2)))
        table = torch.full((len(plan), width or max(need)), -1, dtype=torch.int32)
        at, offsets = 0, [0]
        for b, n in enumerate(need):
            table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
            at += n
            offsets.append(offsets[-1] + plan[b][1])
        self.table, self.lens, self.offsets, self.rows = table.cuda(), i32(lens), i32(offsets), offsets[-1]
        self.first_page = [sum(need[:b]) for b in range(len(plan))]
        self.q = torch.randn(self.rows, Hq, dim, dtype=torch.bfloat16, device="cuda", generator=g)
        self.masks = tree_masks([list(range(-1, m - 1)) for _, m in plan])[0] if tree else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(k3.k3moe_attn_extend_workspace_bytes(self.cache, len(plan), self.rows, Hq), dtype=torch.uint8,
                              device="cuda")
        self.out = torch.empty(self.rows, Hq, dim, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(self.rows, Hq, dtype=torch.float32, device="cuda")

    def place(self, b, p):
        """Page and place in it of sequence b's place p."""
        return self.first_page[b] + p // self.page, p % self.page

    def call(self, masks=None, **kw):
        args = dict(lse=self.lse, ws=self.ws, dev_status=self.status) | kw
        masks = self.masks if masks is None else masks
        if masks is None:
            k3.k3moe_attn_extend(self.cache, self.q, self.offsets, self.table, self.lens, self.out, **args)
        else:
            k3.k3moe_attn_tree(self.cache, self.q, self.offsets, masks, self.table, self.lens, self.out, **args)

    def run(self, **kw):
        self.out.fill_(9), self.lse.fill_(9)
        self.call(**kw)
        return self.out.clone(), self.lse.clone()

    def us(self, calls=7, **kw):
        """The median of a call's times."""
        times = []
        for _ in range(calls + 2):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            self.call(**kw)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times[2:])[calls // 2]
