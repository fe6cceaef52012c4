"""Cases of the operators by which a decoder layer takes several new tokens of a
sequence at once (a prompt, or drafted tokens to be verified) over the paged cache: the keys
and values appended to it with the rotation of their positions, attention with a
sliding window and a few first tokens that stay visible, and attention of a tree of
drafted tokens.

With ``own`` false, ``run`` computes an operator from elementary torch operations
in fp32 (angles in 64 bits), rounded once at the end; with ``own`` true it calls the
framework.

A sequence with n cached tokens, the m newest of which are the new ones, has its new
token i at place n - m + i.  Cached data in 8 bits is E4M3 codes with a power-of-two
(E8M0) scale per (token, head) vector: the smallest power of two X with max|v| <= 448 X.
"""
import math
import random

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step: a new token for each of 13 sequences, 96 separate heads, some rows padding: latency
        dict(name="append_step_8bit", op="append", n=13, Hq=96, Hkv=96, dim=128, page=64, fmt="e4m3", rot=128,
             neighbours=False, start=5000, pad=3),
        # a prompt's chunk of 4096 tokens far into a long conversation, grouped heads
        dict(name="append_prompt_8bit", op="append", n=4096, Hq=64, Hkv=8, dim=128, page=64, fmt="e4m3", rot=128,
             neighbours=False, start=1000000, pad=0),
        # an odd number of tokens, a part of each head rotated in neighbouring pairs, an unquantised cache
        dict(name="append_odd_bf16", op="append", n=777, Hq=15, Hkv=5, dim=64, page=16, fmt="bf16", rot=32,
             neighbours=True, start=0, pad=100),
        # one new token of one conversation, 96 separate heads, past its window: latency
        dict(name="sinks_one_8bit", op="sinks", B=1, new=1, ctx=700, Hq=96, Hkv=96, dim=128, page=64, fmt="e4m3",
             window=500, sinks=4, ragged=False, pad=0, plan=1),
        # a serving batch of very different lengths, one new token each, one slot of it empty
        dict(name="sinks_step_8bit", op="sinks", B=64, new=1, ctx=16384, Hq=64, Hkv=8, dim=128, page=64, fmt="e4m3",
             window=4096, sinks=4, ragged=True, pad=0, plan=2),
        # one prompt of 8192 tokens: the most products
        dict(name="sinks_prompt_bf16", op="sinks", B=1, new=8192, ctx=0, Hq=64, Hkv=8, dim=128, page=64, fmt="bf16",
             window=4096, sinks=4, ragged=False, pad=0, plan=3),
        # chunks of prompts of very different lengths over their histories, the batch padded
        dict(name="sinks_chunks_8bit", op="sinks", B=6, new=1000, ctx=12000, Hq=32, Hkv=4, dim=128, page=16,
             fmt="e4m3", window=3001, sinks=20, ragged=True, pad=77, plan=4),
        # many short prompts that share one key head of 64
        dict(name="sinks_short_bf16", op="sinks", B=24, new=301, ctx=0, Hq=16, Hkv=1, dim=64, page=32, fmt="bf16",
             window=0, sinks=0, ragged=True, pad=0, plan=5),
        # eight drafted tokens of one conversation, 96 separate heads: latency
        dict(name="tree_one_8bit", op="tree", B=1, new=8, ctx=500, Hq=96, Hkv=96, dim=128, page=64, fmt="e4m3",
             window=0, sinks=0, ragged=False, pad=0, plan=6),
        # a serving batch, trees of up to 64 drafted tokens
        dict(name="tree_batch_8bit", op="tree", B=16, new=64, ctx=16384, Hq=64, Hkv=8, dim=128, page=64, fmt="e4m3",
             window=0, sinks=0, ragged=True, pad=9, plan=7),
        # one conversation with a long history
        dict(name="tree_long_8bit", op="tree", B=1, new=60, ctx=131072, Hq=64, Hkv=8, dim=128, page=128, fmt="e4m3",
             window=0, sinks=0, ragged=False, pad=0, plan=8),
        # wide heads, an unquantised cache, a window with sinks, odd sizes
        dict(name="tree_window_bf16", op="tree", B=7, new=13, ctx=5003, Hq=20, Hkv=4, dim=256, page=32, fmt="bf16",
             window=2000, sinks=5, ragged=True, pad=0, plan=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "sinks", "sinks", "tree", "tree"])
    fmt, dim, page = rng.choice(["e4m3", "e4m3", "bf16"]), rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 5, 8, 8, 96])
    group = rng.choice([1, 3, 4, 5, 8, 12, 16]) if heads < 96 else 1
    if op == "append":
        n = _log_int(rng, 1, min(8192, (1 << 25) // (heads * (group + 2) * dim)))
        return dict(op=op, n=n, Hq=heads * group, Hkv=heads, dim=dim, page=page, fmt=fmt,
                    rot=rng.choice([dim, dim, dim // 2, 48]), neighbours=rng.random() < 0.3,
                    start=_log_int(rng, 1, 1 << 21) - 1, pad=rng.choice([0, 0, n // 7]))
    batch = _log_int(rng, 1, 64)
    tokens = rng.random()
    new = 1 if op == "sinks" and tokens < 0.3 else _log_int(rng, 2, 8192 if op == "sinks" and tokens < 0.6 else 100)
    # as many scores as the largest listed case at most, and no more cached bytes than 1 GB
    new = max(1, min(new, int(math.sqrt(4_000_000_000 / (batch * heads * group)))))
    cached = min(131072, 4_000_000_000 // (batch * heads * group * new),
                 1_000_000_000 // (batch * 2 * heads * dim * (1 if fmt == "e4m3" else 2)))
    ctx = _log_int(rng, 1, max(1, cached - new + 1)) - 1
    window = rng.choice([0, _log_int(rng, 1, ctx + new)])
    return dict(op=op, B=batch, new=new, ctx=ctx, Hq=heads * group, Hkv=heads, dim=dim, page=page, fmt=fmt, window=window,
                sinks=rng.choice([0, 4, _log_int(rng, 1, 300)]) if window else 0, ragged=rng.random() < 0.7,
                pad=rng.choice([0, 0, 11]), plan=rng.randrange(1 << 30))


def _plan(case):
    """(cached tokens before the new ones, new ones) of each sequence: all alike, or spread with the longest
    first and, in a batch of three or more, an empty slot last."""
    B, ctx, new = case["B"], case["ctx"], case["new"]
    if not case["ragged"]:
        return [(ctx, new)] * B
    rng = random.Random(case["plan"])
    rows = [(ctx, new)] + [(_log_int(rng, max(1, ctx // 64), ctx + 1) - 1, _log_int(rng, max(1, new // 16), new))
                           for _ in range(B - 1)]
    if B > 2:
        rows[-1] = (0, 0)
    return rows


def _parents(case, b, m):
    """A drafted tree's parents (-1: the sequence's last cached token), each before its children."""
    rng = random.Random(case["plan"] * 1009 + b)
    return [rng.randrange(max(-1, i - 9), i) for i in range(m)]


def _seen_before(case, place):
    """How many cached places below `place` a token there sees, without itself."""
    w = case["window"]
    return place if not w or place < w else w - 1 + min(case["sinks"], place - w + 1)


def work(case):
    vec = case["dim"] + 1 if case["fmt"] == "e4m3" else 2 * case["dim"]  # bytes of a cached vector
    if case["op"] == "append":
        live = case["n"] - case["pad"]
        return {"bytes": live * (2 * case["Hkv"] * (vec + 2 * case["dim"]) + 4 * case["Hq"] * case["dim"]) + 8 * case["n"],
                "flops": 3 * live * (case["Hq"] + case["Hkv"]) * case["rot"]}
    read = pairs = rows = 0
    for b, (ctx, m) in enumerate(_plan(case)):
        rows += m
        if not m:
            continue
        w = case["window"]
        low = max(0, ctx - w + 1) if w else 0  # the first place that the window of the first new token holds
        read += ctx + m - low + min(low, case["sinks"])
        if case["op"] == "sinks":
            pairs += sum(_seen_before(case, ctx + i) + 1 for i in range(m))
        else:
            depth = []
            for p in _parents(case, b, m):
                depth.append(depth[p] + 1 if p >= 0 else 0)
                # of the cached tokens what the window from its position on holds, and its ancestors and itself
                lo = max(0, ctx + depth[-1] - w + 1) if w else 0
                pairs += max(0, ctx - lo) + min(lo, ctx, case["sinks"]) + depth[-1] + 1
    return {"bytes": read * case["Hkv"] * 2 * vec + rows * case["Hq"] * (4 * case["dim"] + 4),
            "flops": 4 * pairs * case["Hq"] * case["dim"]}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cached(g, pages, heads, page, dim, fmt):
    """Cache contents (values and scales, or None): normal values, channels of different size."""
    chan = torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g, device="cuda"))
    x = _normal(g, pages, heads, page, dim).mul_(chan.bfloat16())
    if fmt == "bf16":
        return x, None
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[:-1], dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // max(1, heads * page * dim))
    for p in range(0, pages, step):
        codes[p:p + step], scales[p:p + step] = _quant(x[p:p + step].float())
    return codes, scales


def _forget(s, where):
    """What lies in cache places that hold no token: anything, here NaN."""
    for values, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        if scales is None:
            values[where] = float("nan")
        else:
            values[where] = 0x7F
            scales[where] = 255


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    rng = random.Random(seed)
    page, dim, Hq, Hkv = case["page"], case["dim"], case["Hq"], case["Hkv"]
    if case["op"] == "append":
        n = case["n"]
        pages = -(-n // page) + 2
        order = rng.sample(range(pages), pages)
        if n < 2 * page:  # tokens of a step: anywhere, each at its own position
            slots = rng.sample(range(pages * page), n)
            at = [case["start"] + rng.randrange(4096) for _ in range(n)]
        else:  # consecutive tokens: page after page of a shuffled list
            slots = [order[i // page] * page + i % page for i in range(n)]
            at = [case["start"] + i for i in range(n)]
        for i in rng.sample(range(n), case["pad"]):
            slots[i] = -1
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
        s["positions"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        s["inv_freq"] = 500000.0 ** (torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / -case["rot"])
        s["k"], s["ks"] = _cached(g, pages, Hkv, page, dim, case["fmt"])
        s["v"], s["vs"] = _cached(g, pages, Hkv, page, dim, case["fmt"])
        qkv = _normal(g, n, Hq + 2 * Hkv, dim)  # a fused projection
        s["q_new"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.zeros(n, Hq, dim, dtype=torch.bfloat16, device="cuda")
    else:
        plan, B = _plan(case), case["B"]
        lens = [c + m for c, m in plan]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        order = rng.sample(range(pages), pages)
        table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32)
        s["k"], s["ks"] = _cached(g, pages, Hkv, page, dim, case["fmt"])
        s["v"], s["vs"] = _cached(g, pages, Hkv, page, dim, case["fmt"])
        at = 0
        for b in range(B):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
            if lens[b] % page:
                _forget(s, (mine[-1], slice(None), slice(lens[b] % page, None)))
        _forget(s, torch.tensor(order[at:], device="cuda"))
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        offsets = [0]
        for _, m in plan:
            offsets.append(offsets[-1] + m)
        rows = s["rows"] = offsets[-1] + case["pad"]
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        if case["op"] == "tree":
            words = -(-case["new"] // 64)
            masks = []
            for b, (_, m) in enumerate(plan):
                bits = []
                for i, p in enumerate(_parents(case, b, m)):
                    bits.append((bits[p] if p >= 0 else 0) | 1 << i)
                masks += bits
            masks += [0] * case["pad"]
            parts = [[(x >> 64 * w) & (2 ** 64 - 1) for w in range(words)] for x in masks]
            signed = [[x - 2 ** 64 if x >> 63 else x for x in row] for row in parts]
            s["masks"] = torch.tensor(signed, dtype=torch.int64, device="cuda").view(rows, words)
        s["q"] = _normal(g, rows, Hq + 2 * Hkv, dim)[:, :Hq]  # the query heads of a fused projection
        s["out"] = torch.zeros(rows, Hq, dim, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device="cuda")
    if own:
        import mxfp4_expert_ffn_router_gb300 as k3
        s["cache"] = k3.KVCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "append":
            s["rotation"] = k3.Rotation(case["rot"], inv_freq=s["inv_freq"], neighbours=case["neighbours"])
        else:
            s["ws"] = torch.empty(k3.k3moe_attn_extend_workspace_bytes(s["cache"], case["B"], s["rows"], Hq),
                                  dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _cache_out(s):
    out = {"q": s["q_out"]}
    if s["ks"] is None:
        return dict(out, k=s["k"], v=s["v"])
    return dict(out, k=s["k"].view(E4M3), k_scales=s["ks"].view(E8M0), v=s["v"].view(E4M3), v_scales=s["vs"].view(E8M0))


def _run_own(s):
    import mxfp4_expert_ffn_router_gb300 as k3
    if s["op"] == "append":
        k3.k3moe_kv_append(s["cache"], s["k_new"], s["v_new"], s["slots"], s["positions"], s["rotation"], q=s["q_new"],
                           q_out=s["q_out"])
        return _cache_out(s)
    if s["op"] == "sinks":
        k3.k3moe_attn_extend(s["cache"], s["q"], s["offsets"], s["table"], s["lens"], s["out"], lse=s["lse"],
                             window=s["window"], sinks=s["sinks"], max_new=s["new"], ws=s["ws"])
    else:
        k3.k3moe_attn_tree(s["cache"], s["q"], s["offsets"], s["masks"], s["table"], s["lens"], s["out"], lse=s["lse"],
                           window=s["window"], sinks=s["sinks"], ws=s["ws"])
    return s["out"], s["lse"]


def _pow2(e):
    """2^e in fp32 for whole numbers -126 .. 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quant(x):
    """E4M3 codes of x (fp32) and the E8M0 bytes of the scales of its last axis."""
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    m, ex = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))  # amax = m 2^ex, m in [0.5, 1)
    e = (ex - 9 + (m > 0.875).int()).clamp(-127, 127)  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    half = torch.div(-e, 2, rounding_mode="floor")  # in two steps: 2^-127 is no normal fp32 value
    codes = (x * _pow2(half)[..., None] * _pow2(-e - half)[..., None]).to(E4M3).view(torch.uint8)
    codes = torch.where(bad[..., None], torch.full_like(codes, 0x7F), codes)
    return codes, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _values(values, scales):
    return values.float() if scales is None else values.view(E4M3).float() * scales.view(E8M0).float()[..., None]


def _rotated(x, cos, sin, rot, neighbours):
    """x [n, heads, dim] in fp32 with its first `rot` dimensions turned, cos and sin [n, 1, rot / 2]."""
    head, rest = x[..., :rot], x[..., rot:]
    if neighbours:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _run_plain(s):
    page, dim, Hq, Hkv = s["page"], s["dim"], s["Hq"], s["Hkv"]
    if s["op"] == "append":
        angle = s["positions"].double()[:, None] * s["inv_freq"]
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        q = _rotated(s["q_new"].float(), cos, sin, s["rot"], s["neighbours"])
        k = _rotated(s["k_new"].float(), cos, sin, s["rot"], s["neighbours"])
        slots = s["slots"].long()
        live = slots >= 0
        s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"].float()))
        pg, at = slots[live] // page, slots[live] % page
        if s["ks"] is None:
            s["k"][pg, :, at], s["v"][pg, :, at] = k[live].bfloat16(), s["v_new"][live]
        else:
            s["k"][pg, :, at], s["ks"][pg, :, at] = _quant(k[live])
            s["v"][pg, :, at], s["vs"][pg, :, at] = _quant(s["v_new"][live].float())
        return _cache_out(s)
    B, G, M = s["B"], Hq // Hkv, s["new"]
    pg = s["table"].clamp(min=0).long()

    def gathered(values, scales):  # [B, Hkv, places, dim]
        x = _values(values[pg], None if scales is None else scales[pg])
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, dim)

    k, v = gathered(s["k"], s["ks"]), gathered(s["v"], s["vs"])
    t = torch.arange(k.shape[2], device=k.device)
    v = torch.where((t < s["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    # the new tokens of all sequences, padded to M each
    i = torch.arange(M, device=k.device)
    count = s["offsets"][1:] - s["offsets"][:-1]
    there = i < count[:, None]  # [B, M]
    row = torch.where(there, s["offsets"][:-1, None] + i, torch.zeros_like(there, dtype=torch.int32)).long()
    ctx = (s["lens"] - count)[:, None, None]
    if s["op"] == "sinks":
        place = ctx + i[:, None]  # [B, M, 1]
        seen = t <= place
        new = torch.zeros_like(seen)
    else:
        bits = torch.arange(64, device=k.device)
        seen_new = ((s["masks"][row][..., None] >> bits) & 1).flatten(-2) != 0  # [B, M, 64 words]
        place = ctx + seen_new.sum(-1, keepdim=True) - 1
        j = (t - ctx).expand(B, M, -1)  # which of the drafted tokens a place holds
        new = (j >= 0) & (j < count[:, None, None])
        seen = torch.where(new, torch.gather(seen_new, 2, j.clamp(0, seen_new.shape[2] - 1)), j < 0)
    if s["window"]:
        seen = seen & ((t > place - s["window"]) | (t < s["sinks"]) | new)
    seen = (seen & there[..., None])[:, None, :, None, :]  # [B, 1, M, 1, places]
    q = s["q"][row].float().view(B, M, Hkv, G, dim).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, dim)
    scores = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, M, G, -1) * (1 / math.sqrt(dim))
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    del scores
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, M * G, -1), v).view(B, Hkv, M, G, dim)
    o = torch.where(total == 0, torch.zeros_like(o), o / total).permute(0, 2, 1, 3, 4).reshape(B, M, Hq, dim)
    lse = (m + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(B, M, Hq)
    s["out"][row[there]] = o[there].bfloat16()
    s["lse"][row[there]] = lse[there]
    return s["out"], s["lse"]


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_pow2(e):
    """2^e in 64 bits for whole numbers -1022 .. 1023, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x):
    """Values and scales (64 bits) that E4M3 codes and E8M0 scales of x's last axis stand for."""
    amax = x.abs().amax(-1, keepdim=True)
    scale = _exact_pow2(torch.ceil(torch.log2(amax / 448)).clamp(-127, 127))  # amax = 0: log2 = -inf
    a = x / scale
    step = _exact_pow2(torch.floor(torch.log2(a.abs())).clamp(min=-6) - 3)  # spacing of the values near a
    return torch.round(a / step) * step, scale[..., 0]


def _exact_values(values, scales):
    """What a cache holds, in 64 bits, from its bits."""
    if scales is None:
        return values.double()
    b = values.long()
    ex, mant = (b >> 3) & 15, (b & 7).double()
    size = torch.where(ex == 0, mant / 512, (1 + mant / 8) * _exact_pow2(ex - 7))
    size = torch.where((b & 127) == 127, torch.full_like(size, math.nan), size)
    scale = _exact_pow2(scales.long() - 127)
    scale = torch.where(scales == 255, torch.full_like(scale, math.nan), scale)
    return torch.where(b >= 128, -size, size) * scale[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    page, dim, Hq, Hkv = case["page"], case["dim"], case["Hq"], case["Hkv"]
    if case["op"] == "append":
        # a pair of dimensions as a complex number, times e^(i angle)
        half = case["rot"] // 2
        turn = torch.polar(torch.ones_like(s["inv_freq"]), s["inv_freq"] * s["positions"].double()[:, None])[:, None]

        def turned(x):
            x = x.double().clone()
            first = slice(0, case["rot"], 2) if case["neighbours"] else slice(0, half)
            second = slice(1, case["rot"], 2) if case["neighbours"] else slice(half, 2 * half)
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        slots = s["slots"].long()[live]
        pg, at = slots // page, slots % page
        q = torch.zeros(case["n"], Hq, dim, dtype=torch.float64, device="cuda")
        q[live] = turned(s["q_new"])[live]
        out = {"q": q}
        for name, values, scales, new in (("k", s["k"], s["ks"], turned(s["k_new"])),
                                          ("v", s["v"], s["vs"], s["v_new"].double())):
            if scales is None:
                full = values.double()
                full[pg, :, at] = new[live]
            else:
                full = _exact_values(values, torch.full_like(scales, 127))
                unit = _exact_pow2(scales.long() - 127)
                full[pg, :, at], unit[pg, :, at] = _exact_quant(new[live])
            out[name] = full
            if scales is not None:
                out[name + "_scales"] = unit
        return out
    out = torch.zeros(s["rows"], Hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["rows"], Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (ctx, m) in enumerate(_plan(case)):
        if not m:
            continue
        n = ctx + m
        mine = s["table"][b, :-(-n // page)].long()
        hide = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if case["op"] == "sinks":
            position = ctx + torch.arange(m, device="cuda")
            hide |= torch.arange(n, device="cuda") > position[:, None]
            far = hide.new_ones(n)
        else:
            kin = torch.zeros(m, m, dtype=torch.bool)
            for i, p in enumerate(_parents(case, b, m)):
                if p >= 0:
                    kin[i] = kin[p]
                kin[i, i] = True
            hide[:, ctx:] = ~kin.cuda()
            position = ctx + kin.sum(-1).cuda() - 1
            far = torch.arange(n, device="cuda") < ctx
        if case["window"]:
            gone = torch.arange(n, device="cuda") <= position[:, None] - case["window"]
            gone[:, :case["sinks"]] = False
            hide |= gone & far
        for h in range(Hkv):
            k, v = (_exact_values(x[mine, h], None if y is None else y[mine, h]).reshape(-1, dim)[:n]
                    for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                scores = s["q"][at:at + m, g].double() @ k.T / math.sqrt(dim)
                scores[hide] = -math.inf
                lse[at:at + m, g] = torch.logsumexp(scores, -1)
                out[at:at + m, g] = torch.softmax(scores, -1) @ v
        at += m
    return out, lse
