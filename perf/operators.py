"""Cases of the decoder layer's operators beside the MoE path: RMS norm with the
residual's addition and an 8-bit output, the paged key-value cache (quantised as
it is written, read back), and attention of one new token over that cache.

With ``own`` false, ``run`` computes an operator from elementary torch operations
in fp32, rounded once at the end; with ``own`` true it calls the framework.

8-bit data is E4M3 codes with power-of-two (E8M0) scales: per 32 values of a row
for the norm's output, per (token, head) vector for the cache.  The scale is the
smallest power of two X with max|v| <= 448 X (exponent clamped to -127 .. 127; an
all-zero group has exponent -127); a group holding a NaN or an infinity has the
scale NaN (byte 255) and codes 0x7F.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---------------------------------------------------------------- cases
def listed():
    return [
        # RMS norm: one new token of the repository's decode layer (H = 7168): latency
        dict(name="norm_one_token", op="norm", T=1, H=7168, residual=True, y=True, y8=False),
        # a small ragged decode batch whose output feeds an 8-bit product
        dict(name="norm_batch_8bit", op="norm", T=37, H=7168, residual=True, y=False, y8=True),
        # a prefill chunk (4096 tokens), bf16 and 8-bit outputs
        dict(name="norm_prefill_both", op="norm", T=4096, H=7168, residual=True, y=True, y8=True),
        # cache write of one decode step: a new token for each of 13 sequences, 96 heads of 128
        # (24,576 cached values a position), slots scattered over the pages, some of them padding
        dict(name="write_step_8bit", op="write", n=13, heads=96, dim=128, page=64, fmt="e4m3", fused=True, pad=3),
        # cache write of a prefill chunk, grouped heads, k and v slices of a fused projection
        dict(name="write_prefill_8bit", op="write", n=4096, heads=8, dim=128, page=64, fmt="e4m3", fused=True, pad=0),
        # reading a prefix back for a following chunk
        dict(name="read_prefix_8bit", op="read", n=16384, heads=8, dim=128, page=64, fmt="e4m3", pad=0),
        # an odd number of tokens from an unquantised cache of small heads, padded to a fixed length
        dict(name="read_odd_bf16", op="read", n=777, heads=5, dim=64, page=16, fmt="bf16", pad=100),
        # attention: the first tokens of one conversation, 96 heads: latency
        dict(name="attn_one_short", op="attn", B=1, Hq=96, Hkv=96, dim=128, page=64, fmt="e4m3", max_len=37,
             ragged=False, window=0, lens_seed=1),
        # a serving batch of very different lengths, one slot of it empty, grouped heads
        dict(name="attn_batch_gqa_8bit", op="attn", B=64, Hq=64, Hkv=8, dim=128, page=64, fmt="e4m3", max_len=16384,
             ragged=True, window=0, lens_seed=2),
        # one conversation with a long history
        dict(name="attn_long_one_8bit", op="attn", B=1, Hq=64, Hkv=8, dim=128, page=128, fmt="e4m3", max_len=131072,
             ragged=False, window=0, lens_seed=3),
        # 96 separate heads over an unquantised cache in small pages: the most bytes
        dict(name="attn_batch_mha_bf16", op="attn", B=32, Hq=96, Hkv=96, dim=128, page=16, fmt="bf16", max_len=4001,
             ragged=True, window=0, lens_seed=4),
        # shared single head with a sliding window, odd lengths
        dict(name="attn_window_mqa_bf16", op="attn", B=48, Hq=16, Hkv=1, dim=64, page=32, fmt="bf16", max_len=20011,
             ragged=True, window=1000, lens_seed=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attn", "attn"])
    if op == "norm":
        y = rng.random() < 0.6
        return dict(op="norm", T=_log_int(rng, 1, 4096), H=32 * _log_int(rng, 4, 224), residual=rng.random() < 0.7,
                    y=y, y8=not y or rng.random() < 0.5)
    fmt, dim, page = rng.choice(["e4m3", "e4m3", "bf16"]), rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        heads = rng.choice([1, 2, 4, 5, 8, 96])
        n = _log_int(rng, 1, min(16384, (1 << 24) // (heads * dim)))
        c = dict(op=op, n=n, heads=heads, dim=dim, page=page, fmt=fmt, pad=rng.choice([0, 0, n // 7]))
        return dict(c, fused=rng.random() < 0.5) if op == "write" else c
    heads = rng.choice([1, 2, 4, 8, 8, 96])
    group = rng.choice([1, 4, 5, 8, 12, 16]) if heads < 96 else 1
    batch = _log_int(rng, 1, 128)
    # as many cached bytes and products as the largest listed cases at most
    bytes_each = 2 * heads * dim * (1 if fmt == "e4m3" else 2)
    longest = max(1, min(131072, 1_000_000_000 // (batch * bytes_each), 10_000_000_000 // (4 * batch * heads * group * dim)))
    max_len = _log_int(rng, 1, longest)
    return dict(op="attn", B=batch, Hq=heads * group, Hkv=heads, dim=dim, page=page, fmt=fmt, max_len=max_len,
                ragged=rng.random() < 0.7, window=rng.choice([0, 0, 0, _log_int(rng, 1, max_len)]),
                lens_seed=rng.randrange(1 << 30))


def _lens(case):
    """Lengths of the sequences: all max_len, or spread over the logarithm with the longest
    first and, in a batch of three or more, an empty slot last."""
    if not case["ragged"]:
        return [case["max_len"]] * case["B"]
    rng = random.Random(case["lens_seed"])
    lens = [case["max_len"]] + [_log_int(rng, max(1, case["max_len"] // 64), case["max_len"])
                                for _ in range(case["B"] - 1)]
    if case["B"] > 2:
        lens[-1] = 0
    return lens


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        per = 2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0) + (1 + 1 / 32 if case["y8"] else 0)
        return {"bytes": n * per + 2 * case["H"], "flops": 5 * n}
    vec = case["dim"] + 1 if case["fmt"] == "e4m3" else 2 * case["dim"]  # bytes of a cached vector
    if case["op"] in ("write", "read"):
        live = 2 * (case["n"] - case["pad"]) * case["heads"]
        return {"bytes": live * (vec + 2 * case["dim"]) + 4 * case["n"]
                + (2 * case["pad"] * case["heads"] * 2 * case["dim"] if case["op"] == "read" else 0),
                "flops": 2 * live * case["dim"]}
    tokens = sum(min(n, case["window"] or n) for n in _lens(case))
    return {"bytes": tokens * case["Hkv"] * 2 * vec + case["B"] * case["Hq"] * (4 * case["dim"] + 4),
            "flops": 4 * tokens * case["Hq"] * case["dim"]}


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
        c, s = _quant(x[p:p + step].float())
        codes[p:p + step], scales[p:p + step] = c, s
    return codes, scales


def _forget(values, scales, where):
    """What lies in cache places that hold no token: anything, here NaN."""
    if scales is None:
        values[where] = float("nan")
    else:
        values[where] = 0x7F
        scales[where] = 255


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _normal(g, T, H)
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
        big = torch.exp(1.0 * torch.randn(H, generator=g, device="cuda")).bfloat16()  # a residual stream's channels
        s["res"] = _normal(g, T, H).mul_(big) if case["residual"] else None
        s["res_out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if case["residual"] else None
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if case["y"] else None
        s["codes"] = torch.empty(T, H, dtype=torch.uint8, device="cuda") if case["y8"] else None
        s["scales"] = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda") if case["y8"] else None
        return s
    page, dim = case["page"], case["dim"]
    rng = random.Random(seed)
    if case["op"] in ("write", "read"):
        n, heads = case["n"], case["heads"]
        pages = -(-n // page) + 2
        order = rng.sample(range(pages), pages)
        if n < 2 * page:  # tokens of a step: anywhere
            slots = rng.sample(range(pages * page), n)
        else:  # consecutive tokens: page after page of a shuffled list
            slots = [order[i // page] * page + i % page for i in range(n)]
        for i in rng.sample(range(n), case["pad"]):
            slots[i] = -1
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
        s["k"], s["ks"] = _cached(g, pages, heads, page, dim, case["fmt"])
        s["v"], s["vs"] = _cached(g, pages, heads, page, dim, case["fmt"])
        if case["op"] == "read":
            s["k_out"] = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")
            s["v_out"] = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")
        elif case["fused"]:  # slices of a fused projection of 4 query heads per cached one
            qkv = _normal(g, n, 6 * heads, dim)
            s["k_new"], s["v_new"] = qkv[:, 4 * heads:5 * heads], qkv[:, 5 * heads:]
        else:
            s["k_new"], s["v_new"] = _normal(g, n, heads, dim), _normal(g, n, heads, dim)
    else:
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        lens = _lens(case)
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
                for values, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
                    _forget(values, scales, (mine[-1], slice(None), slice(lens[b] % page, None)))
        for values, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            _forget(values, scales, torch.tensor(order[at:], device="cuda"))
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal(g, B, Hq + 2 * Hkv, dim)[:, :Hq]  # the query heads of a fused projection
        s["out"] = torch.empty(B, Hq, dim, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
    if own:
        import mxfp4_expert_ffn_router_gb300 as k3
        s["cache"] = k3.KVCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "attn":
            s["ws"] = torch.empty(k3.k3moe_attn_decode_workspace_bytes(s["cache"], case["B"], case["Hq"]),
                                  dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _cache_out(s):
    if s["ks"] is None:
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"].view(E4M3), "k_scales": s["ks"].view(E8M0), "v": s["v"].view(E4M3), "v_scales": s["vs"].view(E8M0)}


def _norm_out(s):
    return {"residual": s["res_out"], "y": s["out"], "codes": s["codes"].view(E4M3) if s["y8"] else None,
            "scales": s["scales"].view(E8M0) if s["y8"] else None}


def _run_own(s):
    import mxfp4_expert_ffn_router_gb300 as k3
    if s["op"] == "norm":
        k3.k3moe_rmsnorm(s["x"], s["weight"], EPS, residual=s["res"], residual_out=s["res_out"], y=s["out"],
                         codes=s["codes"], scales=s["scales"])
        return _norm_out(s)
    if s["op"] == "write":
        k3.k3moe_kv_write(s["cache"], s["k_new"], s["v_new"], s["slots"])
        return _cache_out(s)
    if s["op"] == "read":
        k3.k3moe_kv_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    k3.k3moe_attn_decode(s["cache"], s["q"], s["table"], s["lens"], s["out"], lse=s["lse"], window=s["window"], ws=s["ws"])
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


def _run_plain(s):
    if s["op"] == "norm":
        a = s["x"].float()
        if s["residual"]:
            a = a + s["res"].float()
            s["res_out"].copy_(a)
        y = a * torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        if s["y"]:
            s["out"].copy_(y)
        if s["y8"]:
            codes, scales = _quant(y.view(s["T"], -1, 32))
            s["codes"].copy_(codes.view(s["T"], -1))
            s["scales"].copy_(scales)
        return _norm_out(s)
    if s["op"] in ("write", "read"):
        slots, page = s["slots"].long(), s["page"]
        if s["op"] == "write":
            live = slots >= 0
            pg, at = slots[live] // page, slots[live] % page
            k, v = s["k_new"][live], s["v_new"][live]
            if s["ks"] is None:
                s["k"][pg, :, at], s["v"][pg, :, at] = k, v
            else:
                s["k"][pg, :, at], s["ks"][pg, :, at] = _quant(k.float())
                s["v"][pg, :, at], s["vs"][pg, :, at] = _quant(v.float())
            return _cache_out(s)
        live = (slots >= 0)[:, None, None]
        pg, at = slots.clamp(min=0) // page, slots.clamp(min=0) % page
        for values, scales, to in ((s["k"], s["ks"], s["k_out"]), (s["v"], s["vs"], s["v_out"])):
            x = _values(values[pg, :, at], None if scales is None else scales[pg, :, at])
            to.copy_(torch.where(live, x, torch.zeros_like(x)))
        return s["k_out"], s["v_out"]
    B, Hq, Hkv, dim = s["B"], s["Hq"], s["Hkv"], s["dim"]
    pg = s["table"].clamp(min=0).long()

    def gathered(values, scales):  # [B, Hkv, tokens, dim]
        x = _values(values[pg], None if scales is None else scales[pg])
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, dim)

    k, v = gathered(s["k"], s["ks"]), gathered(s["v"], s["vs"])
    t = torch.arange(k.shape[2], device=k.device)
    seen = t < s["lens"][:, None]
    if s["window"]:
        seen = seen & (t >= s["lens"][:, None] - s["window"])
    seen = seen[:, None, None, :]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, dim)
    scores = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(dim))
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(seen.transpose(2, 3), v, torch.zeros_like(v)))
    s["out"].copy_(torch.where(total == 0, torch.zeros_like(o), o / total).view(B, Hq, dim))
    s["lse"].copy_((m + torch.log(total)).view(B, Hq))
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
    if case["op"] == "norm":
        a = s["x"].double() + (s["res"].double() if case["residual"] else 0)
        y = a / torch.sqrt((a * a).sum(-1, keepdim=True) / case["H"] + EPS) * s["weight"].double()
        codes, scales = _exact_quant(y.view(case["T"], -1, 32)) if case["y8"] else (None, None)
        return {"residual": a if case["residual"] else None, "y": y if case["y"] else None,
                "codes": codes.view(case["T"], -1) if case["y8"] else None, "scales": scales}
    if case["op"] in ("write", "read"):
        slots, page = s["slots"].long(), case["page"]
        live = torch.nonzero(slots >= 0)[:, 0]
        pg, at = slots[live] // page, slots[live] % page
        if case["op"] == "read":
            both = []
            for values, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
                out = torch.zeros(case["n"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
                out[live] = _exact_values(values[pg, :, at], None if scales is None else scales[pg, :, at])
                both.append(out)
            return tuple(both)
        out = {}
        for name, values, scales, new in (("k", s["k"], s["ks"], s["k_new"]), ("v", s["v"], s["vs"], s["v_new"])):
            new = new[live].double()
            if scales is None:
                full = values.double()
                full[pg, :, at] = new
            else:
                full = _exact_values(values, torch.full_like(scales, 127))
                unit = _exact_pow2(scales.long() - 127)
                full[pg, :, at], unit[pg, :, at] = _exact_quant(new)
                out[name + "_scales"] = unit
            out[name] = full
        return out
    B, Hq, Hkv, dim, page = case["B"], case["Hq"], case["Hkv"], case["dim"], case["page"]
    out = torch.zeros(B, Hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        mine = s["table"][b, :-(-n // page)].long()
        first = max(0, n - case["window"]) if case["window"] else 0
        k, v = (_exact_values(x[mine], None if y is None else y[mine]).transpose(0, 1).reshape(Hkv, -1, dim)[:, first:n]
                for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        scores = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(Hkv, -1, dim), k) / math.sqrt(dim)
        lse[b] = torch.logsumexp(scores, -1).view(Hq)
        out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(scores, -1), v).reshape(Hq, dim)
    return out, lse
