"""GPU tests of the decoder calls' binding: the C++ way and the ctypes way give the same
bytes and refuse the same arguments (writing nothing), and 8-bit tensors may be typed
(float8) or bytes."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["fast", "ctypes"])
def way(request, monkeypatch):
    k3.lib()
    assert k3._fast is not None
    if request.param == "ctypes":
        monkeypatch.setattr(k3, "_fast", None)
    return request.param


def _bf(*sizes, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*sizes, device="cuda", generator=g).bfloat16()


def _everything(typed=False, stream=None):
    """Each call once; the bytes they wrote."""
    x, r, w = _bf(5, 256), _bf(5, 256, seed=1), _bf(256, seed=2)
    o = [torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    codes, scales = (torch.zeros(5, n, dtype=torch.uint8, device="cuda") for n in (256, 8))
    as8 = (lambda t: t.view(torch.float8_e4m3fn)) if typed else (lambda t: t)
    as_s = (lambda t: t.view(torch.float8_e8m0fnu)) if typed else (lambda t: t)
    k3.k3moe_rmsnorm(x, w, 1e-5, residual=r, residual_out=o[0], y=o[1], codes=as8(codes), scales=as_s(scales), stream=stream)
    k, v = (torch.zeros(3, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(3, 2, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = k3.KVCache(as8(k), as8(v), as_s(ks), as_s(vs))
    qkv = _bf(20, 8, 64, seed=3)
    slots = torch.arange(20, dtype=torch.int32, device="cuda") + 16
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k3.k3moe_kv_write(c, qkv[:, 4:6], qkv[:, 6:], slots, st, stream=stream)
    back = [torch.zeros(20, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k3.k3moe_kv_read(c, slots, *back, st, stream=stream)
    out, lse = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 4, device="cuda")
    ws = torch.zeros(k3.k3moe_attn_decode_workspace_bytes(c, 1, 4), dtype=torch.uint8, device="cuda")
    k3.k3moe_attn_decode(c, qkv[:1, :4], torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"),
                         torch.tensor([20], dtype=torch.int32, device="cuda"), out, lse=lse, scale=0.1, window=15, ws=ws,
                         dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return [t.view(torch.uint8).clone() for t in (*o, codes, scales, k, v, ks, vs, *back, out, lse, st)]


def test_both_ways_and_types_give_the_same(way):
    base = _everything()
    assert base[10].any()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for other in (_everything(typed=True), _everything(stream=torch.cuda.current_stream())):
        for a, b in zip(base, other):
            assert torch.equal(a, b)


def test_the_two_ways_agree(monkeypatch):
    k3.lib()
    a = _everything()
    monkeypatch.setattr(k3, "_fast", None)
    for x, y in zip(a, _everything()):
        assert torch.equal(x, y)


def test_refusals(way):
    x, w = _bf(4, 64), _bf(64)
    y = torch.zeros_like(x)
    u8 = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    bad = [dict(x=x.float()), dict(x=x[:, :32]), dict(weight=w[:32]), dict(weight=w.float()), dict(y=y[:2]), dict(y=y.t()),
           dict(y=y.cpu()), dict(residual=x[:2]), dict(residual_out=y.float()), dict(codes=y, scales=u8[:, :2]),
           dict(codes=u8, scales=u8[:, :1]), dict(codes=u8), dict(scales=u8[:, :2].contiguous()), dict(y=None),
           dict(eps=float("nan")), dict(eps=-1.0), dict(x=x[0])]
    for kw in bad:
        a = dict(dict(x=x, weight=w, eps=1e-6, y=y), **kw)
        with pytest.raises((ValueError, TypeError, k3.K3moeError)):
            k3.k3moe_rmsnorm(a.pop("x"), a.pop("weight"), a.pop("eps"), **a)
    assert not y.any() and not u8.any()
    c = k3.KVCache(*(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    kv, slots = _bf(3, 2, 64), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for args in ((kv[:2], kv, slots), (kv, kv.float(), slots), (kv, kv.cpu(), slots), (kv, kv, slots.long()),
                 (kv, kv, slots[:2]), (kv.transpose(0, 1).contiguous().transpose(0, 1), kv, slots), (kv[..., :32], kv, slots)):
        with pytest.raises((ValueError, TypeError, k3.K3moeError)):
            k3.k3moe_kv_write(c, *args)
    assert not c.k.any() and not c.v.any()
    out = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for args in ((slots, out[:2], out), (slots, out.float(), out), (slots.long(), out, out), (slots, out, out.cpu())):
        with pytest.raises((ValueError, TypeError, k3.K3moeError)):
            k3.k3moe_kv_read(c, *args)
    q, table = _bf(2, 4, 64), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    o = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(k3.k3moe_attn_decode_workspace_bytes(c, 2, 4), dtype=torch.uint8, device="cuda")
    good = dict(q=q, block_table=table, seq_lens=lens, out=o, ws=ws)
    bad = [dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[0]), dict(block_table=table[:1]), dict(block_table=table[0]),
           dict(block_table=table.long()), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long()), dict(out=o[:, :2]),
           dict(out=o.float()), dict(lse=torch.zeros(2, 3, device="cuda")), dict(ws=ws[:-1]), dict(ws=None),
           dict(ws=ws[16:]), dict(window=-1), dict(scale=float("inf")), dict(seq_lens=lens.cpu())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, k3.K3moeError)):
            k3.k3moe_attn_decode(c, **dict(good, **kw))
    torch.cuda.synchronize()
    assert (out == 7).all() and (o == 7).all()
    k3.k3moe_attn_decode(c, **good)
