"""CPU tests of the decoder calls' binding where the library reports an error: the error is
raised, and the call is not made a second time (in place, that would add a residual twice)."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from mxfp4_expert_ffn_router_gb300 import build as k3build


class _Fast:
    """The C++ way, whose calls all fail with `rc`."""

    def __init__(self, rc):
        self.calls, fail = [], lambda name: lambda *a: (self.calls.append(name), rc)[1]
        self.rmsnorm, self.kv_write, self.kv_read, self.attn_decode = map(fail, ("rmsnorm", "kv_write", "kv_read", "attn_decode"))


class _Lib:
    """The library, recording what the ctypes way would launch."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("k3moe_rmsnorm", "k3moe_kv_write", "k3moe_kv_read", "k3moe_attn_decode"):
            return lambda *a: (self.calls.append(name), 0)[1]
        return getattr(self.real, name)


@pytest.mark.parametrize("rc", [k3.K3MOE_ERR_LAUNCH, k3.K3MOE_ERR_ARG, k3.K3MOE_ERR_ALIGN])
def test_a_failed_call_is_not_made_again(rc, monkeypatch):
    k3build.build()
    fast, lib = _Fast(rc), _Lib(k3.lib())
    # CPU tensors stand in for CUDA ones: nothing is launched
    monkeypatch.setattr(k3, "_in", lambda t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(k3, "_ptr", lambda t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(k3, "_rows", lambda t, shape, name: (t.data_ptr(), shape[1] * shape[2]))
    monkeypatch.setattr(k3, "_stream", lambda s: None)
    monkeypatch.setattr(k3, "_fast", fast)
    monkeypatch.setattr(k3, "lib", lambda: lib)
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros(2, 64, **bf), torch.zeros(64, **bf)
    c = k3.KVCache(torch.zeros(2, 2, 16, 64, **bf), torch.zeros(2, 2, 16, 64, **bf))
    kv, i = torch.zeros(3, 2, 64, **bf), torch.zeros(3, dtype=torch.int32)
    for name, call in (("rmsnorm", lambda: k3.k3moe_rmsnorm(x, w, 1e-6, residual=x, residual_out=x)),
                       ("kv_write", lambda: k3.k3moe_kv_write(c, kv, kv, i)),
                       ("kv_read", lambda: k3.k3moe_kv_read(c, i, kv, kv)),
                       ("attn_decode", lambda: k3.k3moe_attn_decode(c, kv, i[:, None], i, kv, ws=i))):
        with pytest.raises(k3.K3moeError) as e:
            call()
        assert e.value.args and k3.status_string(rc) in str(e.value), name
        assert fast.calls.pop() == name and not fast.calls and not lib.calls, name
