"""GPU tests of k3moe_attn_decode's arguments through the binding: numbers past 32 bits
are not cut to their low bits."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from test_gpu_attn_decode import BF, E4, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["fast", "ctypes"])
@pytest.mark.parametrize("fmt", [E4, BF])
def test_windows_past_32_bits(way, fmt, monkeypatch):
    """A window larger than any length sees everything; a negative one is refused."""
    k3.lib()
    if way == "ctypes":
        monkeypatch.setattr(k3, "_fast", None)
    c = Case([100, 33, 0], 4, 2, 64, 16, fmt, seed=1)
    out, lse = c.run()
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63, 2 ** 64 + 5):
        got, gl = c.run(window=window)
        assert torch.equal(got, out) and torch.equal(gl, lse), window
    for window in (-1, -2 ** 31, 5 - 2 ** 32, 5 - 2 ** 64):
        with pytest.raises(k3.K3moeError):
            c.run(window=window)
