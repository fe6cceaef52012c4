"""GPU tests of the prompt-sized calls of the norm and the key-value cache, whose kernels
keep several tokens in flight or share an SM among more rows than a step's do, against
the float64 references with the bounds of the small calls' tests."""
import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
import test_gpu_kv_cache as kv
import test_gpu_rmsnorm as norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(700, 7168), (321, 16352), (311, 8192), (160, 8224), (900, 4096)])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_of_many_rows(T, H, residual):
    x, r, w = norm._inputs(T, H, T + H, residual)
    norm._check(x, r, w, norm._run(x, r, w))


@pytest.mark.parametrize("fmt", [k3.K3MOE_KV_E4M3, k3.K3MOE_KV_BF16])
@pytest.mark.parametrize("n,heads,dim,page,pad", [(4099, 8, 64, 64, 17), (4099, 8, 128, 16, 0), (4099, 8, 256, 128, 5),
                                                  (1999, 40, 64, 32, 1), (130, 200, 128, 16, 3)])
def test_cache_of_many_tokens(fmt, n, heads, dim, page, pad):
    c = kv._cache(n // page + 2, heads, page, dim, fmt)
    before = kv._host(c)
    slots = kv._slots(n, c.pages * page, n, pad)
    new = {"k": kv._vectors(n, heads, dim, 1), "v": kv._vectors(n, heads, dim, 2)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    k3.k3moe_kv_write(c, kv._dev(new["k"]), kv._dev(new["v"]), sl, st)
    after = kv._host(c)
    kv._same(after, kv._expect(before, c, slots, new))
    ko, vo = (torch.full((n, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3.k3moe_kv_read(c, sl, ko, vo, st)
    for got, want in zip((ko, vo), kv._read_expect(after, c, slots)):
        np.testing.assert_array_equal(kv._bits(got), want)
    assert int(st.item()) == 0
