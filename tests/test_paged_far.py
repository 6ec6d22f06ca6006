"""Pages more than 2^32 elements into a paged cache: append, attention of one row and of
trees, and commit give the bits that the same rows give in a small cache."""
import numpy as np
import pytest

import rope_context_extension_jet_b200 as jl
from test_paged import dt, ints, queries, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pages_behind_32_bit_offsets(dtype):
    import torch
    Hkv, ps, d, Hq, L = 2, 64, 128, 8, 1000
    num = (1 << 32) // (Hkv * ps * d) + 64
    kc, vc = (torch.empty((num, Hkv, ps, d), dtype=dt(dtype), device="cuda") for _ in range(2))
    for T in (1, 8, 30, 64):
        g = np.random.default_rng(T)
        N = L + T
        pages = -(-N // ps)
        far = num - 1 - g.permutation(60)[:pages]
        far[1] = 3
        sk, sv = (torch.from_numpy(g.standard_normal((pages, Hkv, ps, d), dtype=np.float32)).cuda().to(dt(dtype)) for _ in range(2))
        rows = lambda c, idx: c[idx].transpose(1, 2).reshape(-1, Hkv, d)[:N].contiguous()
        near, idx = torch.arange(pages, device="cuda"), torch.from_numpy(far.copy()).cuda()
        jl.cache_append(rows(sk, near), rows(sv, near), ints([int(far[r // ps]) * ps + r % ps for r in range(N)]), kc, vc)
        q, par = queries(T, T, Hq, d, dtype), ints(random_parents(g, T, "random"))
        out = []
        for k, v, table in ((sk, sv, near), (kc, vc, idx)):
            args = (k, v, table[None].int(), ints([L]), ints([0, T]), par)
            out.append(jl.decode_tree(q, *args, max_nodes=T, w0=100, w_pretrained=300, rope_theta=1e4))
            jl.tree_commit(*args, ints([T - 1]), max_nodes=T)
        jl.device_status()
        assert torch.equal(out[0], out[1])
        assert torch.equal(rows(kc, idx), rows(sk, near)) and torch.equal(rows(vc, idx), rows(sv, near))
