"""bf16 queries and keys over all of bf16's range in the paged decode: any finite
values whose logits are finite."""
import numpy as np
import pytest

import paged_reference as R
import rope_context_extension_jet_b200 as jl
from test_paged import Pool, check_tree, ints, queries, random_parents, to64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes", [[1, 1], [5, 8], [13, 30], [64, 64]])  # 4 to 256 query rows of a kv head
@pytest.mark.parametrize("q_exp,k_exp,s_exp", [
    (-110, 110, 0), (-120, 120, 0), (-124, 124, 0), (110, -110, 0), (120, -120, 0),
    (60, 60, -120), (110, 10, -120), (10, 110, -120), (-120, 20, 100), (20, -120, 100),
])
def test_ordinary_logits_of_extreme_operands(nodes, q_exp, k_exp, s_exp):
    check_tree(81, [333, 40], nodes, q_scale=2.0 ** q_exp, k_scale=2.0 ** k_exp, scale=2.0 ** s_exp * 128 ** -0.5)


@pytest.mark.parametrize("T", [1, 8, 30, 64])
def test_keys_of_very_different_sizes(T):
    """Rows from 2^-90 to 2^112 in one cache: each is scaled by its own power of two."""
    import torch
    L, Hq, Hkv, d, ps = 500, 8, 2, 128, 64
    pool = Pool(82, [L + T], Hkv, d, ps, "bf16")
    g = np.random.default_rng(82)
    size = torch.from_numpy(2.0 ** g.integers(-90, 113, (pool.num, 1, ps, 1))).float().cuda()
    size[g.random((pool.num, 1, ps, 1)) < 0.2] = 2.0 ** 112
    pool.kc.copy_((pool.kc.float() * size).bfloat16())
    q = queries(82, T, Hq, d, "bf16", 2.0 ** -112)
    par = random_parents(g, T, "random")
    out = jl.decode_tree(q, pool.kc, pool.vc, pool.tab, ints([L]), ints([0, T]), ints(par), max_nodes=T, w0=64,
                         w_pretrained=200, rope_theta=1e4)
    jl.device_status()
    ref, tol = R.attend(to64(q), *pool.host(), pool.table[0], L, par, w0=64, w_pre=200, theta=1e4, scale=d ** -0.5, dtype="bf16")
    assert (np.abs(to64(out) - ref) <= tol).all()


@pytest.mark.parametrize("T", [1, 8, 30, 64])
def test_huge_operands_at_right_angles(T):
    """Logits of 0 from operands whose norms' product is far outside fp32: the plain mean."""
    import torch
    L, Hq, Hkv, d, ps = 300, 8, 2, 128, 64
    pool = Pool(83, [L + T], Hkv, d, ps, "bf16")
    k = torch.zeros_like(pool.kc)
    k[..., 7] = 2.0 ** 125
    q = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 2.0 ** 125
    out = to64(jl.decode_tree(q, k, pool.vc, pool.tab, ints([L]), ints([0, T]), max_nodes=T, w0=64, w_pretrained=200,
                              rope_theta=1e4))
    jl.device_status()
    v = R.gather(pool.host()[1], pool.table[0], L + T)
    for t in range(T):
        for h in range(Hq):
            x = v[h // 4][:L + t + 1]
            want = x.mean(0)
            tol = (2.0 ** -8 + (L + T + d) * 2.0 ** -24) * np.abs(x).mean(0) + 2.0 ** -8 * np.abs(want)
            assert (np.abs(out[t, h] - want) <= tol).all(), (t, h)
