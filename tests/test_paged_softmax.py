"""Running softmax of the paged decode kernels where its references move: logits
that climb by tens of octaves along the cache, in one half of a tile, in every
second tile, for some rows only, or that fall from the first tile on.

Keys and queries have two non-zero elements, in the dimensions that turn slowest,
and rope_theta is so large that those do not turn at all, so a logit is scale <q, k>
whatever the positions, and every operand is exact in fp16 (bf16 values have 8 bits).
"""
import numpy as np
import pytest

import paged_reference as R
import rope_context_extension_jet_b200 as jl
from test_paged import dt, ints, random_parents, to64

pytestmark = pytest.mark.gpu

THETA = 1e30
PS = 64
LENS = [4000, 3970, 4032, 3905, 2500, 130, 0]  # one profile each; together 1000 tiles of 128 keys over 8 kv heads


def profile(kind, n, g):
    """Height in octaves of every key (each with noise of some octaves added later)."""
    j = np.arange(n)
    tile, half = j // 128, (j // 64) % 2
    if kind == 0:    # climbs with every tile
        return 20.0 * tile
    if kind == 1:    # climbs in the second half of odd tiles only
        return np.where((tile % 2 == 1) & (half == 1), 30.0 * tile, 0.0)
    if kind == 2:    # every second tile is far above its neighbours, and climbs
        return np.where(tile % 2 == 0, 0.0, 50.0 + 16.0 * tile)
    if kind == 3:    # falls from the first tile on
        return -24.0 * tile
    if kind == 4:    # single keys stand out, each far above the last
        at = np.sort(g.choice(n, max(1, n // 300), replace=False))
        return np.where(np.isin(j, at), 45.0 * (1 + np.searchsorted(at, j)), 0.0)
    return 64.0 * half  # one tile or two


def case(dtype, d, Hq, Hkv, nodes, k_scale):
    """Caches, queries and what attention over them gives, with its tolerance."""
    import torch
    g = np.random.default_rng([d, Hq, nodes])
    h, group, T = d // 2, Hq // Hkv, nodes
    pages = [-(-(L + T) // PS) for L in LENS]
    num = sum(pages) + 2
    order, at = g.permutation(num), 0
    table = np.full((len(LENS), max(pages) + 1), num - 1, np.int64)
    kc = np.full((num, Hkv, PS, d), np.nan, np.float32)
    vc = np.full((num, Hkv, PS, d), np.nan, np.float32)
    par = random_parents(g, T, "comb")
    up = R.tree(par)[1]
    q = np.zeros((len(LENS) * T, Hq, d), np.float32)
    # most rows see the climb as it is; others at half its height, not at all, or upside down
    rows = g.choice([1.0, 1.0, 1.0, 0.5, 0.0, -1.0], (len(LENS) * T, Hq))
    q[:, :, h - 1] = q[:, :, h - 2] = rows / k_scale
    want, tol = np.zeros((2,) + q.shape)
    for b, L in enumerate(LENS):
        n = L + T
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        r = np.arange(n)
        pg = table[b][r // PS]
        k = np.zeros((n, Hkv, d), np.float32)
        high = profile(b, n, g)[:, None] * np.log(2.0)
        k[:, :, h - 1] = torch.from_numpy(np.broadcast_to(high, (n, Hkv)).copy()).bfloat16().double().numpy()
        k[:, :, h - 2] = torch.from_numpy(g.uniform(-3, 3, (n, Hkv))).bfloat16().double().numpy()
        v = torch.from_numpy(g.standard_normal((n, Hkv, d))).to(dt(dtype)).double().numpy()
        kc[pg, :, r % PS], vc[pg, :, r % PS] = k * k_scale, v
        seen = np.concatenate([np.ones((T, L), bool), up], 1)
        for c in range(Hkv):
            x = rows[b * T:(b + 1) * T, c * group:(c + 1) * group]  # [T, group]
            s = x[:, :, None] * (k[:, c, h - 1].astype(np.float64) + k[:, c, h - 2])
            big = (np.abs(x[:, :, None]) * (np.abs(k[:, c, h - 1]) + np.abs(k[:, c, h - 2])).max()).max(-1)
            s = np.where(seen[:, None], s, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            rw, hd = slice(b * T, (b + 1) * T), slice(c * group, (c + 1) * group)
            want[rw, hd], mass = p @ v[:, c], p @ np.abs(v[:, c])
            # As in the plain implementation, but the operands of the logits are exact (fp32:
            # angles to 2^-21 for each operand), two products are summed and scaled, and each
            # of at most 40 moves of a reference, and the joins, multiply by a power that is
            # off by 2^-21.
            moves = 48 * 2.0 ** -21
            if dtype == "bf16":
                e, w, res = big * 16 * 2.0 ** -24, 2.0 ** -8 + (n + d) * 2.0 ** -24 + moves, 2.0 ** -8
            else:
                e, w, res = big * (2 * 2.0 ** -21 + 16 * 2.0 ** -24), (n + 64) * 2.0 ** -24 + moves, 2.0 ** -24
            tol[rw, hd] = (2 * e + w)[:, :, None] * mass + res * np.abs(want[rw, hd])
    cuda = lambda x: torch.from_numpy(x).cuda().to(dt(dtype))
    args = (cuda(q), cuda(kc), cuda(vc), ints(table), ints(LENS), ints([b * T for b in range(len(LENS) + 1)]),
            ints(par * len(LENS)))
    return args, want, tol


@pytest.mark.parametrize("dtype,Hq,Hkv,nodes,k_scale", [
    # query rows per kv head: 4, 32 (decode_paged_tc.cu), 80, 256 (decode_paged_rows.cu)
    ("bf16", 32, 8, 1, 1.0), ("bf16", 32, 8, 8, 1.0), ("bf16", 32, 8, 20, 1.0), ("bf16", 32, 8, 64, 1.0),
    # keys scaled by a power of two, row by row
    ("bf16", 32, 8, 8, 2.0 ** 30), ("bf16", 32, 8, 20, 2.0 ** 30), ("bf16", 32, 8, 64, 2.0 ** 30),
    # 1, 8, 16, 32
    ("fp32", 8, 8, 1, 1.0), ("fp32", 32, 8, 2, 1.0), ("fp32", 32, 8, 4, 1.0), ("fp32", 32, 8, 8, 1.0),
])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("w0,w_pre", [(100000, 100000), (700, 1500)])
def test_references_move(dtype, Hq, Hkv, nodes, k_scale, d, w0, w_pre):
    """Against the plain result, and the same bits in every run: the two warps that share
    a row, and the two streams, have to use the same references."""
    import torch
    args, want, tol = case(dtype, d, Hq, Hkv, nodes, k_scale)
    kw = dict(max_nodes=nodes, w0=w0, w_pretrained=w_pre, rope_theta=THETA, scale=1.0)
    out = jl.decode_tree(*args, **kw)
    jl.device_status()
    got = to64(out)
    err = np.abs(got - want)
    for b, L in enumerate(LENS):
        rows = slice(b * nodes, (b + 1) * nodes)
        assert np.isfinite(got[rows]).all(), (b, L)
        assert (err[rows] <= tol[rows]).all(), (b, L, float((err[rows] / tol[rows]).max()))
    for _ in range(10):
        assert torch.equal(jl.decode_tree(*args, **kw), out)
    jl.device_status()


@pytest.mark.parametrize("nodes", [9, 20, 32, 33, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_first_tiles_of_many_units(nodes, d):
    """More than 32 rows, hundreds of units of one to three tiles: a unit's first tasks take
    their maxima one after the other without an agreement between them, and those of
    its two streams differ by many octaves."""
    import torch
    g = np.random.default_rng([nodes, d])
    B, Hq, Hkv, h, T = 96, 32, 8, d // 2, nodes
    lens = [int(x) for x in g.integers(0, 384 - T, B)]
    wide = 384 // PS
    kc, vc = (torch.zeros(B * wide, Hkv, PS, d) for _ in range(2))
    high = torch.from_numpy(g.integers(0, 4, (B * wide, Hkv, PS)) * 20.0 + 60.0 * (np.arange(B * wide) % 3)[:, None, None])
    kc[..., h - 1] = high.bfloat16().float()
    vc.copy_(torch.from_numpy(g.standard_normal(vc.shape)))
    vc = vc.bfloat16()
    rows = g.choice([1.0, -1.0, 0.25], (B * T, Hq))
    q = torch.zeros(B * T, Hq, d)
    q[..., h - 1] = torch.from_numpy(rows).float()
    table = g.permutation(B * wide).reshape(B, wide)
    args = (q.cuda().bfloat16(), kc.cuda().bfloat16(), vc.cuda(), ints(table), ints(lens), ints([b * T for b in range(B + 1)]))
    kw = dict(max_nodes=T, w0=1 << 20, w_pretrained=1 << 20, rope_theta=THETA, scale=1.0)
    out = jl.decode_tree(*args, **kw)
    jl.device_status()
    got = to64(out)
    k64, v64 = kc[..., h - 1].double().numpy(), vc.double().numpy()
    for b, L in enumerate(lens):
        n = L + T
        r = np.arange(n)
        k, v = k64[table[b][r // PS], :, r % PS], v64[table[b][r // PS], :, r % PS]
        seen = np.concatenate([np.ones((T, L), bool), np.tri(T, dtype=bool)], 1)
        for c in range(Hkv):
            x = rows[b * T:(b + 1) * T, 4 * c:4 * c + 4]
            s = np.where(seen[:, None], x[:, :, None] * k[:, c], -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            want, mass = p @ v[:, c], p @ np.abs(v[:, c])
            # logits of at most 180, off by 16 * 2^-24 of that; else as above
            tol = (2 * 180 * 16 * 2.0 ** -24 + 2.0 ** -8 + (n + d) * 2.0 ** -24 + 8 * 2.0 ** -21) * mass + 2.0 ** -8 * np.abs(want)
            err = np.abs(got[b * T:(b + 1) * T, 4 * c:4 * c + 4] - want)
            assert (err <= tol).all(), (b, c, float((err / tol).max()))
    for _ in range(20):
        assert torch.equal(jl.decode_tree(*args, **kw), out)
    jl.device_status()


@pytest.mark.parametrize("dtype,Hq,nodes", [("bf16", 32, 1), ("bf16", 24, 3), ("bf16", 32, 5), ("bf16", 32, 9), ("bf16", 32, 20),
                                            ("bf16", 32, 33), ("bf16", 32, 50), ("fp32", 32, 1), ("fp32", 24, 3), ("fp32", 32, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_results_do_not_depend_on_what_ran_before(dtype, Hq, nodes, d):
    """Units with fewer rows than their kernel's tile has, and last tiles with fewer keys:
    what an earlier kernel left in shared memory in their place (NaN, infinities, large and
    small numbers) changes no bit."""
    import torch
    g = np.random.default_rng([Hq, nodes, d])
    Hkv, T = 8, nodes
    lens = [int(x) for x in g.integers(0, 400, 60)] + [2000, 1500, 0, 1]
    wide = 2 + (2000 + T) // 16
    num = sum(-(-(L + T) // 16) for L in lens) + 1
    order, at = g.permutation(num), 0
    table = np.zeros((len(lens), wide), np.int64)
    for b, L in enumerate(lens):
        p = -(-(L + T) // 16)
        table[b, :p] = order[at:at + p]
        at += p
    rnd = lambda *s: torch.from_numpy(g.standard_normal(s, dtype=np.float32)).cuda().to(dt(dtype))
    # logits that differ by tens of octaves, and elements that are subnormal in fp16
    q, kc, vc = rnd(len(lens) * T, Hq, d), rnd(num, Hkv, 16, d), rnd(num, Hkv, 16, d)
    kc *= (2.0 ** torch.randint(-16, 2, (num, Hkv, 16, 1), generator=torch.Generator().manual_seed(3))).cuda().to(kc.dtype)
    args = (q, kc, vc, ints(table), ints(lens), ints([b * T for b in range(len(lens) + 1)]))
    kw = dict(max_nodes=T, w0=100, w_pretrained=300, rope_theta=1e4, scale=4.0)
    before = []
    for value in (1.0, float("nan"), float("inf"), 3e38, -3e38, 1e-38, 0.0):
        # every SM's shared memory full of it
        x = torch.full((64 * 4, 32, d), value, device="cuda", dtype=dt(dtype))
        c = torch.full((200, Hkv, 64, d), value, device="cuda", dtype=dt(dtype))
        tab = ints(np.arange(200).reshape(4, 50))
        run = lambda: jl.decode_tree(x, c, c, tab, ints([3100] * 4), ints([64 * b for b in range(5)]), max_nodes=64, w0=100,
                                     w_pretrained=10000, rope_theta=1e4)
        before.append(run)
    out = jl.decode_tree(*args, **kw)
    assert torch.isfinite(out).all()
    for run in before:
        for _ in range(3):
            run()
            assert torch.equal(jl.decode_tree(*args, **kw), out)
    jl.device_status()
