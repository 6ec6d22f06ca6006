"""Paged cache on the GPU: block tables, cache append, decode of one row or a
drafted tree per request, commit of a draft, and a run of them together,
against plain 64-bit implementations."""
import numpy as np
import pytest

import paged_reference as R
import rope_context_extension_jet_b200 as jl

pytestmark = pytest.mark.gpu


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Pool:
    """Random caches with room for rows[b] rows of each request in shuffled
    pages; every row no request owns holds NaN."""

    def __init__(self, seed, rows, Hkv, d, ps, dtype, spare=3, k_scale=1.0):
        import torch
        g = np.random.default_rng(seed)
        per = [-(-n // ps) for n in rows]
        num = sum(per) + spare
        order = g.permutation(num)
        wide = max(max(per), 1) + 1
        self.table = np.full((len(rows), wide), num - 1, np.int64)
        shape = (num, Hkv, ps, d)
        k = np.full(shape, np.nan, np.float32)
        v = np.full(shape, np.nan, np.float32)
        at = 0
        for b, (n, p) in enumerate(zip(rows, per)):
            self.table[b, :p] = order[at:at + p]
            at += p
            r = np.arange(n)
            pg = self.table[b][r // ps]
            k[pg, :, r % ps] = k_scale * g.standard_normal((n, Hkv, d), dtype=np.float32)
            v[pg, :, r % ps] = g.standard_normal((n, Hkv, d), dtype=np.float32)
        self.kc = torch.from_numpy(k).cuda().to(dt(dtype))
        self.vc = torch.from_numpy(v).cuda().to(dt(dtype))
        self.tab = ints(self.table)
        self.num, self.ps, self.Hkv, self.d, self.dtype = num, ps, Hkv, d, dtype

    def host(self):
        return to64(self.kc), to64(self.vc)


def queries(seed, N, Hq, d, dtype, scale=1.0):
    import torch
    x = scale * np.random.default_rng([seed, 9]).standard_normal((N, Hq, d), dtype=np.float32)
    return torch.from_numpy(x).cuda().to(dt(dtype))


def random_parents(g, T, kind):
    if kind == "chain":
        return [t - 1 for t in range(T)]
    if kind == "star":
        return [-1] * T
    if kind == "comb":  # a path with one leaf beside each node
        return [-1 if t == 0 else (t - 1 if t % 2 else max(0, t - 2)) for t in range(T)]
    return [-1 if t == 0 else int(g.integers(-1, t)) for t in range(T)]


def starts_of(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def check_tree(seed, lens, nodes, kind="random", Hq=8, Hkv=2, d=128, ps=64, dtype="bf16", w0=64, w_pre=400, theta=1e4,
               scale=None, q_scale=1.0, k_scale=1.0, pad=3, none_parents=False):
    import torch
    g = np.random.default_rng([seed, 1])
    pool = Pool(seed, [max(0, a) + t for a, t in zip(lens, nodes)], Hkv, d, ps, dtype, k_scale=k_scale)
    N = sum(nodes) + pad
    q = queries(seed, N, Hq, d, dtype, q_scale)
    par = [random_parents(g, t, kind) for t in nodes]
    flat = ints([x for p in par for x in p] + [-1] * pad)
    out = torch.full_like(q, 7.5)
    kw = dict(w0=w0, w_pretrained=w_pre, rope_theta=theta)
    scale = d ** -0.5 if scale is None else scale
    jl.decode_tree(q, pool.kc, pool.vc, pool.tab, ints(lens), ints(starts_of(nodes)), None if none_parents else flat, out,
                   max_nodes=max(1, max(nodes)), scale=scale, **kw)
    jl.device_status()
    got, q64 = to64(out), to64(q)
    k64, v64 = pool.host()
    at = 0
    for b, (L, T) in enumerate(zip(lens, nodes)):
        if T:
            ref, tol = R.attend(q64[at:at + T], k64, v64, pool.table[b], L, par[b], w0=w0, w_pre=w_pre, theta=theta,
                                scale=scale, dtype=dtype)
            err = np.abs(got[at:at + T] - ref)
            assert np.isfinite(got[at:at + T]).all(), (b, L, T)
            assert (err <= tol).all(), (b, L, T, float((err / tol).max()))
        at += T
    assert (got[at:] == 7.5).all(), "rows behind the last request were written"
    return out


# ------------------------------------------------------------------ decode_tree
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,nodes", [
    ([0], [1]), ([0], [5]), ([1], [2]), ([63], [1]), ([64], [1]), ([127], [2]), ([128], [3]),
    ([300, 0, 17], [7, 1, 4]), ([500, 130, 255], [0, 9, 16]), ([0, 0, 0], [64, 0, 33]), ([777], [64]),
])
def test_tree_lengths(dtype, lens, nodes):
    check_tree(11, lens, nodes, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["chain", "star", "comb", "random"])
def test_tree_shapes(dtype, kind):
    check_tree(12, [201, 390], [13, 31], kind=kind, dtype=dtype)


def test_chain_without_parents():
    check_tree(13, [150, 395], [6, 12], kind="chain", none_parents=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("w0", [0, 1, 3, 130, 100000])
@pytest.mark.parametrize("w_pre", [1, 50, 400, 100000])
def test_tree_windows_and_group_sizes(dtype, w0, w_pre):
    """Trees whose nodes have different G (w_pre = 1: every depth its own)."""
    check_tree(14, [396, 95], [9, 20], kind="comb", w0=w0, w_pre=w_pre, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (7, 1, 128), (6, 2, 64), (8, 8, 128), (32, 8, 128), (16, 1, 64),
                                      (71, 1, 64)])
def test_tree_heads(dtype, Hq, Hkv, d):
    check_tree(15, [270, 33], [11, 3], Hq=Hq, Hkv=Hkv, d=d, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_page_sizes(dtype, ps):
    check_tree(16, [15, 16, 17, 255, 256, 300], [1, 2, 3, 1, 4, 10], ps=ps, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_and_short_requests_cut_into_pieces(dtype):
    check_tree(17, [6000, 3, 2500, 0, 4097], [1, 4, 2, 3, 6], w_pre=1000, w0=300, dtype=dtype)


@pytest.mark.parametrize("d,nodes,dtype", [(d, t, "bf16") for d in (128, 64) for t in (1, 4, 8, 16, 40)] +
                         [(d, t, "fp32") for d in (128, 64) for t in (1, 2, 4, 10)])
def test_long_batches_keep_their_tiles_apart(d, nodes, dtype):
    """Every CTA works through dozens of tiles, several units and phases with its
    rings of tiles always full; runs repeat bit for bit.  Rows no request owns hold
    NaN, so that a tile taken too early or repaired too late shows."""
    import torch
    B, Hq, Hkv, ps = 8, 32, 8, 64
    lens = [20000, 19999, 3, 12345, 20011, 0, 16384, 7777]
    pages = (max(lens) + nodes + ps - 1) // ps
    gen = torch.Generator(device="cuda").manual_seed(5)
    num = B * pages + 1
    table = torch.randperm(num, generator=gen, device="cuda")[:B * pages].view(B, pages).int()
    kc, vc = (torch.randn(num, Hkv, ps, d, generator=gen, device="cuda").to(dt(dtype)) for _ in range(2))
    for b, L in enumerate(lens):
        n = L + nodes
        for c in (kc, vc):
            c[table[b, -(-n // ps):].long()] = float("nan")
            if n % ps:
                c[int(table[b, n // ps]), :, n % ps:] = float("nan")
    q = queries(5, B * nodes, Hq, d, dtype)
    par = random_parents(np.random.default_rng(5), nodes, "comb")
    args = (q, kc, vc, table, ints(lens), ints([b * nodes for b in range(B + 1)]), ints(par * B))
    kw = dict(max_nodes=nodes, w0=700, w_pretrained=5000, rope_theta=1e6)
    got = jl.decode_tree(*args, **kw)
    jl.device_status()
    for _ in range(20):
        again = jl.decode_tree(*args, **kw)
        assert torch.equal(again.view(torch.int16), got.view(torch.int16))  # (bits: no NaN may hide)
    jl.device_status()
    got, q64, tab = to64(got), to64(q), table.cpu().numpy()
    for b, L in enumerate(lens):
        h, rows = b % Hkv, slice(b * nodes, (b + 1) * nodes)
        heads = slice(4 * h + b % 4, 4 * h + b % 4 + 1)  # one query head of each request
        k1, v1 = (torch.zeros(pages, 1, ps, d) for _ in range(2))
        k1[:, 0], v1[:, 0] = (c[table[b].long(), h].float().cpu() for c in (kc, vc))
        ref, tol = R.attend(q64[rows, heads], k1.numpy().astype(np.float64), v1.numpy().astype(np.float64), np.arange(pages), L,
                            par, w0=700, w_pre=5000, theta=1e6, scale=d ** -0.5, dtype=dtype)
        err = np.abs(got[rows, heads] - ref)
        assert (err <= tol).all(), (b, L, float((err / tol).max()))


def test_many_requests():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 90, 700)]
    check_tree(18, lens, [1 + (i % 3) for i in range(700)], Hq=2, Hkv=1, d=64, ps=16)


@pytest.mark.parametrize("q_scale,k_scale", [(1e-3, 1e-3), (1e-6, 1e6), (1e6, 1e-6), (2e-16, 2e15), (30.0, 1.0)])
def test_bf16_operand_range(q_scale, k_scale):
    """Keys and queries far outside fp16's range whose logits are ordinary."""
    s = min(1.0, 1.0 / (q_scale * k_scale * 128 ** 0.5)) if q_scale * k_scale > 1 else None
    check_tree(19, [333, 40], [5, 9], q_scale=q_scale, k_scale=k_scale, scale=s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_in_rows_a_node_does_not_attend_stay_out(dtype, value):
    """One drafted row holds NaN or infinities: only its descendants see it."""
    import torch
    L, T, Hq, Hkv, d, ps = 100, 8, 8, 2, 128, 16
    parents = [-1, 0, 0, 1, 1, 2, 2, -1]
    pool = Pool(21, [L + T], Hkv, d, ps, dtype)
    row, bad = L + 2, 2
    page = int(pool.table[0][row // ps])
    q = queries(21, T, Hq, d, dtype)
    args = (ints([L]), ints([0, T]), ints(parents))
    kw = dict(max_nodes=T, w0=16, w_pretrained=60, rope_theta=1e4)
    ref = jl.decode_tree(q, pool.kc, pool.vc, pool.tab, *args, **kw)
    sees = R.tree(parents)[1][:, bad]
    for which in ("v", "k"):
        kc, vc = pool.kc.clone(), pool.vc.clone()
        (vc if which == "v" else kc)[page, :, row % ps, 5::7] = value
        got = jl.decode_tree(q, kc, vc, pool.tab, *args, **kw)
        jl.device_status()
        for t in range(T):
            if not sees[t]:
                assert torch.equal(got[t], ref[t]), (which, t)
            elif which == "v":
                hit = torch.zeros(d, dtype=torch.bool, device="cuda")
                hit[5::7] = True
                assert not torch.isfinite(got[t][:, hit]).any() and torch.equal(got[t][:, ~hit], ref[t][:, ~hit]), t
            elif value != value:
                assert torch.isnan(got[t]).all()


# ------------------------------------------------------------------ decode_paged
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_paged_decode_with_idle_requests(dtype):
    import torch
    lens = [700, -1, 0, 399, 400, -1, 63]
    pool = Pool(31, [max(0, x + 1) for x in lens], 2, 128, 32, dtype)
    q = queries(31, len(lens), 8, 128, dtype)
    out = torch.full_like(q, 7.5)
    jl.decode_paged(q, pool.kc, pool.vc, pool.tab, ints(lens), out, w0=50, w_pretrained=400, rope_theta=1e6)
    jl.device_status()
    got, q64 = to64(out), to64(q)
    k64, v64 = pool.host()
    for b, L in enumerate(lens):
        if L < 0:
            assert (got[b] == 7.5).all()
            continue
        ref, tol = R.attend(q64[b:b + 1], k64, v64, pool.table[b], L, [-1], w0=50, w_pre=400, theta=1e6, scale=128 ** -0.5,
                            dtype=dtype)
        assert (np.abs(got[b] - ref[0]) <= tol[0]).all(), (b, L)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_paged_decode_equals_decode_on_a_contiguous_cache(dtype):
    import torch
    B, Hq, Hkv, d, L, ps = 3, 8, 2, 128, 1300, 64
    pool = Pool(32, [L + 1] * B, Hkv, d, ps, dtype)
    q = queries(32, B, Hq, d, dtype)
    pages = -(-(L + 1) // ps)
    kc, vc = (c[pool.tab[:, :pages].long()].transpose(1, 2).reshape(B, Hkv, pages * ps, d).contiguous()
              for c in (pool.kc, pool.vc))
    kw = dict(w0=100, w_pretrained=500, rope_theta=1e6)
    a = jl.decode(q, kc, vc, L + 1, **kw)
    b = jl.decode_paged(q, pool.kc, pool.vc, pool.tab, ints([L] * B), **kw)
    jl.device_status()
    k64, v64 = pool.host()
    for i in range(B):
        _, tol = R.attend(to64(q)[i:i + 1], k64, v64, pool.table[i], L, [-1], w0=100, w_pre=500, theta=1e6,
                          scale=d ** -0.5, dtype=dtype)
        assert (np.abs(to64(a)[i] - to64(b)[i]) <= 2 * tol[0]).all()


def test_results_do_not_depend_on_the_workspace_or_the_run():
    import torch
    lens, nodes = [3000, 5, 1200], [4, 2, 7]
    pool = Pool(33, [a + t for a, t in zip(lens, nodes)], 2, 128, 64, "bf16")
    q = queries(33, sum(nodes), 8, 128, "bf16")
    ws = torch.empty(jl.decode_tree_workspace_size(3, 8, 2, 128, 7), dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0xFF, 0x5A, 0):
        ws.fill_(fill)
        outs.append(jl.decode_tree(q, pool.kc, pool.vc, pool.tab, ints(lens), ints(starts_of(nodes)), max_nodes=7, w0=64,
                                   w_pretrained=900, rope_theta=1e4, workspace=ws).clone())
    jl.device_status()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_streams_with_their_own_workspaces():
    import torch
    lens, nodes = [2000, 900], [8, 8]
    pool = Pool(34, [a + t for a, t in zip(lens, nodes)], 2, 128, 64, "bf16")
    q = queries(34, 16, 8, 128, "bf16")
    args = (pool.kc, pool.vc, pool.tab, ints(lens), ints(starts_of(nodes)))
    kw = dict(max_nodes=8, w0=64, w_pretrained=900, rope_theta=1e4)
    ref = jl.decode_tree(q, *args, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    size = jl.decode_tree_workspace_size(2, 8, 2, 128, 8)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [torch.empty_like(q) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, o in zip(streams, ws, outs):
            jl.decode_tree(q, *args, None, o, workspace=w, stream=s, **kw)
    torch.cuda.synchronize()
    jl.device_status()
    assert all(torch.equal(o, ref) for o in outs)


# ------------------------------------------------------------------ cache_append
def test_own_tensors_of_a_call_on_another_stream():
    """Workspaces and results that a call makes for itself belong to the stream it runs
    on: work of the current stream before and after it does not touch them."""
    import torch
    pool = Pool(23, [3000, 200], 2, 128, 64, "bf16")
    q = queries(23, 2, 8, 128, "bf16")
    args = (q, pool.kc, pool.vc, pool.tab, ints([2999, 199]))
    kw = dict(w0=64, w_pretrained=400, rope_theta=1e4)
    ref = jl.decode_paged(*args, **kw)
    size = jl.decode_tree_workspace_size(2, 8, 2, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # the call starts some 10 ms later
        out = jl.decode_paged(*args, stream=s, **kw)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        jl.device_status()
        assert torch.equal(out, ref)
        del junk


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,Hkv,d,ps", [(0, 2, 64, 16), (1, 1, 64, 16), (5, 3, 128, 32), (1000, 8, 128, 64)])
@pytest.mark.parametrize("layout", ["plain", "fused", "heads_first"])
def test_append(dtype, N, Hkv, d, ps, layout):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    num = N // ps + 4
    kc = torch.full((num, Hkv, ps, d), 3.0, dtype=dt(dtype), device="cuda")
    vc = torch.full_like(kc, 4.0)
    if layout == "fused":
        x = torch.randn((N, (4 + 2 * Hkv) * d), dtype=dt(dtype), device="cuda", generator=g)
        k, v = x[:, 4 * d:(4 + Hkv) * d].view(N, Hkv, d), x[:, (4 + Hkv) * d:].view(N, Hkv, d)
    elif layout == "heads_first":
        k, v = (torch.randn((Hkv, N, d), dtype=dt(dtype), device="cuda", generator=g).transpose(0, 1) for _ in range(2))
    else:
        k, v = (torch.randn((N, Hkv, d), dtype=dt(dtype), device="cuda", generator=g) for _ in range(2))
    slots = torch.randperm(num * ps, device="cuda", generator=g)[:N].to(torch.int32)
    slots[3::5] = -1
    want_k, want_v = kc.clone(), vc.clone()
    for n, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // ps, :, s % ps] = k[n]
            want_v[s // ps, :, s % ps] = v[n]
    jl.cache_append(k, v, slots, kc, vc)
    jl.device_status()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


# ------------------------------------------------------------------ block_tables
@pytest.mark.parametrize("B,ps,wide,pages,most", [(1, 16, 4, 9, 20), (3, 32, 6, 14, 70), (40, 16, 9, 200, 60),
                                                  (700, 64, 5, 1500, 130), (2000, 16, 3, 3000, 9), (8192, 16, 2, 9000, 3)])
@pytest.mark.parametrize("in_place", [True, False])
def test_tables_over_many_steps(B, ps, wide, pages, most, in_place):
    """Requests grow, are refused, finish and start again; every step equals the
    plain one, and no page ever has two owners."""
    g = np.random.default_rng([B, ps])
    ref = R.Tables([[0] * wide for _ in range(B)], [0] * B, [0] * B, [int(x) for x in g.permutation(pages)], ps)
    table, free = ints(ref.table), ints(ref.free + [0] * 0)
    lens, held, count = ints([0] * B), ints([0] * B), ints([pages])
    for step in range(6):
        grow = [int(x) for x in g.integers(0, most + 1, B)]
        release = [int(x) for x in (g.random(B) < 0.2)] if step % 2 else [0] * B
        n_rows = sum(grow) + (5 if step % 3 else 0)
        out = dict(lens_out=lens, held_out=held, free_count_out=count) if in_place else {}
        r = jl.block_tables(lens, ints(grow), table, held, free, count, page_size=ps, num_pages=pages, n_rows=n_rows,
                            release=ints(release) if step % 2 else None, **out)
        jl.device_status()
        slots, starts, status = ref.step(grow, release, n_rows)
        assert r.slot_map.tolist() == slots and r.row_start.tolist() == starts and r.status.tolist() == status
        assert r.lens.tolist() == ref.lens and r.held.tolist() == ref.held
        n = int(r.free_count)
        assert free[:n].tolist() == ref.free
        got = table.tolist()
        owned = [got[b][c] for b in range(B) for c in range(ref.held[b])]
        assert got == [a[:] for a in got] and owned == [ref.table[b][c] for b in range(B) for c in range(ref.held[b])]
        assert sorted(owned + ref.free) == list(range(pages))
        # what was granted becomes committed
        ref.lens = [a + (x if s == 0 else 0) for a, x, s in zip(ref.lens, grow, status)]
        lens, held, count = ints(ref.lens), r.held, r.free_count


def test_tables_of_a_long_prompt():
    """One request with more rows than any block: a million slots."""
    ps, rows = 16, 1_000_003
    pages = -(-rows // ps) + 5
    order = np.random.default_rng(2).permutation(pages)
    r = jl.block_tables(ints([0, 0]), ints([rows, 1]), ints(np.zeros((2, pages))), ints([0, 0]), ints(order), ints([pages]),
                        page_size=ps, num_pages=pages, n_rows=rows + 1)
    jl.device_status()
    mine = order[::-1][:-(-rows // ps)]
    n = np.arange(rows)
    assert np.array_equal(r.slot_map.cpu().numpy()[:rows], mine[n // ps] * ps + n % ps)
    assert r.held.tolist() == [-(-rows // ps), 1] and r.status.tolist() == [0, 0]


# ------------------------------------------------------------------ tree_commit
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 9, 64])
@pytest.mark.parametrize("kind", ["chain", "random", "comb"])
def test_commit(dtype, T, kind):
    import torch
    g = np.random.default_rng([T, 7])
    lens, nodes = [0, 30, 100, 5, 77], [T, max(1, T // 2), T, 0, T]
    pool = Pool(41, [a + t for a, t in zip(lens, nodes)], 2, 64, 16, dtype)
    par = [random_parents(g, t, kind) for t in nodes]
    last = [T - 1, nodes[1] - 1, -1, -1, T // 2]
    want_k, want_v = pool.kc.clone(), pool.vc.clone()
    counts = []
    for b, (L, n) in enumerate(zip(lens, last)):
        path = []
        while n >= 0:
            path.append(n)
            n = par[b][n]
        path.reverse()
        counts.append(len(path))
        for cache, want in ((pool.kc, want_k), (pool.vc, want_v)):
            for j, x in enumerate(path):
                s, t = L + x, L + j
                want[pool.table[b][t // 16], :, t % 16] = cache[pool.table[b][s // 16], :, s % 16]
    flat = ints([x for p in par for x in p])
    # rows nobody owns hold NaN: compare bit patterns
    view = (lambda t: t.view(torch.int16)) if dtype == "bf16" else (lambda t: t.view(torch.int32))
    n, acc = jl.tree_commit(pool.kc, pool.vc, pool.tab, ints(lens), ints(starts_of(nodes)), flat, ints(last), max_nodes=T)
    jl.device_status()
    assert torch.equal(view(pool.kc), view(want_k)) and torch.equal(view(pool.vc), view(want_v))
    assert acc.tolist() == counts and n.tolist() == [a + c for a, c in zip(lens, counts)]


# ------------------------------------------------------------------ out-of-range device values
def test_out_of_range_values_are_reported_and_not_followed():
    import torch
    lens, nodes = [40, 20], [3, 2]
    pool = Pool(51, [a + t for a, t in zip(lens, nodes)], 1, 64, 16, "bf16")
    q = queries(51, 5, 2, 64, "bf16")
    kw = dict(max_nodes=3, w0=8, w_pretrained=30, rope_theta=1e4)
    rs = starts_of(nodes)

    def status(match):
        with pytest.raises(jl.JetLongError, match=match):
            jl.device_status()
        jl.device_status()

    good = jl.decode_tree(q, pool.kc, pool.vc, pool.tab, ints(lens), ints(rs), **kw)
    jl.device_status()

    def run(table=None, lens_=lens, rows=rs, parents=None):
        out = torch.full_like(q, 7.5)
        jl.decode_tree(q, pool.kc, pool.vc, pool.tab if table is None else table, ints(lens_), ints(rows), parents, out, **kw)
        return out

    for page in (-1, pool.num, 2 ** 31 - 1, -2 ** 31):
        bad = pool.tab.clone()
        bad[0, 1] = page
        out = run(table=bad)
        status("page number")
        assert torch.equal(out[3:], good[3:])
    for bad_lens in ([-3, 20], [2 ** 31 - 1, 20], [10 ** 6, 20]):
        out = run(lens_=bad_lens)
        status("length")
        assert (out[:3] == 7.5).all() and torch.equal(out[3:], good[3:])
    for bad_rows in ([0, -1, 2], [0, 4, 6], [3, 0, 2], [-2, 0, 2], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1 - 4]):
        run(rows=bad_rows)
        status("row_start")
    out = run(parents=ints([-1, 5, -7, -1, 0]))  # taken as -1
    status("parent")
    assert torch.equal(out, run(parents=ints([-1, -1, -1, -1, 0])))
    # slots
    k = torch.randn((3, 1, 64), device="cuda").bfloat16()
    kc, vc = torch.zeros_like(pool.kc), torch.zeros_like(pool.vc)
    jl.cache_append(k, k, ints([-2, pool.num * 16, 5]), kc, vc)
    status("slot")
    assert int((kc != 0).any(-1).sum()) == 1 and torch.equal(kc[0, :, 5], k[2])
    # commit
    for bad_last in ([3, -1], [-2, -1]):
        n, acc = jl.tree_commit(kc, vc, pool.tab, ints(lens), ints(rs), None, ints(bad_last), max_nodes=3)
        status("node or parent")
        assert acc.tolist() == [0, 0] and n.tolist() == lens
    # tables: a free count beyond the list, a negative length, a page number outside the pool
    t = lambda **k2: jl.block_tables(**{**dict(lens=ints([0]), grow=ints([1]), block_table=ints([[0, 0]]), held=ints([0]),
                                               free_list=ints([0, 1]), free_count=ints([2]), page_size=16, num_pages=2,
                                               n_rows=1), **k2})
    t(free_count=ints([3]))
    status("free_count")
    t(lens=ints([-4]))
    status("length")
    assert t(free_list=ints([0, 9])).slot_map.tolist() == [-1]
    status("page number")
    t(grow=ints([2]))
    status("row count")


# ------------------------------------------------------------------ together
def test_generation_with_drafts_over_the_paged_cache():
    """Requests of different lengths draft trees, attend, accept a path and go on,
    one joining late and one finishing: every accepted row's output equals the
    one-row decode of the same sequence in a contiguous cache."""
    import torch
    g = np.random.default_rng(61)
    B, Hq, Hkv, d, ps, wide = 3, 8, 2, 128, 16, 24
    kw = dict(w0=24, w_pretrained=40, rope_theta=1e4)
    pages = B * wide
    kc = torch.full((pages, Hkv, ps, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    table, free, count = ints(np.zeros((B, wide))), ints(g.permutation(pages)), ints([pages])
    lens, held = ints([0] * B), ints([0] * B)
    seqs = [([], []) for _ in range(B)]  # committed rows of each request
    checked = 0
    for step in range(9):
        release = [0] * B
        if step == 5:
            release[1] = 1
            seqs[1] = ([], [])
        if step == 0:
            nodes = [37, 0, 1]     # prompts (a chain of up to 64 rows is a prompt chunk)
        elif step == 1:
            nodes = [6, 50, 1]
        else:
            nodes = [int(x) for x in g.integers(0, 12, B)]
        prompt = step < 2
        par = [[t - 1 for t in range(n)] if prompt else random_parents(g, n, "random") for n in nodes]
        N = sum(nodes)
        if N == 0:
            continue
        q, k, v = (torch.from_numpy(g.standard_normal((N, h, d), dtype=np.float32)).cuda().bfloat16() for h in (Hq, Hkv, Hkv))
        r = jl.block_tables(lens, ints(nodes), table, held, free, count, page_size=ps, num_pages=pages, n_rows=N,
                            release=ints(release), lens_out=lens, held_out=held, free_count_out=count)
        assert r.status.tolist() == [0] * B
        jl.cache_append(k, v, r.slot_map, kc, vc)
        out = jl.decode_tree(q, kc, vc, table, lens, r.row_start, ints([x for p in par for x in p]), max_nodes=64, **kw)
        last = [n - 1 if prompt else int(g.integers(-1, n)) if n else -1 for n in nodes]
        jl.tree_commit(kc, vc, table, lens, r.row_start, ints([x for p in par for x in p]), ints(last), max_nodes=64,
                       lens_out=lens)
        jl.device_status()
        at = 0
        for b in range(B):
            path, x = [], last[b]
            while x >= 0:
                path.append(x)
                x = par[b][x]
            for x in reversed(path):
                seqs[b][0].append(k[at + x])
                seqs[b][1].append(v[at + x])
                L = len(seqs[b][0])
                kk, vv = (torch.stack(s, 1)[None].contiguous() for s in seqs[b])
                ref = jl.decode(q[at + x][None].contiguous(), kk, vv, L, **kw)
                _, tol = R.attend(to64(q[at + x])[None], to64(kk)[0][None], to64(vv)[0][None], [0] * L, L - 1, [-1], w0=24,
                                  w_pre=40, theta=1e4, scale=d ** -0.5, dtype="bf16")
                assert (np.abs(to64(out[at + x]) - to64(ref[0])) <= 2 * tol[0]).all(), (step, b, x)
                checked += 1
            at += nodes[b]
        assert lens.tolist() == [len(s[0]) for s in seqs]
    assert checked > 100


@pytest.mark.parametrize("dtype,nodes,codes", [("bf16", 1, (0x601, 0x641)), ("bf16", 8, (0x601, 0x641)),
                                               # 48, 160 rows a kv head: the kernel for more than 32
                                               ("bf16", 12, (0x501, 0x641)), ("bf16", 40, (0x501, 0x641)), ("fp32", 1, (0x701, 0x711)),
                                               ("fp32", 12, (0x701, 0x711))])
def test_expired_wait_is_reported_and_the_context_recovers(dtype, nodes, codes):
    """The first key tile is never loaded and every wait is limited to about a
    millisecond: the launch ends by itself, says so, and leaves nothing behind."""
    import torch
    jl.device_status()
    lens, Hq, Hkv, d = [2000, 700, 5], 8, 2, 128
    pool = Pool(61, [L + nodes for L in lens], Hkv, d, 64, dtype)
    N = 3 * nodes
    q = queries(61, N, Hq, d, dtype)
    par = random_parents(np.random.default_rng(61), nodes, "random")
    args = (q, pool.kc, pool.vc, pool.tab, ints(lens), ints([0, nodes, 2 * nodes, N]), ints(par * 3))
    kw = dict(max_nodes=nodes, w0=64, w_pretrained=400, rope_theta=1e4)
    before = jl.decode_tree(*args, **kw)
    jl.device_status()
    jl.debug_inject_timeout(jl.INJECT_DECODE_COPY, 2_000_000)
    jl.decode_tree(*args, **kw)
    with pytest.raises(jl.JetLongError) as ei:
        jl.device_status()
    assert ei.value.status == 4, str(ei.value)  # JETLONG_ERR_TIMEOUT
    msg = str(ei.value)
    assert codes[0] <= int(msg[msg.index("code 0x") + 5:].split(")")[0], 16) <= codes[1], msg
    jl.device_status()
    again = jl.decode_tree(*args, **kw)
    jl.device_status()
    assert torch.equal(again, before)


def test_captured_step_follows_growing_requests():
    """One decode step (tables, append, attention, lengths) captured once and
    replayed: lengths, tables and pages advance on the device."""
    import torch
    g = np.random.default_rng(71)
    B, Hq, Hkv, d, ps, wide, steps = 3, 8, 2, 128, 16, 8, 40
    kw = dict(w0=10, w_pretrained=25, rope_theta=1e4)
    pages = B * wide
    kc = torch.full((pages, Hkv, ps, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    table, free, count = ints(np.zeros((B, wide))), ints(g.permutation(pages)), ints([pages])
    start = [0, 15, 60]
    lens, held, grow = ints([0] * B), ints([0] * B), ints(start)
    state = dict(lens_out=lens, held_out=held, free_count_out=count)
    ks, vs = ([torch.from_numpy(g.standard_normal((n, Hkv, d), dtype=np.float32)).cuda().bfloat16() for n in start]
              for _ in range(2))
    r = jl.block_tables(lens, grow, table, held, free, count, page_size=ps, num_pages=pages, n_rows=sum(start), **state)
    jl.cache_append(torch.cat(ks), torch.cat(vs), r.slot_map, kc, vc)
    lens += grow
    one = ints([1] * B)
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(jl.decode_tree_workspace_size(B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    bufs = dict(slot_map=ints([0] * B), row_start=ints([0] * (B + 1)), status=ints([0] * B))

    def step():
        t = jl.block_tables(lens, one, table, held, free, count, page_size=ps, num_pages=pages, n_rows=B, **state, **bufs)
        jl.cache_append(k, v, t.slot_map, kc, vc)
        jl.decode_paged(q, kc, vc, table, lens, out, workspace=ws, **kw)
        lens.add_(one)

    def check(x):
        torch.cuda.synchronize()
        jl.device_status()
        for b in range(B):
            ks[b], vs[b] = torch.cat([ks[b], x[1][b:b + 1]]), torch.cat([vs[b], x[2][b:b + 1]])
            L = ks[b].shape[0]
            ref, tol = R.attend(to64(x[0][b:b + 1]), to64(ks[b].transpose(0, 1))[None], to64(vs[b].transpose(0, 1))[None],
                                [0] * L, L - 1, [-1], w0=10, w_pre=25, theta=1e4, scale=d ** -0.5, dtype="bf16")
            assert (np.abs(to64(out[b]) - ref[0]) <= tol[0]).all(), (b, L)

    def fresh():
        x = [torch.from_numpy(g.standard_normal(t.shape, dtype=np.float32)).cuda().bfloat16() for t in (q, k, v)]
        for t, y in zip((q, k, v), x):
            t.copy_(y)
        return x

    side = torch.cuda.Stream()
    x = fresh()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(steps):
        x = fresh()
        graph.replay()
        check(x)
    assert lens.tolist() == [n + 1 + steps for n in start]
    del graph
