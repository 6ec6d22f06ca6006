"""Requests that take no part in a step of the paged cache: refused ones, idle
places, requests whose numbers are out of range.  Nothing of theirs is written, and
nobody else's rows are read for them or written by them."""
import numpy as np
import pytest

import paged_reference as R
import rope_context_extension_jet_b200 as jl
from test_paged import dt, ints, random_parents, starts_of, to64

pytestmark = pytest.mark.gpu

HQ, HKV, D, PS = 8, 2, 64, 16
KW = dict(w0=24, w_pretrained=40, rope_theta=1e4)


def bits(t):
    import torch
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


class Server:
    """A pool of pages and the requests on it; the host keeps every row it has committed."""

    def __init__(self, B, wide, pages, dtype="bf16", seed=1, free=None):
        import torch
        self.g = np.random.default_rng(seed)
        self.kc = torch.full((pages, HKV, PS, D), float("nan"), dtype=dt(dtype), device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        free = self.g.permutation(pages) if free is None else free
        self.free, self.count = ints(list(free) + [0] * (pages - len(free))), ints([len(free)])
        self.table, self.held, self.lens = ints(np.zeros((B, wide))), ints([0] * B), ints([0] * B)
        self.B, self.pages, self.dtype = B, pages, dtype
        self.rows = [([], []) for _ in range(B)]

    def randn(self, *shape):
        import torch
        return torch.from_numpy(self.g.standard_normal(shape, dtype=np.float32)).cuda().to(dt(self.dtype))

    def tables(self, grow, release=None):
        return jl.block_tables(self.lens, ints(grow), self.table, self.held, self.free, self.count, page_size=PS,
                               num_pages=self.pages, n_rows=max(0, sum(max(0, x) for x in grow)),
                               release=None if release is None else ints(release), lens_out=self.lens, held_out=self.held,
                               free_count_out=self.count)

    def step(self, nodes, last, release=None, kind="chain", report=None):
        """One whole step, checked against the rows the host has kept.  Returns (status, out)."""
        import torch
        par = [random_parents(self.g, n, kind) for n in nodes]
        flat = ints([x for p in par for x in p])
        N = sum(nodes)
        q, k, v = self.randn(N, HQ, D), self.randn(N, HKV, D), self.randn(N, HKV, D)
        out = torch.full_like(q, 7.5)
        before = [self.lens.tolist(), bits(self.kc).clone(), bits(self.vc).clone()]
        r = self.tables(nodes, release)
        if release is not None:
            for b in range(self.B):
                if release[b]:
                    self.rows[b] = ([], [])
        status, lens = r.status.tolist(), self.lens.tolist()
        jl.cache_append(k, v, r.slot_map, self.kc, self.vc)
        mid = bits(self.kc).clone(), bits(self.vc).clone()
        jl.decode_tree(q, self.kc, self.vc, self.table, self.lens, r.row_start, flat, out, max_nodes=64, **KW)
        _, acc = jl.tree_commit(self.kc, self.vc, self.table, self.lens, r.row_start, flat, ints(last), max_nodes=64,
                                lens_out=self.lens)
        if report:
            with pytest.raises(jl.JetLongError, match=report):
                jl.device_status()
        jl.device_status()
        want_k, want_v = mid[0].clone(), mid[1].clone()
        at, table = 0, self.table.tolist()
        for b, n in enumerate(nodes):
            if status[b]:
                assert (out[at:at + n] == 7.5).all(), ("rows of a refused request were written", b)
                assert int(acc[b]) == 0 and int(self.lens[b]) == before[0][b]
            else:
                L, path, x = lens[b], [], last[b]
                while x >= 0:
                    path.append(x)
                    x = par[b][x]
                path.reverse()
                if n:
                    own = [torch.stack(self.rows[b][i] + list((k, v)[i][at:at + n])) for i in range(2)]  # [L + n, HKV, D]
                    k64, v64 = (to64(x)[:, :, None] for x in own)  # pages of one row
                    ref, tol = R.attend(to64(q[at:at + n]), k64, v64, list(range(L + n)), L, par[b], w0=KW["w0"],
                                        w_pre=KW["w_pretrained"], theta=KW["rope_theta"], scale=D ** -0.5, dtype=self.dtype)
                    assert (np.abs(to64(out[at:at + n]) - ref) <= tol).all(), b
                assert int(acc[b]) == len(path) and int(self.lens[b]) == L + len(path)
                for j, x in enumerate(path):
                    self.rows[b][0].append(k[at + x])
                    self.rows[b][1].append(v[at + x])
                    for want, old in ((want_k, mid[0]), (want_v, mid[1])):
                        s, t = L + x, L + j
                        want[table[b][t // PS], :, t % PS] = old[table[b][s // PS], :, s % PS]
            at += n
        # the commit has moved what it should and nothing else
        assert torch.equal(bits(self.kc), want_k) and torch.equal(bits(self.vc), want_v)
        return status, out


# ------------------------------------------------------------------ refused
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("grow", [12, 60])
def test_refused_requests_stay_out_of_the_whole_step(dtype, grow):
    """The free pages end in the middle of a batch.  The table rows of the refused requests
    hold other requests' pages behind their own: those are neither attended nor written, and
    once pages are free again the request goes on where it was."""
    s = Server(4, 8, 12, dtype)
    s.table.copy_(ints([[s.g.integers(0, 12) for _ in range(8)] for _ in range(4)]))
    assert s.step([30, 14, 31, 10], [29, 13, 30, 9])[0] == [0, 0, 0, 0]     # 2 + 1 + 2 + 1 pages; 6 left
    assert s.step([50, grow, 20, 3], [49, grow - 1, 19, 2])[0] == [0, 0 if grow == 12 else 1, 0 if grow == 12 else 1, 0]
    if grow == 12:                                                          # 3 + 1 + 2: none left
        assert s.step([3, 9, 20, 2], [2, 8, 19, 1], kind="random")[0] == [1, 1, 1, 0]
    else:                                                                   # 3 left
        assert s.step([0, 60, 1, 60], [-1, 59, 0, 59], kind="random")[0] == [0, 1, 0, 1]
        assert s.step([5, 64, 60, 3], [4, 63, 59, 2], kind="star")[0][1:3] == [1, 1]
    assert s.step([0, 9, 2, 1], [-1, 8, 1, 0], release=[1, 0, 0, 0], kind="comb")[0] == [0, 0, 0, 0]
    s.step([20, 4, 6, 9], [11, 3, 5, 8], kind="random")


def test_a_refused_request_in_decode_paged():
    import torch
    s = Server(3, 4, 4)
    assert s.step([16, 32, 5], [15, 31, 4])[0] == [0, 0, 0]
    s.table[0, 1:] = s.table[1, 0]
    r = s.tables([1, 1, 1])
    assert r.status.tolist() == [1, 1, 0] and r.slot_map.tolist()[:2] == [-1, -1]
    q, k, v = s.randn(3, HQ, D), s.randn(3, HKV, D), s.randn(3, HKV, D)
    jl.cache_append(k, v, r.slot_map, s.kc, s.vc)
    out = jl.decode_paged(q, s.kc, s.vc, s.table, s.lens, torch.full_like(q, 7.5), **KW)
    jl.device_status()
    assert (out[:2] == 7.5).all() and (out[2] != 7.5).all()


def test_a_request_longer_than_its_table_stays_out_and_is_reported():
    s = Server(2, 2, 8)
    assert s.step([30, 9], [29, 8])[0] == [0, 0]
    assert s.step([3, 2], [2, 1], report="length")[0] == [2, 0]
    assert s.step([2, 2], [1, 1])[0] == [0, 0]


def test_captured_step_with_trees_refusals_and_idle_places():
    """Tables, append, tree attention and commit captured once and replayed.  The pool is too
    small: requests are refused and go on when others release their pages; places are idle,
    and filled again."""
    import torch
    g = np.random.default_rng(5)
    B, wide, T, steps = 5, 6, 6, 40
    s = Server(B, wide, 5, seed=6)
    s.table.copy_(ints(g.integers(0, 5, (B, wide))))
    N = B * T
    grow, release, last, flat = ints([0] * B), ints([0] * B), ints([-1] * B), ints([-1] * N)
    q, k, v = s.randn(N, HQ, D), s.randn(N, HKV, D), s.randn(N, HKV, D)
    out, acc = torch.zeros_like(q), ints([0] * B)
    bufs = dict(slot_map=ints([0] * N), row_start=ints([0] * (B + 1)), status=ints([0] * B))
    ws = torch.empty(jl.decode_tree_workspace_size(B, HQ, HKV, D, T), dtype=torch.uint8, device="cuda")

    def step():
        r = jl.block_tables(s.lens, grow, s.table, s.held, s.free, s.count, page_size=PS, num_pages=s.pages, n_rows=N,
                            release=release, lens_out=s.lens, held_out=s.held, free_count_out=s.count, **bufs)
        jl.cache_append(k, v, r.slot_map, s.kc, s.vc)
        jl.decode_tree(q, s.kc, s.vc, s.table, s.lens, r.row_start, flat, out, max_nodes=T, workspace=ws, **KW)
        jl.tree_commit(s.kc, s.vc, s.table, s.lens, r.row_start, flat, last, max_nodes=T, lens_out=s.lens, n_accepted=acc)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    seen = {"refused": 0, "idle": 0, "granted": 0}
    idle = [False] * B
    for n in range(steps):
        nodes, rel = [int(x) for x in g.integers(0, T + 1, B)], [0] * B
        lens = s.lens.tolist()
        for b in range(B):
            if idle[b]:
                if g.random() < 0.4:  # a new request in this place
                    idle[b], rel[b], nodes[b] = False, 1, max(1, nodes[b])
                else:
                    nodes[b] = 0
            elif lens[b] > 60 or g.random() < 0.05:
                idle[b], nodes[b], rel[b] = True, 0, 1
                lens[b] = -1
            if rel[b]:
                s.rows[b] = ([], [])
        s.lens.copy_(ints(lens))
        par = [random_parents(g, x, "random") for x in nodes]
        lst = [int(g.integers(-1, x)) if x else -1 for x in nodes]
        at = starts_of(nodes)
        flat.copy_(ints([x for p in par for x in p] + [-1] * (N - at[-1])))
        for t, x in ((grow, nodes), (release, rel), (last, lst)):
            t.copy_(ints(x))
        for t in (q, k, v):
            t.copy_(s.randn(*t.shape))
        out.fill_(7.5)
        graph.replay()
        jl.device_status()
        status, now = bufs["status"].tolist(), s.lens.tolist()
        assert (out[at[-1]:] == 7.5).all()
        for b in range(B):
            L, rows = 0 if rel[b] and not idle[b] else lens[b], slice(at[b], at[b + 1])
            if idle[b]:
                assert now[b] == -1 and status[b] == 0 and int(acc[b]) == 0
                seen["idle"] += 1
                continue
            if status[b]:
                assert status[b] == 1 and now[b] == L and int(acc[b]) == 0 and (out[rows] == 7.5).all(), (n, b)
                seen["refused"] += 1
                continue
            path, x = [], lst[b]
            while x >= 0:
                path.append(x)
                x = par[b][x]
            assert now[b] == L + len(path) and int(acc[b]) == len(path) and L == len(s.rows[b][0]), (n, b)
            if nodes[b]:
                own = [torch.stack(s.rows[b][i] + list((k, v)[i][rows])) for i in range(2)]
                ref, tol = R.attend(to64(q[rows]), *(to64(x)[:, :, None] for x in own), list(range(L + nodes[b])), L, par[b],
                                    w0=KW["w0"], w_pre=KW["w_pretrained"], theta=KW["rope_theta"], scale=D ** -0.5, dtype="bf16")
                assert (np.abs(to64(out[rows]) - ref) <= tol).all(), (n, b)
                seen["granted"] += 1
            for x in reversed(path):
                s.rows[b][0].append(k[at[b] + x].clone())
                s.rows[b][1].append(v[at[b] + x].clone())
    assert min(seen.values()) > 10, seen
    del graph


# ------------------------------------------------------------------ idle
@pytest.mark.parametrize("in_place", [True, False])
def test_idle_places_pass_through_a_step(in_place):
    """lens[b] < 0 and no new rows: the place keeps its length (and its pages, unless it
    releases them), and no call reports it."""
    import torch
    s = Server(4, 4, 10)
    assert s.step([20, 3, 18, 7], [19, 2, 17, 6])[0] == [0] * 4
    s.lens[1], s.lens[2] = -1, -7
    lens = s.lens.clone()
    out = dict(lens_out=s.lens, held_out=s.held, free_count_out=s.count) if in_place else {}
    r = jl.block_tables(s.lens, ints([1, 0, 0, 1]), s.table, s.held, s.free, s.count, page_size=PS, num_pages=s.pages, n_rows=2,
                        release=ints([0, 0, 1, 0]), **out)
    jl.device_status()
    assert r.lens.tolist() == lens.tolist() and r.status.tolist() == [0] * 4 and r.row_start.tolist() == [0, 1, 1, 1, 2]
    assert r.held.tolist() == [2, 1, 0, 1] and int(r.free_count) == 10 - 4
    q = s.randn(4, HQ, D)
    o = jl.decode_paged(q, s.kc, s.vc, s.table, r.lens, torch.full_like(q, 7.5), **KW)
    n, acc = jl.tree_commit(s.kc, s.vc, s.table, r.lens, r.row_start, None, ints([0, -1, -1, 0]), max_nodes=1)
    jl.device_status()
    assert (o[1:3] == 7.5).all() and n.tolist() == [21, -1, -7, 8] and acc.tolist() == [1, 0, 0, 1]


# ------------------------------------------------------------------ out of range
BAD = [dict(lens=-4, grow=1), dict(lens=-4, grow=40), dict(grow=-1), dict(grow=-2 ** 31), dict(held=-1), dict(held=5),
       dict(held=2 ** 31 - 1), dict(held=5, release=1), dict(held=-3, release=1), dict(grow=-5, release=1),
       dict(lens=-2, grow=-1), dict(lens=-2 ** 31, grow=2 ** 31 - 1)]


@pytest.mark.parametrize("bad", BAD, ids=lambda x: ",".join(f"{k}={v}" for k, v in x.items()))
@pytest.mark.parametrize("place", [0, 1, 2])
def test_tables_leave_out_of_range_requests_as_they_are(bad, place):
    """Such a request takes no page and gives none back; its length, its pages and its table
    row stay (but new rows behind its committed pages have no page), its status is 3, and
    the others go on as without it."""
    wide, pages = 4, 16
    lens, grow, held, release = [20, 5, 33], [7, 20, 2], [2, 1, 3], [0, 0, 0]
    table = [[3, 4, 9, 9], [5, 9, 9, 9], [6, 7, 8, 9]]
    free = [15, 14, 13, 12, 11]
    for k, v in bad.items():
        {"lens": lens, "grow": grow, "held": held, "release": release}[k][place] = v
    ref = R.Tables(table, lens, held, free, PS)
    rows = max(0, grow[place])
    big = rows > 1000
    use = [0 if b == place else grow[b] for b in range(3)]
    ref.lens[place] = ref.held[place] = 0
    slots, _, status = ref.step(use, [0] * 3, 0)
    n_rows = 100
    t, f = ints(table), ints(free + [-1] * 11)
    r = jl.block_tables(ints(lens), ints(grow), t, ints(held), f, ints([5]), page_size=PS, num_pages=pages, n_rows=n_rows,
                        release=ints(release))
    with pytest.raises(jl.JetLongError, match="length|row count" if big else "length"):
        jl.device_status()
    jl.device_status()
    status[place] = 3
    assert r.status.tolist() == status
    if lens[place] >= 0 and grow[place] > 0:
        last = (lens[place] + grow[place] - 1) // PS
        if last > (lens[place] - 1) // PS:
            table[place][last] = jl.NO_PAGE
    for b in range(3):
        keep = b == place
        assert int(r.lens[b]) == lens[b] and int(r.held[b]) == (held[b] if keep else ref.held[b])
        assert t[b].tolist() == (table[b] if keep else ref.table[b])
    n = int(r.free_count)
    assert f[:n].tolist() == ref.free
    # its token rows are counted and have no slot
    if not big:
        counts = [max(0, x) for x in grow]
        assert r.row_start.tolist() == starts_of(counts)
        want, it = [], iter(slots)
        for b in range(3):
            want += [-1] * counts[b] if b == place else [next(it) for _ in range(counts[b])]
        assert r.slot_map.tolist() == want + [-1] * (n_rows - len(want))


def test_pages_out_of_range_are_not_handed_on():
    """A page number outside the pool, in a table row given back or in the free list, is
    reported, and is nobody's page afterwards."""
    import torch
    bad = [99, -5, 2 ** 31 - 1]
    for x in bad:
        t, f = ints([[3, x, 4], [0, 0, 0]]), ints([7, 6, 0, 0, 0, 0, 0, 0])
        r = jl.block_tables(ints([40, 0]), ints([0, 0]), t, ints([3, 0]), f, ints([2]), page_size=PS, num_pages=8, n_rows=0,
                            release=ints([1, 0]))
        with pytest.raises(jl.JetLongError, match="page number"):
            jl.device_status()
        assert int(r.free_count) == 5 and f[:5].tolist() == [7, 6, 4, jl.NO_PAGE, 3]
    s = Server(2, 4, 8, free=[0, 1, 2, 99, 4])
    s.kc.zero_(), s.vc.zero_()
    r = s.tables([16, 20])  # pages 4, then 99 and 2
    with pytest.raises(jl.JetLongError, match="page number"):
        jl.device_status()
    assert s.table.tolist()[1][:2] == [jl.NO_PAGE, 2] and s.table.tolist()[0][0] == 4
    assert r.slot_map.tolist() == [64 + x for x in range(16)] + [-1] * 16 + [32 + x for x in range(4)]


@pytest.mark.parametrize("page", [-1, 50, 2 ** 31 - 1, -2 ** 31])
def test_commit_leaves_out_a_request_with_a_bad_page(page):
    """Rows that cannot be moved are not committed: the request stays as it was."""
    import torch
    s = Server(3, 4, 10)
    assert s.step([14, 30, 20], [13, 29, 19])[0] == [0] * 3
    r = s.tables([9, 6, 3])
    k, v = s.randn(18, HKV, D), s.randn(18, HKV, D)
    jl.cache_append(k, v, r.slot_map, s.kc, s.vc)
    par = ints([-1, 0, 0, 1, 1, 3, 3, 5, 5] + [-1, 0, 0, 0, 0, 0] + [-1, 0, 1])
    s.table[0, 1] = page
    before = bits(s.kc).clone(), bits(s.vc).clone()
    n, acc = jl.tree_commit(s.kc, s.vc, s.table, s.lens, r.row_start, par, ints([8, -1, -1]), max_nodes=9)
    with pytest.raises(jl.JetLongError, match="page number"):
        jl.device_status()
    assert n.tolist() == [14, 30, 20] and acc.tolist() == [0, 0, 0]
    assert torch.equal(bits(s.kc), before[0]) and torch.equal(bits(s.vc), before[1])


def test_commit_leaves_out_a_request_with_a_bad_parent():
    import torch
    s = Server(2, 4, 10)
    assert s.step([14, 30], [13, 29])[0] == [0, 0]
    r = s.tables([5, 4])
    k, v = s.randn(9, HKV, D), s.randn(9, HKV, D)
    jl.cache_append(k, v, r.slot_map, s.kc, s.vc)
    for x in (2, 3, -2, 2 ** 31 - 1, -2 ** 31):  # of node 2
        before = bits(s.kc).clone(), bits(s.vc).clone()
        n, acc = jl.tree_commit(s.kc, s.vc, s.table, s.lens, r.row_start, ints([-1, 0, x, 2, 3] + [-1, 0, 1, 2]), ints([4, 3]),
                                max_nodes=9)
        with pytest.raises(jl.JetLongError, match="parent"):
            jl.device_status()
        assert n.tolist() == [14, 34] and acc.tolist() == [0, 4]
        assert torch.equal(bits(s.kc), before[0]) and torch.equal(bits(s.vc), before[1])  # (a chain's rows stay in place)
