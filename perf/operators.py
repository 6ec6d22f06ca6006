"""Timing cases of the paged-cache operators: block tables and slot maps, cache
append, decode over a paged cache (one new token, or a tree of drafted tokens),
and the commit of an accepted draft.

The method is the library's: unrotated key rows, pairs closer than w0 rotated to
their exact positions, all others to floor(x / G) with G = max(1, ceil(L /
w_pretrained)) of the query's own length L = position + 1.  Caches are pages
[num_pages, Hkv, page_size, d]; table[b][p] is the page of request b's rows
[p page_size, (p + 1) page_size).
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small running batch: every request takes one more row
        dict(name="tables_step", op="tables", B=16, top=8192, grow="one", release=0, ps=64, mix=1),
        # a scheduler step that mixes decoding requests, prompt chunks and finished requests
        dict(name="tables_prompts", op="tables", B=512, top=131072, grow="chunks", release=1, ps=16, mix=2),
        # the rows of one decode step, as slices of a fused q/k/v projection
        dict(name="append_step", op="append", N=16, Hq=32, Hkv=8, d=128, ps=64, dtype="bf16", fused=True),
        # a prompt chunk written to the pages
        dict(name="append_prompt", op="append", N=32768, Hq=32, Hkv=8, d=128, ps=64, dtype="bf16", fused=True),
        # one user, a short conversation: latency
        dict(name="paged_one_short", op="paged", B=1, top=1000, ragged=False, Hq=32, Hkv=8, d=128, ps=64,
             dtype="bf16", w0=4096, w_pre=32768, theta=1e6, mix=3),
        # eight users at 128K, where G goes from 4 to 5
        dict(name="paged_b8_128k", op="paged", B=8, top=131072, ragged=False, Hq=32, Hkv=8, d=128, ps=64,
             dtype="bf16", w0=4096, w_pre=32768, theta=1e6, mix=4),
        # a batch of very different lengths in fp32, small pages, head dim 64
        dict(name="paged_ragged_fp32", op="paged", B=7, top=16383, ragged=True, Hq=6, Hkv=2, d=64, ps=16,
             dtype="fp32", w0=512, w_pre=4096, theta=1e4, mix=5),
        # one user, a drafted chain of four tokens over a short cache
        dict(name="tree_one_chain", op="tree", B=1, top=4093, ragged=False, T=4, chain=True, Hq=32, Hkv=8, d=128,
             ps=64, dtype="bf16", w0=4096, w_pre=32768, theta=1e6, mix=6),
        # sixteen users of different lengths with trees of up to 24 tokens
        dict(name="tree_ragged", op="tree", B=16, top=32780, ragged=True, T=24, chain=False, Hq=16, Hkv=8, d=128,
             ps=128, dtype="bf16", w0=4096, w_pre=32768, theta=1e6, mix=7),
        # the largest trees at 128K: 64 tokens, 256 query rows per kv head
        dict(name="tree_b8_128k", op="tree", B=8, top=131060, ragged=False, T=64, chain=False, Hq=32, Hkv=8, d=128,
             ps=64, dtype="bf16", w0=4096, w_pre=32768, theta=1e6, mix=8),
        # accepted paths of a small batch
        dict(name="commit_step", op="commit", B=8, top=4096, T=32, Hkv=8, d=128, ps=64, dtype="bf16", mix=9),
        # accepted paths of a large batch in fp32
        dict(name="commit_batch", op="commit", B=256, top=900, T=64, Hkv=8, d=128, ps=16, dtype="fp32", mix=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "paged", "paged", "tree", "tree", "commit"])
    mix = rng.randrange(1 << 30)
    ps = rng.choice([16, 32, 64, 128, 256])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 512), top=_log(rng, 64, 131072), grow=rng.choice(["one", "chunks"]),
                    release=rng.randrange(2), ps=ps, mix=mix)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 7, 8])
    if op == "append":
        return dict(op=op, N=_log(rng, 1, 16384), Hq=Hkv * group, Hkv=Hkv, d=d, ps=ps, dtype=dtype,
                    fused=rng.random() < 0.5)
    if op == "commit":
        return dict(op=op, B=_log(rng, 1, 256), top=_log(rng, 1, 900), T=_log(rng, 1, 64), Hkv=Hkv, d=d, ps=ps,
                    dtype=dtype, mix=mix)
    w_pre = rng.choice([4096, 8192, 32768])
    T = _log(rng, 1, 64) if op == "tree" else 1
    # rows of the cache in all, so that no case costs more than the largest listed one
    B = _log(rng, 1, 64)
    budget = (1 << 20) if dtype == "bf16" else (1 << 17)
    top = _log(rng, 1, max(1, min(131072, budget // B)))
    case = dict(op=op, B=B, top=top, ragged=rng.random() < 0.7, Hq=Hkv * group, Hkv=Hkv, d=d, ps=ps, dtype=dtype,
                w0=rng.choice([0, 1, 512, 4096]), w_pre=w_pre, theta=rng.choice([1e4, 1e6]), mix=mix)
    if op == "tree":
        case.update(T=T, chain=rng.random() < 0.25)
    return case


# ------------------------------------------------------------------ host-side shapes of a case
def _lens(case):
    """Rows each request holds before the step."""
    r = random.Random(case["mix"])
    if not case.get("ragged", True):
        return [case["top"]] * case["B"]
    return [_log(r, 1, case["top"]) - 1 if case["op"] == "tables" else _log(r, 1, case["top"])
            for _ in range(case["B"])]


def _nodes(case):
    """Drafted tokens of each request."""
    r = random.Random(case["mix"] + 1)
    if case["op"] == "paged":
        return [1] * case["B"]
    if not case.get("ragged", True):
        return [case["T"]] * case["B"]
    return [r.randint(max(1, case["T"] // 2), case["T"]) for _ in range(case["B"])]


def _growth(case):
    """(new rows, released) of each request of a table step."""
    r = random.Random(case["mix"] + 2)
    grow, rel = [], []
    for _ in range(case["B"]):
        gone = case["release"] and r.random() < 0.1
        rel.append(1 if gone else 0)
        if gone:
            grow.append(0)
        elif case["grow"] == "one":
            grow.append(1)
        else:
            grow.append(_log(r, 1, 2048) if r.random() < 0.3 else 1)
    return grow, rel


def _paths(case):
    """Accepted drafted tokens of each request (ascending node indices; may be empty)."""
    r = random.Random(case["mix"] + 3)
    out = []
    for T in _nodes(case):
        n = r.randint(0, min(T, 8))
        first = [0] if n else []
        rest = sorted(r.sample(range(n, T), min(n - 1, T - n))) if n > 1 else []
        out.append(first + rest)
    return out


def _pages(rows, ps):
    return (rows + ps - 1) // ps


def work(case):
    op = case["op"]
    if op == "tables":
        lens, (grow, _) = _lens(case), _growth(case)
        n = sum(grow)
        new = sum(_pages(a + g, case["ps"]) - _pages(a, case["ps"]) for a, g in zip(lens, grow))
        return {"bytes": 4 * n + 8 * new + 4 * 9 * case["B"], "flops": n}
    el = 2 if case["dtype"] == "bf16" else 4
    row = case["Hkv"] * case["d"] * el
    if op == "append":
        return {"bytes": case["N"] * (4 * row + 4), "flops": 0}
    if op == "commit":
        n = sum(len(p) for p in _paths(case))
        return {"bytes": 4 * n * row + 4 * sum(_nodes(case)) + 16 * case["B"], "flops": 0}
    lens, nodes = _lens(case), _nodes(case)
    rows = sum(a + t for a, t in zip(lens, nodes))
    pairs = sum(t * (a + (t + 1) // 2) for a, t in zip(lens, nodes))
    q = sum(nodes) * case["Hq"] * case["d"] * el
    return {"bytes": 2 * rows * row + 2 * q + 4 * _pages(rows, case["ps"]) + 8 * case["B"],
            "flops": 4 * case["d"] * case["Hq"] * pairs}


# ------------------------------------------------------------------ inputs
def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))


def _randn(shape, dtype, g):
    return torch.randn(shape, dtype=DT[dtype], device="cuda", generator=g)


def _pool(case, seed, rows):
    """A pool with room for `rows` rows per request, pages handed out in a shuffled order."""
    per = [_pages(n, case["ps"]) for n in rows]
    num_pages = sum(per) + 8
    order = torch.randperm(num_pages, generator=torch.Generator().manual_seed(77 * seed + 5)).tolist()
    wide = max(1, max(per)) + 1
    table, at = [], 0
    for p in per:
        table.append(order[at:at + p] + [0] * (wide - p))
        at += p
    return num_pages, table, order[at:]


def _parents(case, seed, nodes):
    """Each drafted token's parent within its request (-1: the last committed token)."""
    r = random.Random(91 * seed + case["mix"])
    out = []
    for T in nodes:
        for t in range(T):
            out.append(t - 1 if case.get("chain") or t == 0 else r.randint(max(0, (t - 1) // 4), t - 1))
    return out


def _starts(counts):
    s = [0]
    for c in counts:
        s.append(s[-1] + c)
    return s


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    st = dict(case=case)
    if op == "tables":
        lens, (grow, rel) = _lens(case), _growth(case)
        ps = case["ps"]
        num_pages, table, spare = _pool(case, seed, lens)
        want = sum(_pages(a + n, ps) - _pages(a, ps) for a, n in zip(lens, grow))
        extra = want + 16
        free = spare + list(range(num_pages, num_pages + extra))
        random.Random(seed).shuffle(free)
        num_pages += extra
        wide = max(_pages(a + n, ps) for a, n in zip(lens, grow)) + 1
        table = [(row + [0] * wide)[:wide] for row in table]
        room = free + [0] * (num_pages - len(free))
        st.update(lens=_int(lens), grow=_int(grow), release=_int(rel) if case["release"] else None,
                  table=_int(table), held=_int([_pages(a, ps) for a in lens]), free=_int(room),
                  count=_int([len(free)]), ps=ps, num_pages=num_pages, n_rows=sum(grow))
        if own:
            st.update(outs=dict(lens_out=_int(lens), held_out=_int(lens), free_count_out=_int([0]), status=_int(lens),
                                row_start=_int(lens + [0]), slot_map=_int([0] * sum(grow))))
        return st
    if op == "append":
        N, Hkv, d, ps = case["N"], case["Hkv"], case["d"], case["ps"]
        num_pages = _pages(N, ps) + 4
        if case["fused"]:
            qkv = _randn((N, (case["Hq"] + 2 * Hkv) * d), case["dtype"], g)
            at = case["Hq"] * d
            k = qkv[:, at:at + Hkv * d].view(N, Hkv, d)
            v = qkv[:, at + Hkv * d:].view(N, Hkv, d)
        else:
            k, v = _randn((N, Hkv, d), case["dtype"], g), _randn((N, Hkv, d), case["dtype"], g)
        # runs of rows in shuffled pages, as a block table gives them
        order = torch.randperm(num_pages, device="cuda", generator=g)[:_pages(N, ps)]
        slots = (order[:, None] * ps + torch.arange(ps, device="cuda")).reshape(-1)[:N].to(torch.int32)
        st.update(k=k, v=v, slots=slots, kcache=_randn((num_pages, Hkv, ps, d), case["dtype"], g),
                  vcache=_randn((num_pages, Hkv, ps, d), case["dtype"], g))
        return st
    lens, nodes = _lens(case), _nodes(case)
    num_pages, table, _ = _pool(case, seed, [a + t for a, t in zip(lens, nodes)])
    shape = (num_pages, case["Hkv"], case["ps"], case["d"])
    kcache = _randn(shape, case["dtype"], g)
    # one key row in a hundred is an outlier, eight times the others
    kcache *= 1 + 7 * (torch.rand((num_pages, case["Hkv"], case["ps"], 1), device="cuda", generator=g) < 0.01).to(
        kcache.dtype)
    st.update(kcache=kcache, vcache=_randn(shape, case["dtype"], g), table=_int(table), lens=_int(lens),
              row_start=_int(_starts(nodes)), host_lens=lens, host_nodes=nodes)
    if op == "commit":
        parents, last = [], []
        r = random.Random(57 * seed + case["mix"])
        for T, path in zip(nodes, _paths(case)):
            par = [-1] + [r.randint(0, t - 1) for t in range(1, T)]
            for a, b in zip(path, path[1:]):
                par[b] = a
            parents += par
            last.append(path[-1] if path else -1)
        st.update(parents=_int(parents), last=_int(last), host_parents=parents, host_last=last)
        if own:
            st.update(lens_out=torch.empty_like(st["lens"]), accepted=torch.empty_like(st["lens"]))
        return st
    N = sum(nodes)
    st["q"] = _randn((N, case["Hq"], case["d"]), case["dtype"], g)
    if op == "tree":
        st["host_parents"] = _parents(case, seed, nodes)
        st["parents"] = None if case["chain"] else _int(st["host_parents"])
    else:
        st["host_parents"] = [-1] * N
    if own:
        import rope_context_extension_jet_b200 as jl
        size = jl.decode_tree_workspace_size(case["B"], case["Hq"], case["Hkv"], case["d"], case.get("T", 1))
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty_like(st["q"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _RUN_OWN[op](st)
    return _RUN_PLAIN[op](st)


def _own_tables(st):
    import rope_context_extension_jet_b200 as jl
    r = jl.block_tables(st["lens"], st["grow"], st["table"], st["held"], st["free"], st["count"], page_size=st["ps"],
                        num_pages=st["num_pages"], n_rows=st["n_rows"], release=st["release"], **st["outs"])
    return dict(table=st["table"], free=st["free"], lens=r.lens, held=r.held, count=r.free_count, slots=r.slot_map,
                row_start=r.row_start, status=r.status)


def _own_append(st):
    import rope_context_extension_jet_b200 as jl
    jl.cache_append(st["k"], st["v"], st["slots"], st["kcache"], st["vcache"])
    return dict(kcache=st["kcache"], vcache=st["vcache"])


def _own_paged(st):
    import rope_context_extension_jet_b200 as jl
    c = st["case"]
    return jl.decode_paged(st["q"], st["kcache"], st["vcache"], st["table"], st["lens"], st["out"], w0=c["w0"],
                           w_pretrained=c["w_pre"], rope_theta=c["theta"], workspace=st["workspace"])


def _own_tree(st):
    import rope_context_extension_jet_b200 as jl
    c = st["case"]
    return jl.decode_tree(st["q"], st["kcache"], st["vcache"], st["table"], st["lens"], st["row_start"],
                          st["parents"], st["out"], max_nodes=c["T"], w0=c["w0"], w_pretrained=c["w_pre"],
                          rope_theta=c["theta"], workspace=st["workspace"])


def _own_commit(st):
    import rope_context_extension_jet_b200 as jl
    jl.tree_commit(st["kcache"], st["vcache"], st["table"], st["lens"], st["row_start"], st["parents"], st["last"],
                   max_nodes=st["case"]["T"], lens_out=st["lens_out"], n_accepted=st["accepted"])
    return dict(kcache=st["kcache"], vcache=st["vcache"], lens=st["lens_out"], accepted=st["accepted"])


_RUN_OWN = dict(tables=_own_tables, append=_own_append, paged=_own_paged, tree=_own_tree, commit=_own_commit)


def _plain_tables(st):
    ps, n_rows, table, free = st["ps"], st["n_rows"], st["table"], st["free"]
    B, wide = table.shape
    lens, held, count, grow = st["lens"].long(), st["held"].long(), st["count"].long(), st["grow"].long()
    cols = torch.arange(wide, device="cuda")
    if st["release"] is not None:
        gone = st["release"] != 0
        back = torch.where(gone, held, 0)
        # the last request's pages go back first, each request's last page first
        order = back.flip(0)
        first = (torch.cumsum(order, 0) - order).flip(0)
        at = count + first[:, None] + (back[:, None] - 1 - cols)
        ok = cols < back[:, None]
        buf = torch.cat([free, free.new_zeros(1)])
        buf.scatter_(0, torch.where(ok, at, free.numel()).reshape(-1), table.reshape(-1))
        free.copy_(buf[:-1])
        count = count + back.sum()
        lens, held = torch.where(gone, 0, lens), torch.where(gone, 0, held)
    total = (lens + grow + ps - 1) // ps
    need = torch.clamp(total - held, min=0)
    long = total > wide
    need = torch.where(long, 0, need)
    incl = torch.cumsum(need, 0)
    short = (incl > count) & (need > 0)
    status = torch.where(long, 2, torch.where(short, 1, 0))
    take = torch.where(short, 0, need)
    # pages come from the top of the list, in request order
    src = count - 1 - ((incl - need)[:, None] + (cols - held[:, None]))
    fresh = (cols >= held[:, None]) & (cols < (held + take)[:, None])
    page = free[torch.clamp(src, 0, free.numel() - 1)]
    table.copy_(torch.where(fresh, page, table))
    held = held + take
    count = count - take.sum()
    ends = torch.cumsum(grow, 0)
    row_start = torch.cat([ends.new_zeros(1), ends])
    n = torch.arange(n_rows, device="cuda")
    req = torch.searchsorted(ends, n, right=True).clamp(max=B - 1)
    pos = lens[req] + n - row_start[req]
    slot = table[req, torch.clamp(pos // ps, max=wide - 1)].long() * ps + pos % ps
    slot = torch.where((status[req] != 0) | (n >= ends[-1]), -1, slot)
    i32 = torch.int32
    return dict(table=table, free=free, lens=lens.to(i32), held=held.to(i32), count=count.to(i32), slots=slot.to(i32),
                row_start=row_start.to(i32), status=status.to(i32))


def _plain_append(st):
    slots, ps = st["slots"].long(), st["kcache"].shape[2]
    st["kcache"][slots // ps, :, slots % ps] = st["k"]
    st["vcache"][slots // ps, :, slots % ps] = st["v"]
    return dict(kcache=st["kcache"], vcache=st["vcache"])


def _rotate(x, pos, theta):
    """Rows of x turned to positions pos (half-split pairs); angles in 64 bits."""
    h = x.shape[-1] // 2
    freq = theta ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    ang = pos.to(torch.float64)[:, None] * freq
    c, s = torch.cos(ang).to(x.dtype), torch.sin(ang).to(x.dtype)
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _depths(parents):
    """(depth, ancestors-or-self) of each drafted token of one request."""
    depth, anc = [], []
    for t, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        anc.append({t} | (anc[p] if p >= 0 else set()))
    return depth, anc


def _plain_attend(st):
    c = st["case"]
    Hq, Hkv, d, ps, w0, theta = c["Hq"], c["Hkv"], c["d"], c["ps"], c["w0"], c["theta"]
    group = Hq // Hkv
    out = torch.empty_like(st["q"])
    at = 0
    for b, (L, T) in enumerate(zip(st["host_lens"], st["host_nodes"])):
        n = L + T
        pages = st["table"][b, :_pages(n, ps)].long()
        k = st["kcache"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        v = st["vcache"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        depth, anc = _depths(st["host_parents"][at:at + T])
        qpos = L + torch.tensor(depth, device="cuda")
        kpos = torch.cat([torch.arange(L, device="cuda"), qpos])
        seen = torch.ones((T, n), dtype=torch.bool, device="cuda")
        seen[:, L:] = torch.tensor([[u in a for u in range(T)] for a in anc], device="cuda")
        q = st["q"][at:at + T].float().transpose(0, 1)
        local = qpos[:, None] - kpos[None, :] < w0
        logit = torch.empty((Hkv, group, T, n), dtype=torch.float32, device="cuda")
        if w0 > 0:
            qe = _rotate(q, qpos, theta).reshape(Hkv, group * T, d)
            logit.copy_((qe @ _rotate(k, kpos, theta).transpose(1, 2)).view(Hkv, group, T, n))
        sizes = [max(1, -(-(L + x + 1) // c["w_pre"])) for x in depth]
        for G in sorted(set(sizes)):
            mine = torch.tensor([i for i, s in enumerate(sizes) if s == G], device="cuda")
            qr = _rotate(q[:, mine], qpos[mine] // G, theta).reshape(Hkv, -1, d)
            far = (qr @ _rotate(k, kpos // G, theta).transpose(1, 2)).view(Hkv, group, len(mine), n)
            logit[:, :, mine] = torch.where(local[mine], logit[:, :, mine], far)
        logit *= 1 / math.sqrt(d)
        logit = torch.where(seen, logit, -math.inf)
        p = torch.exp(logit - logit.amax(-1, keepdim=True))
        o = (p.view(Hkv, group * T, n) @ v).view(Hkv, group, T, d) / p.sum(-1, keepdim=True)
        out[at:at + T] = o.view(Hq, T, d).transpose(0, 1).to(out.dtype)
        at += T
    return out


def _plain_commit(st):
    ps, lens, table = st["case"]["ps"], st["host_lens"], st["table"]
    src_b, src_r, dst_r, counts, at = [], [], [], [], 0
    for b, (L, T, last) in enumerate(zip(lens, st["host_nodes"], st["host_last"])):
        path = []
        while last >= 0:
            path.append(last)
            last = st["host_parents"][at + last]
        path.reverse()
        src_b += [b] * len(path)
        src_r += [L + x for x in path]
        dst_r += range(L, L + len(path))
        counts.append(len(path))
        at += T
    b, s, t = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (src_b, src_r, dst_r))
    sp, tp = table[b, s // ps].long(), table[b, t // ps].long()
    for cache in (st["kcache"], st["vcache"]):
        cache[tp, :, t % ps] = cache[sp, :, s % ps]
    accepted = _int(counts)
    return dict(kcache=st["kcache"], vcache=st["vcache"], lens=st["lens"] + accepted, accepted=accepted)


_RUN_PLAIN = dict(tables=_plain_tables, append=_plain_append, paged=_plain_attend, tree=_plain_attend,
                  commit=_plain_commit)


# ------------------------------------------------------------------ 64-bit answers
def exact(case, seed):
    if case["op"] not in ("paged", "tree"):
        return None
    st = prepare(case, seed)
    Hq, Hkv, d, ps = case["Hq"], case["Hkv"], case["d"], case["ps"]
    group, w0, w_pre = Hq // Hkv, case["w0"], case["w_pre"]
    nu = torch.pow(torch.tensor(float(case["theta"]), dtype=torch.float64, device="cuda"),
                   -2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    answer = torch.zeros((sum(st["host_nodes"]), Hq, d), dtype=torch.float64, device="cuda")

    def turned(x, where):  # pairs as complex numbers, times e^(i where nu)
        z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double())
        a = where.double()[:, None] * nu
        return z * torch.complex(torch.cos(a), torch.sin(a))

    def dots(x, y):  # real part of <x, conj y>, over [.., d/2] complex
        return x.real @ y.real.transpose(-1, -2) + x.imag @ y.imag.transpose(-1, -2)

    first = 0
    for b in range(case["B"]):
        L, T = st["host_lens"][b], st["host_nodes"][b]
        par = st["host_parents"][first:first + T]
        up = torch.zeros((T, T), dtype=torch.bool)
        hops = [0] * T
        for t in range(T):
            x = t
            while x >= 0:
                up[t, x] = True
                x = par[x]
            hops[t] = int(up[t].sum()) - 1
        where_q = torch.tensor([L + h for h in hops], device="cuda")
        rows = torch.arange(L + T, device="cuda")
        where_k = torch.where(rows < L, rows, where_q[(rows - L).clamp(min=0)])
        page, off = st["table"][b].long()[rows // ps], rows % ps
        open_ = torch.cat([torch.ones((T, L), dtype=torch.bool), up], 1).cuda()
        near = (where_q[:, None] - where_k[None]) < w0
        size = torch.clamp((where_q + 1 + w_pre - 1) // w_pre, min=1)
        for h in range(Hkv):
            k, v = st["kcache"][page, h, off], st["vcache"][page, h, off].double()
            heads = st["q"][first:first + T, h * group:(h + 1) * group].transpose(0, 1)
            s = torch.empty((group, T, L + T), dtype=torch.float64, device="cuda")
            if w0 > 0:
                s.copy_(dots(turned(heads, where_q), turned(k, where_k)))
            for G in size.unique().tolist():
                pick = (size == G).nonzero()[:, 0]
                far = dots(turned(heads[:, pick], where_q[pick] // G), turned(k, where_k // G))
                s[:, pick] = torch.where(near[pick], s[:, pick], far)
            s = s.div_(d ** 0.5).masked_fill_(~open_, -math.inf)
            answer[first:first + T, h * group:(h + 1) * group] = (torch.softmax(s, -1) @ v).transpose(0, 1)
        first += T
    return answer
