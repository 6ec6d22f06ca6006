"""CPU checks of the paged-cache calls: refusals by the C ABI before any launch,
tensor checks of the binding, workspace sizes, and the plain implementations
the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_reference as R
import rope_context_extension_jet_b200 as jl
from rope_context_extension_jet_b200 import _build

Z = ctypes.c_void_p(0)
P = ctypes.c_void_p(1 << 20)      # aligned, never followed
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return jl.load_library()


def refused(lib, status, code, text):
    assert status == code and text in lib.jetlong_last_error().decode(), lib.jetlong_last_error()


TABLES = dict(lens=P, grow=P, release=Z, held=P, free_count=P, table=P, free_list=P, lens_out=P, held_out=P, count_out=P,
              slots=P, row_start=P, status=P, B=4, max_pages=8, page_size=64, num_pages=32, free_cap=32, n_rows=4, stream=Z)


@pytest.mark.parametrize("change,code,text", [
    (dict(lens=Z), 1, "null"), (dict(grow=Z), 1, "null"), (dict(table=Z), 1, "null"), (dict(slots=Z), 1, "null"),
    (dict(status=Z), 1, "null"), (dict(release=ODD), 1, "4-byte"), (dict(B=0), 1, "B >= 1"), (dict(n_rows=-1), 1, "n_rows"),
    (dict(free_cap=0), 1, "free_cap"), (dict(B=8193), 2, "8192"), (dict(page_size=48), 2, "page_size"),
    (dict(page_size=8), 2, "page_size"), (dict(page_size=512), 2, "page_size"), (dict(num_pages=0), 1, "num_pages"),
    (dict(max_pages=0), 1, "max_pages"), (dict(num_pages=1 << 26), 2, "31 bits"),
    (dict(max_pages=1 << 20, B=4096), 2, "31 bits"),
])
def test_tables_refusals(lib, change, code, text):
    refused(lib, lib.jetlong_block_tables(*{**TABLES, **change}.values()), code, text)


APPEND = dict(k=P, v=P, slots=P, kc=P, vc=P, N=4, Hkv=2, d=128, kt=256, kh=128, vt=256, vh=128, num_pages=8, page_size=64,
              dtype=0, stream=Z)


@pytest.mark.parametrize("change,code,text", [
    (dict(k=Z), 1, "null"), (dict(vc=Z), 1, "null"), (dict(slots=Z), 1, "null"), (dict(k=ODD), 1, "16-byte"),
    (dict(kt=257), 1, "16-byte"), (dict(vh=4), 1, "16-byte"), (dict(N=-1), 1, "N must"), (dict(Hkv=0), 1, "Hkv"),
    (dict(d=96), 2, "head dim"), (dict(dtype=7), 1, "dtype"), (dict(page_size=20), 2, "page_size"),
])
def test_append_refusals(lib, change, code, text):
    refused(lib, lib.jetlong_cache_append(*{**APPEND, **change}.values()), code, text)


TREE = dict(q=P, kc=P, vc=P, out=P, table=P, lens=P, row_start=P, parents=Z, B=2, N=6, Hq=8, Hkv=2, d=128, num_pages=8,
            page_size=64, max_pages=4, max_nodes=4, w0=16, w_pre=64, theta=1e4, scale=0.1, dtype=0, ws=P, ws_bytes=1 << 40,
            stream=Z)


@pytest.mark.parametrize("change,code,text", [
    (dict(q=Z), 1, "null"), (dict(table=Z), 1, "null"), (dict(lens=Z), 1, "null"), (dict(ws=Z), 1, "null"),
    (dict(out=ODD), 1, "16-byte"), (dict(parents=ctypes.c_void_p((1 << 20) + 1)), 1, "4-byte"), (dict(N=-1), 1, "N must"),
    (dict(B=0), 1, "positive"), (dict(Hq=9), 1, "multiple"), (dict(d=80), 2, "head dim"), (dict(w0=-1), 1, "w0"),
    (dict(w_pre=0), 1, "w_pretrained"), (dict(theta=1.0), 1, "rope_theta"), (dict(scale=0.0), 1, "scale"),
    (dict(dtype=5), 1, "dtype"), (dict(max_nodes=0), 1, "max_nodes"), (dict(max_nodes=65), 1, "max_nodes"),
    (dict(row_start=Z), 1, "without row_start"), (dict(page_size=100), 2, "page_size"), (dict(ws_bytes=64), 1, "workspace too small"),
    (dict(row_start=Z, N=2, max_nodes=1, parents=P), 1, "without row_start"),
])
def test_tree_refusals(lib, change, code, text):
    refused(lib, lib.jetlong_decode_tree(*{**TREE, **change}.values()), code, text)


COMMIT = dict(kc=P, vc=P, table=P, lens=P, row_start=P, parents=Z, last=P, lens_out=P, acc=Z, B=2, N=6, Hkv=2, d=64,
              num_pages=8, page_size=32, max_pages=4, max_nodes=8, dtype=1, stream=Z)


@pytest.mark.parametrize("change,code,text", [
    (dict(kc=Z), 1, "null"), (dict(last=Z), 1, "null"), (dict(row_start=Z), 1, "null"), (dict(vc=ODD), 1, "16-byte"),
    (dict(lens=ctypes.c_void_p((1 << 20) + 1)), 1, "4-byte"), (dict(B=0), 1, "B >= 1"), (dict(max_nodes=65), 1, "max_nodes"),
    (dict(d=32), 2, "head dim"), (dict(dtype=2), 1, "dtype"), (dict(page_size=1), 2, "page_size"),
])
def test_commit_refusals(lib, change, code, text):
    refused(lib, lib.jetlong_tree_commit(*{**COMMIT, **change}.values()), code, text)


def test_nothing_was_launched(lib):
    assert lib.jetlong_launch_count() == 0 or torch.cuda.is_available()


def test_empty_calls_do_nothing(lib):
    assert lib.jetlong_cache_append(*{**APPEND, "N": 0, "k": Z, "v": Z, "slots": Z}.values()) == 0
    assert lib.jetlong_decode_tree(*{**TREE, "N": 0, "q": Z, "out": Z}.values()) == 0


def test_workspace_sizes(lib):
    size = jl.decode_tree_workspace_size
    assert size(4, 32, 8, 128, 1) > 0 and size(4, 32, 8, 128, 64) >= size(4, 32, 8, 128, 1)
    assert size(4, 32, 8, 128, 64) > size(4, 32, 8, 64, 64)
    for bad in ((0, 32, 8, 128, 1), (4, 30, 8, 128, 1), (4, 32, 8, 100, 1), (4, 32, 8, 128, 0), (4, 32, 8, 128, 65)):
        assert size(*bad) == 0


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


KW = dict(w0=4, w_pretrained=8, rope_theta=1e4)
C = (4, 1, 16, 64)  # cache shape


def tables(**kw):
    a = dict(lens=i(2), grow=i(2), block_table=i(2, 3), held=i(2), free_list=i(4), free_count=i(1), page_size=16,
             num_pages=4, n_rows=2)
    a.update(kw)
    return jl.block_tables(**a)


@pytest.mark.parametrize("call", [
    lambda: tables(),
    lambda: jl.cache_append(t(2, 1, 64), t(2, 1, 64), i(2), t(*C), t(*C)),
    lambda: jl.decode_paged(t(2, 2, 64), t(*C), t(*C), i(2, 3), i(2), **KW),
    lambda: jl.decode_tree(t(5, 2, 64), t(*C), t(*C), i(2, 3), i(2), i(3), max_nodes=4, **KW),
    lambda: jl.tree_commit(t(*C), t(*C), i(2, 3), i(2), i(3), None, i(2), max_nodes=4),
])
def test_host_tensors_raise(call):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        call()


@pytest.mark.parametrize("call,text", [
    (lambda: tables(lens=i(3)), "lens must be an int32"), (lambda: tables(grow=i(2).long()), "must be a CUDA|grow must be an int32"),
    (lambda: tables(block_table=i(2)), "block_table must be"),
    (lambda: jl.cache_append(t(2, 2, 64), t(2, 1, 64), i(2), t(*C), t(*C)), "k must be"),
    (lambda: jl.cache_append(t(2, 1, 64, dtype=torch.float32), t(2, 1, 64), i(2), t(*C), t(*C)), "k must be"),
    (lambda: jl.cache_append(t(2, 1, 64), t(2, 1, 64), i(2), t(*C), t(4, 1, 16, 128)), "kcache and vcache"),
    (lambda: jl.decode_paged(t(3, 2, 64), t(*C), t(*C), i(2, 3), i(2), **KW), "one row per request"),
    (lambda: jl.decode_paged(t(2, 2, 128), t(*C), t(*C), i(2, 3), i(2), **KW), "q must be"),
    (lambda: jl.decode_tree(t(2, 2, 64), t(*C), t(*C), i(6), i(2), i(3), max_nodes=2, **KW), "block_table must be"),
    (lambda: jl.decode_tree(t(2, 2, 64), t(*C), t(*C), i(2, 3), i(2), i(3), None, t(3, 2, 64), max_nodes=2, **KW), "out must match q"),
    (lambda: jl.tree_commit(t(*C), t(*C), i(2), i(2), i(3), None, i(2), max_nodes=4), "block_table must be"),
])
def test_mismatched_tensors_raise(call, text):
    with pytest.raises(ValueError, match=text):
        call()


def test_mixed_element_types_raise():
    with pytest.raises(TypeError, match="must share a dtype"):
        jl.decode_paged(t(2, 2, 64, dtype=torch.float32), t(*C), t(*C), i(2, 3), i(2), **KW)


@pytest.mark.parametrize("w0,w_pre", [(0, 7), (5, 7), (9, 100), (1000, 7)])
def test_plain_tree_attention_of_a_chain_is_the_oracle_decode(w0, w_pre):
    """The plain implementation the GPU tests use, pinned to the oracle: node t of
    a chain is a decode at length len + t + 1."""
    g = np.random.default_rng(4)
    L, T, Hq, Hkv, d, ps = 21, 4, 4, 2, 64, 16
    kc, vc = (g.standard_normal((1, Hkv, L + T, d)).astype(np.float32) for _ in range(2))
    q = g.standard_normal((T, Hq, d)).astype(np.float32)
    pages, k2, v2 = [2, 0], np.zeros((3, Hkv, ps, d)), np.zeros((3, Hkv, ps, d))
    for r in range(L + T):
        k2[pages[r // ps], :, r % ps], v2[pages[r // ps], :, r % ps] = kc[0, :, r], vc[0, :, r]
    out, _ = R.attend(q.astype(np.float64), k2, v2, pages, L, [-1, 0, 1, 2], w0=w0, w_pre=w_pre, theta=1e4, scale=0.125,
                      dtype="fp32")
    for x in range(T):
        ref = oracle.decode(q[x][None], kc, vc, L + x + 1, w0=w0, w_pretrained=w_pre, rope_theta=1e4, scale=0.125)
        assert np.abs(out[x] - ref[0]).max() < 1e-12


def test_plain_tree_attention_of_a_branch_is_its_path():
    """A node of a tree attends as if its path alone had been drafted."""
    g = np.random.default_rng(5)
    L, Hq, Hkv, d, ps = 9, 2, 1, 64, 16
    parents, leaf, path = [-1, 0, 0, 2, 1], 3, [0, 2, 3]
    k, v = (g.standard_normal((1, Hkv, ps, d)) for _ in range(2))
    q = g.standard_normal((5, Hq, d))
    kw = dict(w0=3, w_pre=4, theta=1e4, scale=0.125, dtype="fp32")
    out, _ = R.attend(q, k, v, [0], L, parents, **kw)
    k2, v2 = k.copy(), v.copy()
    for j, x in enumerate(path):
        k2[0, :, L + j], v2[0, :, L + j] = k[0, :, L + x], v[0, :, L + x]
    ref, _ = R.attend(q[path], k2, v2, [0], L, [-1, 0, 1], **kw)
    assert np.abs(out[leaf] - ref[-1]).max() < 1e-13


def test_plain_tables():
    a = R.Tables([[0] * 3, [0] * 3], [0, 0], [0, 0], [5, 6, 7], 16)
    assert a.step([17, 16], [0, 0], 34) == ([112 + x for x in range(16)] + [96] + [80 + x for x in range(16)] + [-1],
                                            [0, 17, 33], [0, 0])
    a.lens = [17, 16]
    assert a.step([0, 1], [0, 0], 1) == ([-1], [0, 0, 1], [0, 1]) and a.free == []
    assert a.step([1, 0], [1, 0], 1) == ([112], [0, 1, 1], [0, 0]) and a.free == [6]
    assert a.step([60, 0], [0, 0], 60)[2] == [2, 0]
