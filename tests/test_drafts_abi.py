"""Host-side checks of the calls for drafted tokens and eviction (nothing is launched, no GPU is needed)."""

import ctypes as C
import os

import numpy as np
import pytest

from indexer_driven_sparse_gb300 import binding as qb
from indexer_driven_sparse_gb300 import build as qbuild
from indexer_driven_sparse_gb300.pipeline import PagedCache
from oracle import drafts_oracle as T
from tests.test_paged_abi import BAD, FAKE, SMALL, UNSUPPORTED, rope_cfg


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qb.load()


def paged_cfg(**kw):
    base = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, window=0, softmax_scale=0.0)
    base.update(kw)
    return qb.qsa_paged_config(*[base[n] for n, _ in qb.qsa_paged_config._fields_])


GEOMETRY = [(dict(head_dim=96), UNSUPPORTED), (dict(n_q_heads=0), BAD), (dict(n_q_heads=9), UNSUPPORTED),
            (dict(n_q_heads=34), UNSUPPORTED), (dict(page_size=0), BAD), (dict(window=-1), BAD),
            (dict(softmax_scale=float("inf")), BAD)]


def test_workspace_sizes(lib):
    cfg = paged_cfg()
    assert lib.qsa_tree_workspace_size(C.byref(cfg), 1) >= 256
    assert lib.qsa_tree_workspace_size(C.byref(cfg), 128) >= lib.qsa_tree_workspace_size(C.byref(cfg), 1)
    assert lib.qsa_tree_workspace_size(C.byref(cfg), 0) == lib.qsa_tree_workspace_size(C.byref(cfg), 129) == 0
    assert lib.qsa_tree_workspace_size(None, 4) == 0
    small, large = (lib.qsa_paged_weights_workspace_size(C.byref(cfg), 4, n) for n in (0, 10 ** 6))
    assert small > lib.qsa_paged_workspace_size(C.byref(cfg)) and large >= small + 10 ** 6 * 8 * 4
    for b, n in ((-1, 5), (65536, 5), (4, -1)):
        assert lib.qsa_paged_weights_workspace_size(C.byref(cfg), b, n) == 0
    for kw, _ in GEOMETRY:
        assert lib.qsa_tree_workspace_size(C.byref(paged_cfg(**kw)), 4) == 0
        assert lib.qsa_paged_weights_workspace_size(C.byref(paged_cfg(**kw)), 4, 4) == 0
    assert lib.qsa_keep_workspace_size(0, 0) >= 256
    assert lib.qsa_keep_workspace_size(7, 1000) >= 256 + 7 * (1000 * 4 + 1000 * 8)     # keys, and the two lists
    for rows, tokens in ((-1, 0), (65537, 0), (4, -1), (4, 2 ** 31)):
        assert lib.qsa_keep_workspace_size(rows, tokens) == 0


def test_tree_decode_refusals(lib):
    def call(fp8=False, cfg=paged_cfg(), q=FAKE, q_ld=1024, off=FAKE, parent=FAKE, n=5, most=4, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE,
             pages=10, table=FAKE, ld=4, lens=FAKE, b=3, out=FAKE, lse=FAKE, ws=FAKE, bytes=1 << 32):
        head = (C.byref(cfg) if cfg else None, q, q_ld, off, parent, n, most)
        tail = (pages, table, ld, lens, b, out, lse, ws, bytes, None)
        if fp8:
            return lib.qsa_tree_decode_fp8kv(*head, k, ks, v, vs, *tail)
        return lib.qsa_tree_decode(*head, k, v, *tail)

    assert call(n=0) == call(b=0) == qb.QSA_OK
    for kw, code in GEOMETRY:
        assert call(cfg=paged_cfg(**kw)) == code, kw
    for kw in (dict(cfg=None), dict(n=-1), dict(b=-1), dict(b=65536), dict(q=0), dict(q=FAKE + 8), dict(q_ld=1016), dict(q_ld=1028),
               dict(off=0), dict(off=FAKE + 2), dict(parent=0), dict(parent=FAKE + 1), dict(k=0), dict(v=0), dict(k=FAKE + 8),
               dict(v=FAKE + 4), dict(pages=-1), dict(ld=-1), dict(table=0), dict(table=FAKE + 2), dict(lens=0), dict(out=0),
               dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(ws=0), dict(ws=FAKE + 128)):
        assert call(**kw) == BAD, kw
    for kw in (dict(ks=0), dict(vs=0), dict(ks=FAKE + 4), dict(vs=FAKE + 4)):
        assert call(fp8=True, **kw) == BAD, kw
    assert call(most=0) == call(most=129) == UNSUPPORTED
    assert call(fp8=True, cfg=paged_cfg(head_dim=64)) == UNSUPPORTED
    assert call(pages=2 ** 28) == UNSUPPORTED
    assert call(bytes=100) == SMALL
    # no memory of this process is the GPU's
    host = np.zeros(4096, np.uint8)
    at = host.ctypes.data + (-host.ctypes.data) % 256
    assert call(k=at) == call(v=at) == BAD and b"device memory" in lib.qsa_last_error()


def test_weights_refusals(lib):
    def call(fp8=False, cfg=paged_cfg(), q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, table=FAKE, ld=4, lens=FAKE, b=3,
             out=FAKE, lse=FAKE, weights=FAKE, w_ld=64, ws=FAKE, bytes=1 << 32):
        head, tail = (C.byref(cfg) if cfg else None, q, 1024), (pages, table, ld, lens, b, out, lse, weights, w_ld, ws, bytes, None)
        if fp8:
            return lib.qsa_paged_decode_weights_fp8kv(*head, k, ks, v, vs, *tail)
        return lib.qsa_paged_decode_weights(*head, k, v, *tail)

    assert call(b=0) == qb.QSA_OK
    for kw in (dict(weights=0), dict(weights=FAKE + 2), dict(w_ld=-1), dict(cfg=None), dict(q=0), dict(k=0), dict(v=0), dict(table=0),
               dict(lens=0), dict(out=0), dict(ws=0), dict(b=-1)):
        assert call(**kw) == BAD, kw
    for kw, code in GEOMETRY:
        assert call(cfg=paged_cfg(**kw)) == code, kw
    assert call(fp8=True, ks=0) == BAD
    assert call(bytes=lib.qsa_paged_workspace_size(C.byref(paged_cfg()))) == SMALL


def test_append_at_refusals(lib):
    def call(fp8=False, place=FAKE, positions=FAKE, p_ld=8, pos=FAKE, n=3):
        cfg, rope = paged_cfg(), rope_cfg()
        head = (C.byref(cfg), C.byref(rope), FAKE, 1.0, None, 0, FAKE, 256, FAKE, 256, None, pos, place, n, None, 0)
        tail = (10, FAKE, 4, 3, positions, p_ld, FAKE, 1 << 20, None)
        if fp8:
            return lib.qsa_rope_append_at_fp8kv(*head, FAKE, FAKE, FAKE, FAKE, *tail)
        return lib.qsa_rope_append_at(*head, FAKE, FAKE, *tail)

    for fp8 in (False, True):
        assert call(fp8, n=0) == qb.QSA_OK
        for kw in (dict(place=0), dict(place=FAKE + 2), dict(positions=FAKE + 1), dict(p_ld=-1), dict(pos=0), dict(n=-1)):
            assert call(fp8, **kw) == BAD, kw


def test_keep_refusals(lib):
    def planes(**kw):
        base = dict(base=FAKE, plane_stride=4096, page_bytes=64, n_planes=2)
        base.update(kw)
        return (qb.qsa_page_planes * 1)(qb.qsa_page_planes(**base))

    other = FAKE + 256

    def accept(ps=4, off=FAKE, parent=FAKE, n=5, accepted=FAKE, table=FAKE, lens=FAKE, rows=3, ld=4, ref=FAKE, pages=9,
               t_out=other, l_out=other, r_out=other, positions=FAKE, p_ld=16, groups=None, count=1, ws=FAKE, bytes=1 << 30):
        return lib.qsa_accept_drafts(ps, off, parent, n, accepted, table, lens, rows, ld, ref, pages, t_out, l_out, r_out, positions,
                                     p_ld, planes() if groups is None else groups, count, ws, bytes, None)

    def evict(ps=4, budget=FAKE, first=1, recent=2, weights=FAKE, positions=FAKE, t_ld=16, table=FAKE, lens=FAKE, rows=3, ld=4,
              ref=FAKE, pages=9, w_out=other, p_out=other, t_out=other, l_out=other, r_out=other, groups=None, count=1, ws=FAKE,
              bytes=1 << 30):
        return lib.qsa_evict_tokens(ps, budget, first, recent, weights, positions, t_ld, table, lens, rows, ld, ref, pages, w_out,
                                    p_out, t_out, l_out, r_out, planes() if groups is None else groups, count, ws, bytes, None)

    shared = [dict(ps=0), dict(table=0), dict(lens=0), dict(rows=-1), dict(rows=65537), dict(ld=-1), dict(ref=0), dict(pages=-1),
              dict(t_out=0), dict(l_out=0), dict(r_out=0), dict(t_out=FAKE), dict(l_out=FAKE), dict(r_out=FAKE), dict(table=FAKE + 2),
              dict(l_out=other + 1), dict(ws=0), dict(ws=FAKE + 64), dict(groups=planes(base=0)), dict(groups=planes(page_bytes=6)),
              dict(groups=planes(page_bytes=20)), dict(groups=planes(page_bytes=8)), dict(groups=planes(base=FAKE + 4)),
              dict(groups=planes(n_planes=-1)), dict(count=9), dict(count=-1), dict(positions=FAKE + 2)]
    for kw in shared + [dict(off=0), dict(off=FAKE + 2), dict(parent=0), dict(accepted=0), dict(accepted=FAKE + 1), dict(n=-1),
                        dict(p_ld=-1)]:
        assert accept(**kw) == BAD, kw
    for kw in shared + [dict(budget=0), dict(first=-1), dict(recent=-1), dict(weights=0), dict(positions=0), dict(w_out=0), dict(p_out=0),
                        dict(w_out=FAKE), dict(p_out=FAKE), dict(t_ld=-1), dict(t_ld=2 ** 31), dict(budget=FAKE + 2), dict(w_out=other + 2)]:
        assert evict(**kw) == BAD, kw
    for call in (accept, evict):
        assert call(bytes=256) == SMALL
        assert call(pages=(1 << 30) + 1) == UNSUPPORTED and call(ps=1 << 20, pages=1 << 12, count=0) == UNSUPPORTED
        assert call(rows=0, pages=0) == qb.QSA_OK
    assert lib.qsa_evict_tokens(4, FAKE, 1, 2, FAKE, FAKE, 1000, FAKE, FAKE, 3, 4, FAKE, 9, other, other, other, other, other, planes(), 1,
                                FAKE, lib.qsa_keep_workspace_size(3, 999), None) == SMALL


def test_accept_weights_refusals(lib):
    def call(off=FAKE, parent=FAKE, n=5, accepted=FAKE, weights=FAKE, positions=FAKE, t_ld=16, table=FAKE, rows=3, t_out=FAKE + 256,
             ws=FAKE, bytes=1 << 30):
        return lib.qsa_accept_drafts_weights(4, off, parent, n, accepted, weights, positions, t_ld, table, FAKE, rows, 4, FAKE,
                                             9 if rows else 0, t_out, FAKE + 256, FAKE + 256, None, 0, ws, bytes, None)

    assert call(rows=0) == call(rows=0, weights=0, positions=0) == qb.QSA_OK
    for kw in (dict(weights=0), dict(positions=0), dict(weights=FAKE + 2), dict(positions=FAKE + 1), dict(t_ld=-1), dict(off=0),
               dict(accepted=0), dict(parent=0), dict(n=-1), dict(rows=-1), dict(table=0), dict(t_out=FAKE), dict(ws=0)):
        assert call(**kw) == BAD, kw
    assert call(bytes=256) == SMALL


def test_binding_refuses_wrong_tensors(lib):
    import torch
    bf16, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    cfg = paged_cfg()
    q, kv = torch.zeros(5, 8, 128, **bf16), [torch.zeros(6, 16, 2, 128, **bf16) for _ in range(2)]
    table, lens, ws = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(512, dtype=torch.uint8)
    off, parent, lse, weights = torch.zeros(3, **i32), torch.zeros(5, **i32), torch.zeros(5, 8), torch.zeros(2, 48)

    def refused(error, text, fn, *args):
        with pytest.raises(error, match=text):
            fn(*args)

    tree = qb.qsa_tree_decode
    refused(ValueError, "q is on cpu", tree, cfg, q, off, parent, 4, *kv, table, lens, q, lse, ws)
    refused(TypeError, "q must be torch.BFloat16", tree, cfg, q.float(), off, parent, 4, *kv, table, lens, q, lse, ws)
    refused(ValueError, "q must be", tree, cfg, q[:, :4], off, parent, 4, *kv, table, lens, q, lse, ws)
    refused(TypeError, "table must be torch.Int", tree, cfg, q, off, parent, 4, *kv, table.long(), lens, q, lse, ws)
    refused(ValueError, r"q must be \[2", qb.qsa_paged_decode_weights, cfg, q, *kv, table, lens, q, lse, weights, ws)
    refused(ValueError, "q is on cpu", qb.qsa_paged_decode_weights, cfg, q[:2], *kv, table, lens, q[:2], lse[:2], weights, ws)
    planes, ref = [torch.zeros(3, 6, 4)], torch.zeros(6, **i32)
    refused(ValueError, "table is on cpu", qb.qsa_accept_drafts, 4, off, parent, lens, table, lens, ref, table, lens, ref, planes, ws)
    refused(ValueError, "table is on cpu", qb.qsa_evict_tokens, 4, lens, 0, 0, weights, table, table, lens, ref, weights, table, table,
            lens, ref, planes, ws)
    with pytest.raises(qb.QsaError):
        qb.tree_workspace(cfg, 0, device="cpu")
    with pytest.raises(qb.QsaError):
        qb.weights_workspace(paged_cfg(head_dim=96), 4, 4, device="cpu")
    with pytest.raises(qb.QsaError):
        qb.keep_workspace(-1, device="cpu")


def test_kernels_that_begin_early_use_no_read_only_loads():
    for name in ("paged_decode.cuh", "paged_weights.cu", "tree_decode.cu", "keep.cu"):
        with open(os.path.join(qbuild.CSRC, name)) as f:
            code = [line.split("//")[0] for line in f]
        assert not any("ld.global.nc" in line or "ldg_nc" in line or "__ldg(" in line for line in code), name


def test_oracle_of_trees_and_eviction_by_hand():
    #        0 -> 1 -> 3, 0 -> 2, and 4 alone; five cached tokens before them
    parent = [-1, 0, 0, 1, -1]
    assert T.lines(parent) == [[0], [0, 1], [0, 2], [0, 1, 3], [4]]
    seen = T.attended(10, parent)
    assert seen[3] == [0, 1, 2, 3, 4, 5, 6, 8] and seen[4] == [0, 1, 2, 3, 4, 9]
    assert T.attended(10, parent, 3)[3] == [5, 6, 8] and T.attended(10, parent, 4)[0] == [2, 3, 4, 5]
    assert T.accept(10, parent, 3) == (8, [(7, 8)]) and T.accept(10, parent, -1) == (5, []) and T.accept(10, parent, 4) == (6, [(5, 9)])
    w, pos = [5.0, 1.0, 1.0, 7.0, 0.0, 2.0], [3, 0, 9, 5, 10, 4]
    none = [False] * 6
    assert T.evict(w, pos, none, 6, 0, 0) == (6, []) and T.evict(w, pos, none, -1, 0, 0) == (6, [])
    assert T.evict(w, pos, none, 3, 0, 0) == (3, [(1, 3), (2, 5)])          # 5, 7 and 2 stay
    assert T.evict(w, pos, none, 3, 1, 1) == (3, [(0, 3), (2, 4)])          # positions 0 and 10, and 7
    assert T.evict(w, pos, [True] * 4 + [False] * 2, 2, 0, 0) == (4, [])    # four in shared pages
    table, ref = T.release([[4, 2, -1], [1, 0, 3]], [1, 1, 1, 1, 1], [5, 9], [3, 4], 4)
    assert table.tolist() == [[4, -1, -1], [1, -1, -1]] and ref.tolist() == [0, 1, 0, 0, 1]


def test_a_cache_refuses_what_it_was_not_made_for():
    cache = object.__new__(PagedCache)                    # no GPU here: only what the checks read
    cache.max_draft, cache.evictable, cache.planes = 0, False, []
    for call in (lambda: cache.attend_tree(0, None, None, None, None), lambda: cache.accept(None, None, None)):
        with pytest.raises(ValueError, match="max_draft"):
            call()
    for call in (lambda: cache.evict(None, 0, 0), lambda: cache.attend(0, None, None, weigh=True)):
        with pytest.raises(ValueError, match="evictable"):
            call()
