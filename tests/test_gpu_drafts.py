"""The paged cache's operators for drafted tokens and eviction on the GPU against a plain 64-bit implementation: tokens
stored at a place that is not their position, attention of a tree of drafted tokens, accepting its path, attention that
accumulates each token's weight, evicting the lightest tokens, and runs of them together.

Tolerances. Those of the paged attention's tests (scores: D 2^-24 of the terms and 2^-21; a weight twice that, 2^-15 and the
fp32 sums over n tokens; the result's own rounding to bf16, 2^-8), and:
- a tree's weights enter the second product as bf16, half a step of its 8 bits, 2^-8 of each (over FP8 rows with V's scale
  as f16: 2^-11 of each, and 2^-31 of the largest below f16's normal range);
- an accumulated weight sums Hq weights, each off by twice its score's error and 2^-21 for the exponential, and adds them
  in fp32: (Hq + 1) 2^-24 of the sum."""

import numpy as np
import pytest
import torch

from indexer_driven_sparse_gb300 import binding as qb
from indexer_driven_sparse_gb300.pipeline import PagedCache
from oracle import drafts_oracle as T
from oracle import paged_oracle as P
from tests.test_gpu_paged import DECODE_GEOMETRY, DEV, check_decode, f64, ints, paged_inputs, randn, run_decode, status

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ places and positions
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_append_at_a_place(cuda_lib, fp8, inter):
    """The bits that qsa_rope_append writes at position p are those that qsa_rope_append_at writes at place x for position p."""
    n, Hq, Hkv, D, page, rows, ld = 37, 8, 2, 128, 5, 3, 9
    rng = np.random.default_rng(3)
    room = ld * page
    flat = rng.permutation(rows * room)[:n]
    seq, place = flat // room, flat % room
    seq[5], pos = -1, rng.integers(0, room, n)
    used = {}
    for i in range(n):                                    # positions distinct within a row, to compare by
        while (seq[i], pos[i]) in used:
            pos[i] = (pos[i] + 1) % room
        used[(seq[i], pos[i])] = i
    table = ints(rng.permutation(rows * ld).reshape(rows, ld).tolist())
    x = randn((n, Hq + 2 * Hkv, D), 1)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cfg = qb.make_paged_config(Hq, Hkv, D, page)
    ws = qb.paged_workspace(cfg)
    rope = qb.rope_table(D, 64, interleaved=inter, base=1e5)

    def planes():
        shape = (rows * ld, page, Hkv, D)
        if fp8:
            return [torch.full(shape[:3] + (w,), 9, dtype=t, device=DEV)
                    for w, t in ((D, torch.uint8), (1, torch.float32)) * 2]
        return [torch.full(shape, 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    a, b = planes(), planes()
    qa, qb_ = torch.full((2, n, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    positions = torch.full((rows, room - 2), -7, dtype=torch.int32, device=DEV)
    s, p, at = ints(seq.tolist()), ints(pos.tolist()), ints(place.tolist())
    if fp8:
        qb.qsa_rope_append_fp8kv(cfg, rope, q, k, v, p, s, qa, a, table, ws)
        qb.qsa_rope_append_at_fp8kv(cfg, rope, q, k, v, p, at, s, qb_, b, table, ws, positions)
    else:
        qb.qsa_rope_append(cfg, rope, q, k, v, p, s, qa, *a, table, ws)
        qb.qsa_rope_append_at(cfg, rope, q, k, v, p, at, s, qb_, *b, table, ws, positions)
    assert torch.equal(qa, qb_) and status(ws) == (0, 0)
    tab, want = table.cpu().numpy(), np.full((rows, room - 2), -7)
    for i in range(n):
        if seq[i] < 0:
            continue
        if place[i] < room - 2:
            want[seq[i], place[i]] = pos[i]
        for u, w in zip(a, b):
            assert torch.equal(u[tab[seq[i], pos[i] // page], pos[i] % page], w[tab[seq[i], place[i] // page], place[i] % page])
    assert np.array_equal(positions.cpu().numpy(), want)
    places = {(tab[s_, x_ // page], x_ % page) for s_, x_ in zip(seq, place) if s_ >= 0}
    for w in b:                                           # nothing else is written
        rest = [(g, o) for g in range(rows * ld) for o in range(page) if (g, o) not in places]
        assert bool((w[[g for g, _ in rest], [o for _, o in rest]] == 9).all())


@pytest.mark.parametrize("seq,place,page", [(3, 0, 0), (0, -1, 0), (0, 16, 0), (0, 3, -1), (0, 3, 4)])
def test_append_at_skips_and_records_bad_places(cuda_lib, seq, place, page):
    cfg = qb.make_paged_config(4, 1, 64, 4)
    ws = qb.paged_workspace(cfg)
    kc, vc = torch.full((2, 4, 4, 1, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    table = ints([[page, page, page, page]] * 3)
    positions = torch.full((3, 16), -7, dtype=torch.int32, device=DEV)
    q = randn((1, 4, 64), 1)
    out = torch.zeros_like(q)
    qb.qsa_rope_append_at(cfg, qb.rope_table(64), q, q[:, :1], q[:, 1:2], ints([2]), ints([place]), ints([seq]), out, kc, vc,
                          table, ws, positions)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0)
    assert bool((vc == 5).all()) and bool((kc == 5).all()) and bool((positions == -7).all()) and bool(out.any())


# ------------------------------------------------------------------------------------------ trees
def random_parents(rng, count, chain=0.6):
    """Parents of `count` tokens: mostly chains."""
    return [i - 1 if rng.random() < chain else int(rng.integers(-1, i)) if i else -1 for i in range(count)]


def tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed, spare_rows=3, scale=1.0, chain=0.6):
    rng = np.random.default_rng(seed)
    q0, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, page, fp8, seed, scale=scale)
    off = np.concatenate([[0], np.cumsum(counts)])
    parents = [random_parents(rng, c, chain) for c in counts]
    n = int(off[-1]) + spare_rows
    q = randn((n, Hq, D), seed + 7)
    return q, planes, values, tab, table, off.tolist(), parents


def run_tree(cfg, q, planes, tab, lens, off, parents, max_draft, ws, out=None, lse=None, stream=None):
    n = q.shape[0]
    out = torch.full((n, cfg.n_q_heads, cfg.head_dim), 8.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((n, cfg.n_q_heads), 8.0, device=DEV) if lse is None else lse
    flat = [p for row in parents for p in row]
    parent = ints(flat + [-5] * (n - len(flat)))
    if len(planes) == 2:
        qb.qsa_tree_decode(cfg, q, ints(off), parent, max_draft, *planes, tab, ints(lens), out, lse, ws, stream)
    else:
        qb.qsa_tree_decode_fp8kv(cfg, q, ints(off), parent, max_draft, planes, tab, ints(lens), out, lse, ws, stream)
    return out, lse


def check_tree(out, lse, q, values, table, lens, off, parents, page, scale, window=0, fp8=False, leave_out={}):
    out, lse, q = f64(out), f64(lse), f64(q)
    D = q.shape[-1]
    for r, n in enumerate(lens):
        slots = P.slots_of(np.maximum(table[r], 0), n, page)
        K, V = (x.reshape(-1, *x.shape[2:])[slots] for x in values)
        for i, (want, want_lse, mass, terms, seen) in enumerate(
                T.tree(q[off[r]:off[r + 1]], K, V, parents[r], scale, window, leave_out.get(r, ()))):
            got, got_lse = out[off[r] + i], lse[off[r] + i]
            if seen == 0:
                assert np.all(got == 0) and np.all(np.isneginf(got_lse))
                continue
            ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1)
            sums = seen / 8 * 2.0 ** -24 + 2.0 ** -15
            tol = 2.0 ** -8 * np.abs(want) + (2 * ds[:, None] + sums + (2.0 ** -11 if fp8 else 2.0 ** -8)) * mass
            if fp8:
                tol += seen * 2.0 ** -31 * mass.max(1, keepdims=True)
            assert np.all(np.abs(got - want) <= tol), (r, i, np.abs(got - want).max(), tol.min())
            assert np.all(np.abs(got_lse - want_lse) <= ds + sums + 2.0 ** -22 * np.abs(want_lse)), (r, i)
    assert np.all(out[off[-1]:] == 8) and np.all(lse[off[-1]:] == 8)      # rows that no sequence names


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", DECODE_GEOMETRY)
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([5, 0, 3, 64, 65, 66, 1], [5, 0, 2, 1, 0, 66, 0]), ([127, 128, 129, 130, 200, 257], [1, 2, 7, 33, 16, 128]),
    ([3000, 700], [12, 31]), ([17, 1500, 64, 700], [16, 20, 64, 100])])
@pytest.mark.parametrize("window", [0, 50])
def test_tree(cuda_lib, Hq, Hkv, D, page, fp8, lens, counts, window):
    if max(counts) * Hq > 600:                            # keeps the oracle quick
        counts = [min(c, 600 // Hq) for c in counts]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed=Hq + D + len(lens))
    cfg = qb.make_paged_config(Hq, Hkv, D, page, window=window)
    ws = qb.tree_workspace(cfg, max(counts))
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, max(counts), ws)
    assert status(ws) == (0, 0)
    check_tree(out, lse, q, values, table, lens, off, parents, page, D ** -0.5, window, fp8)
    again, lse2 = run_tree(cfg, q, planes, tab, lens, off, parents, max(counts), ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    third = torch.full_like(out, 8.0)                     # without lse
    parent = ints([p for row in parents for p in row] + [-1] * 3)
    if fp8:
        qb.qsa_tree_decode_fp8kv(cfg, q, ints(off), parent, max(counts), planes, tab, ints(lens), third, None, ws)
    else:
        qb.qsa_tree_decode(cfg, q, ints(off), parent, max(counts), *planes, tab, ints(lens), third, None, ws)
    assert torch.equal(out, third)


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", [(16, 2, 256, 64, False), (8, 2, 128, 16, False), (4, 4, 64, 100, False),
                                               (16, 1, 256, 48, True), (32, 8, 128, 24, True)])
@pytest.mark.parametrize("max_draft", [8, 64])
def test_tree_long_and_many(cuda_lib, Hq, Hkv, D, page, fp8, max_draft):
    """Rows of very different lengths and trees, more of them than fit in one wave; a scale of its own."""
    rng = np.random.default_rng(max_draft)
    lens = [9000] + rng.integers(0, 200, 150).tolist() + [4000, 1]
    counts = [min(n, int(c)) for n, c in zip(lens, rng.integers(0, 4, len(lens)))]
    counts[0], counts[7] = min(max_draft, 12), min(lens[7], max_draft)
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed=9)
    cfg = qb.make_paged_config(Hq, Hkv, D, page, softmax_scale=0.11)
    ws = qb.tree_workspace(cfg, max_draft)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, max_draft, ws)
    assert status(ws) == (0, 0)
    check_tree(out, lse, q, values, table, lens, off, parents, page, float(np.float32(0.11)), 0, fp8)


@pytest.mark.parametrize("Hq,Hkv,D,fp8", [(16, 2, 256, False), (6, 1, 128, False), (8, 1, 64, False), (16, 2, 256, True),
                                          (9, 1, 128, True)])
def test_a_tree_of_one_token_is_the_decode(cuda_lib, Hq, Hkv, D, fp8):
    """One drafted token a row: the attention of qsa_paged_decode, within both operators' roundings."""
    lens = [1, 64, 130, 1000, 4097]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, [1] * 5, Hq, Hkv, D, 16, fp8, seed=4, spare_rows=0)
    cfg = qb.make_paged_config(Hq, Hkv, D, 16)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 1, qb.tree_workspace(cfg, 1))
    want, want_lse = run_decode(cfg, q, planes, tab, ints(lens), qb.paged_workspace(cfg))
    # both are 2^-8 of a value off by their own rounding, and 2^-8 of the mean |V| by the weights'; |V| is below 5 here
    assert bool(((out - want).abs().float() <= 2.0 ** -7 * want.abs().float() + 2.0 ** -8 * 5).all())
    assert bool(((lse - want_lse).abs() <= 1e-4).all())
    check_tree(out, lse, q, values, table, lens, off, parents, 16, D ** -0.5, 0, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_chain_is_causal_attention(cuda_lib, fp8):
    lens, counts = [40, 300], [40, 37]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, 8, 2, 128, 16, fp8, seed=2, chain=2.0)
    assert parents[1] == list(range(-1, 36))
    cfg = qb.make_paged_config(8, 2, 128, 16)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 40, qb.tree_workspace(cfg, 40))
    for r, n in enumerate(lens):
        for i in (0, 1, counts[r] - 1):                   # token i sees what a row cut behind it holds
            cut = n - counts[r] + i + 1
            w = run_tree(cfg, q[off[r] + i:off[r] + i + 1], planes, tab[r:r + 1], [cut], [0, 1], [[-1]], 1,
                         qb.tree_workspace(cfg, 1))
            diff = (w[0][0] - out[off[r] + i]).abs().float()
            assert bool((diff <= 2.0 ** -7 * w[0][0].abs().float() + 2.0 ** -8 * 5).all())
            assert bool(((w[1][0] - lse[off[r] + i]).abs() <= 1e-4).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_sharp_scores(cuda_lib, fp8):
    """Scores of hundreds: the weights of almost all tokens vanish, and the running maximum moves often."""
    lens, counts = [1500, 260], [9, 16]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, 16, 2, 256, 32, fp8, seed=8, scale=12.0)
    cfg = qb.make_paged_config(16, 2, 256, 32, softmax_scale=1.0)
    ws = qb.tree_workspace(cfg, 16)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 16, ws)
    check_tree(out, lse, q, values, table, lens, off, parents, 32, 1.0, 0, fp8)


def test_tree_strided_queries_and_another_stream(cuda_lib):
    lens, counts = [400, 20], [6, 3]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, 16, 2, 256, 16, False, seed=3)
    wide = torch.full((q.shape[0], 20, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:18] = q
    cfg = qb.make_paged_config(16, 2, 256, 16)
    ws = qb.tree_workspace(cfg, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = run_tree(cfg, wide[:, 2:18], planes, tab, lens, off, parents, 6, ws, stream=side)
    side.synchronize()
    check_tree(out, lse, q, values, table, lens, off, parents, 16, 1 / 16, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_leaves_out_and_records_bad_pages(cuda_lib, fp8):
    lens, counts = [100, 50, 70], [4, 2, 3]
    Hq, Hkv, D, page = 8, 2, 128, 8
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed=5)
    bad = tab.clone()
    bad[0, 3], bad[1, 0], bad[1, 6] = -1, planes[0].shape[0], 2 ** 31 - 1
    cfg = qb.make_paged_config(Hq, Hkv, D, page)
    ws = qb.tree_workspace(cfg, 4)
    out, lse = run_tree(cfg, q, planes, bad, lens, off, parents, 4, ws)
    st, detail = status(ws)
    assert st == qb.QSA_ERR_DEVICE_BOUNDS and detail in (0, 1)
    gone = {0: range(24, 32), 1: list(range(8)) + [48, 49]}
    check_tree(out, lse, q, values, table, lens, off, parents, page, D ** -0.5, 0, fp8, gone)


@pytest.mark.parametrize("lens,off,max_draft,bad", [
    ([30, 40, 20], [0, 5, 9, 12], 4, 0),                  # more drafted tokens than max_draft
    ([30, 2, 20], [0, 4, 8, 12], 4, 1),                   # more drafted tokens than cached ones
    ([30, 40, 10 ** 6], [0, 4, 8, 12], 4, 2),             # longer than its table row
    ([30, -3, 20], [0, 4, 8, 12], 4, 1)])
def test_tree_rows_out_of_range_attend_nothing(cuda_lib, lens, off, max_draft, bad):
    fine = [30, 40, 20]
    counts = np.diff(off).tolist()
    q, planes, values, tab, table, _, parents = tree_inputs(fine, counts, 8, 2, 128, 8, False, seed=6)
    cfg = qb.make_paged_config(8, 2, 128, 8)
    ws = qb.tree_workspace(cfg, max_draft)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, max_draft, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, bad)
    assert not out[off[bad]:off[bad + 1]].any() and bool(torch.isneginf(lse[off[bad]:off[bad + 1]]).all())
    want, _ = run_tree(cfg, q, planes, tab, fine, off, parents, 5, qb.tree_workspace(cfg, 5))
    for r in range(3):
        if r != bad:
            diff = (out[off[r]:off[r + 1]] - want[off[r]:off[r + 1]]).abs().float()
            assert bool((diff <= 0.05).all()) and bool((lse[off[r]:off[r + 1]] < 8).all())


def test_tree_offsets_out_of_range(cuda_lib):
    """Descending offsets and offsets behind N: those rows attend nothing, and nothing outside the arrays is touched."""
    lens, counts = [30, 40, 20], [4, 4, 4]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, 8, 2, 128, 8, False, seed=6, spare_rows=0)
    cfg = qb.make_paged_config(8, 2, 128, 8)
    ws = qb.tree_workspace(cfg, 8)
    good, _ = run_tree(cfg, q, planes, tab, lens, off, parents, 8, ws)
    assert status(ws) == (0, 0)
    for bad in ([0, 4, 2, 12], [0, 4, 8, 15], [-2, 4, 8, 12], [0, 4, 2 ** 31 - 1, 12], [5, 4, -2 ** 31, 2 ** 31 - 1]):
        ws = qb.tree_workspace(cfg, 8)
        out, lse = run_tree(cfg, q, planes, tab, lens, bad, parents, 8, ws)
        assert status(ws)[0] == qb.QSA_ERR_DEVICE_BOUNDS
        if bad[:2] == [0, 4]:
            assert bool(((out[:4] - good[:4]).abs() <= 0.05).all())


@pytest.mark.parametrize("parent,as_if", [([-1, 5, 1, 2], [-1, -1, 1, 2]), ([-1, 0, 2, 2], [-1, 0, -1, 2]), ([-2, 0, 1, 9], [-1, 0, 1, -1])])
def test_tree_parents_out_of_range_count_as_none(cuda_lib, parent, as_if):
    lens = [60]
    q, planes, values, tab, table, off, _ = tree_inputs(lens, [4], 8, 2, 128, 8, False, seed=6)
    cfg = qb.make_paged_config(8, 2, 128, 8)
    ws = qb.tree_workspace(cfg, 4)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, [parent], 4, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0)
    check_tree(out, lse, q, values, table, lens, off, [as_if], 8, 128 ** -0.5, 0)


def test_tree_captured_replays_with_new_lengths(cuda_lib):
    lens, counts = [500, 90], [6, 5]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, 16, 2, 256, 16, False, seed=12)
    cfg = qb.make_paged_config(16, 2, 256, 16)
    ws = qb.tree_workspace(cfg, 9)
    first = run_tree(cfg, q, planes, tab, lens, off, parents, 9, ws)       # before the capture
    out, lse = (torch.full_like(t, 8.0) for t in first)
    lens_d, off_d = ints(lens), ints(off)
    parent = ints([p for row in parents for p in row] + [-1] * 3)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        qb.qsa_tree_decode(cfg, q, off_d, parent, 9, *planes, tab, lens_d, out, lse, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    lens_d.copy_(ints([333, 47]))
    off_d.copy_(ints([0, 2, 11]))
    out.fill_(8.0), lse.fill_(8.0)
    parents = [[-1, 0], random_parents(np.random.default_rng(1), 9)]
    parent.copy_(ints(parents[0] + parents[1] + [-1] * 3))
    graph.replay()
    torch.cuda.synchronize()
    check_tree(out, lse, q, values, table, [333, 47], [0, 2, 11], parents, 16, 1 / 16, 0)
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", [(16, 2, 256, 64, False), (16, 2, 256, 5, False), (8, 2, 128, 16, True),
                                               (16, 2, 256, 5, True), (16, 2, 64, 16, False)])
@pytest.mark.parametrize("lens,counts", [([30000, 700], [9, 16]), ([150] * 200, [3, 32] * 100)])
def test_tree_device_timeout_is_reported(cuda_lib, Hq, Hkv, D, page, fp8, lens, counts):
    """The header's test knob stops every CTA's index warp at its fourth tile: all roles that wait for what it would have named give up
    within the limit, in the middle of a sequence's tiles and between sequences, and the next call is as if nothing had been."""
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed=7)
    cfg = qb.make_paged_config(Hq, Hkv, D, page)
    ws = qb.tree_workspace(cfg, max(counts))
    good, good_lse = run_tree(cfg, q, planes, tab, lens, off, parents, max(counts), ws)
    assert status(ws) == (0, 0)
    ws.view(torch.int32)[3] = 0x5741171
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    run_tree(cfg, q, planes, tab, lens, off, parents, max(counts), ws)
    end.record()
    assert status(ws)[0] == qb.QSA_ERR_DEVICE_TIMEOUT
    assert begin.elapsed_time(end) < 2 * 250              # one limit of 250 ms for all waits of a CTA, all CTAs at once
    qb.qsa_workspace_init(ws)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, max(counts), ws)
    assert status(ws) == (0, 0) and torch.equal(out, good) and torch.equal(lse, good_lse)


# ------------------------------------------------------------------------------------------ accumulated weights
def run_weights(cfg, q, planes, tab, lens, weights, ws, stream=None, lse=True):
    out = torch.full((q.shape[0], cfg.n_q_heads, cfg.head_dim), 8.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((q.shape[0], cfg.n_q_heads), 8.0, device=DEV) if lse else None
    if len(planes) == 2:
        qb.qsa_paged_decode_weights(cfg, q, *planes, tab, lens, out, lse, weights, ws, stream)
    else:
        qb.qsa_paged_decode_weights_fp8kv(cfg, q, planes, tab, lens, out, lse, weights, ws, stream)
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", DECODE_GEOMETRY)
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 0, 127, 129], [5, 0, 1500, 700, 64, 0] + [3] * 40])
@pytest.mark.parametrize("window", [0, 50])
def test_weights(cuda_lib, Hq, Hkv, D, page, fp8, lens, window):
    q, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, page, fp8, seed=Hq + D + len(lens))
    cfg = qb.make_paged_config(Hq, Hkv, D, page, window=window)
    want = run_decode(cfg, q, planes, tab, ints(lens), qb.paged_workspace(cfg))
    ws = qb.weights_workspace(cfg, len(lens), sum(lens))
    before = torch.rand(len(lens), max(lens) + 3, generator=torch.Generator().manual_seed(1)).to(DEV)
    weights = before.clone()
    out, lse = run_weights(cfg, q, planes, tab, ints(lens), weights, ws)
    assert status(ws) == (0, 0)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])        # bit for bit
    got, old, q64 = f64(weights), f64(before), f64(q)
    for r, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        assert np.array_equal(got[r, n:], old[r, n:]) and np.array_equal(got[r, :lo], old[r, :lo])
        if n == 0:
            continue
        slots = P.slots_of(table[r], n, page)
        K, V = (x.reshape(-1, *x.shape[2:])[slots] for x in values)
        add = T.token_weights(q64[r], K, lo, D ** -0.5)
        terms = P.decode(q64[r], K, V, lo, D ** -0.5)[3].max()
        ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1)
        tol = (4 * ds + 2.0 ** -20 + n / 8 * 2.0 ** -24 + (Hq + 1) * 2.0 ** -24) * add + 2.0 ** -24 * (old[r, :n] + add)
        assert np.all(np.abs(got[r, :n] - old[r, :n] - add) <= tol + 1e-37), r
    twice = before.clone()                                # the same bits again, and without lse
    run_weights(cfg, q, planes, tab, ints(lens), twice, ws, lse=False)
    assert torch.equal(twice, weights)


def test_weights_behind_the_array_or_the_workspace_add_nothing(cuda_lib):
    lens = [300, 200]
    q, planes, values, tab, table = paged_inputs(lens, 8, 2, 128, 16, False, seed=1)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    full = torch.zeros(2, 300, device=DEV)
    run_weights(cfg, q, planes, tab, ints(lens), full, qb.weights_workspace(cfg, 2, 500))
    ws = qb.weights_workspace(cfg, 2, 500)
    short = torch.zeros(2, 250, device=DEV)
    out, _ = run_weights(cfg, q, planes, tab, ints(lens), short, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0) and torch.equal(short, full[:, :250])
    ws = qb.weights_workspace(cfg, 2, 0)                  # room for four tiles of the nine
    some = torch.zeros(2, 300, device=DEV)
    again, _ = run_weights(cfg, q, planes, tab, ints(lens), some, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, -1) and torch.equal(again, out)
    held = some != 0
    assert bool(held.any()) and not bool(held.all()) and torch.equal(some[held], full[held])


def test_weights_sum_to_the_heads_over_many_steps(cuda_lib):
    """Every step adds a total of Hq to a row: each weight is within 2^-18 relative (scores' and exponential's errors are
    below that here), each of the 50 additions rounds a total below 2^10 in fp32."""
    lens = [777, 64, 1]
    q, planes, values, tab, table = paged_inputs(lens, 16, 2, 256, 16, False, seed=1)
    cfg = qb.make_paged_config(16, 2, 256, 16)
    ws = qb.weights_workspace(cfg, 3, sum(lens))
    weights = torch.zeros(3, 800, device=DEV)
    for _ in range(50):
        run_weights(cfg, q, planes, tab, ints(lens), weights, ws)
    assert np.allclose(f64(weights).sum(1), 800.0, rtol=2.0 ** -18 + 50 * 2.0 ** -24, atol=0)


# ------------------------------------------------------------------------------------------ accepting
def token_planes(n_pages, page, seed):
    """Plane groups of tokens of 48 bytes (16-byte words), of 4 bytes and of 20 bytes."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-2 ** 15, 2 ** 15, (3, n_pages, page, 24), dtype=torch.int16, generator=g).to(DEV),
            torch.randn((2, n_pages, page, 1), generator=g).to(DEV), torch.randn((1, n_pages, page, 5), generator=g).to(DEV)]


def moved(plane, table, moves, page):
    """The plane after moves {row: [(to, from)]}, all read before any is written."""
    want = plane.clone()
    for r, some in moves.items():
        for to, at in some:
            want[:, table[r][to // page], to % page] = plane[:, table[r][at // page], at % page]
    return want


def private_pool(lens, page, seed, spare=3, shared=0):
    """Page table, references and lengths; the last row shares row 0's first `shared` pages."""
    rng = np.random.default_rng(seed)
    count = [-(-n // page) for n in lens]
    ld, n_pages = max(count + [1]) + 1, sum(count) + spare
    order, at = rng.permutation(n_pages), 0
    table, ref = np.full((len(lens), ld), -1, np.int32), np.zeros(n_pages, np.int32)
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        at += c
    if shared:
        k = min(shared, lens[0] // page, lens[-1] // page)
        table[-1, :k] = table[0, :k]
    for r, c in enumerate(count):
        np.add.at(ref, table[r, :c], 1)
    return table, ref


def filled(*shape):
    return torch.full(shape, 77, dtype=torch.int32, device=DEV)


ACCEPT_ROWS = [([9], [4]), ([40, 0, 7, 1, 200, 128], [8, 0, 7, 1, 128, 128]), ([300] * 70, [33] * 70),
               ([20, 21, 22] * 500, [3, 0, 1] * 500)]


@pytest.mark.parametrize("lens,counts", ACCEPT_ROWS)
@pytest.mark.parametrize("page", [1, 4, 24])
def test_accept(cuda_lib, lens, counts, page):
    rng = np.random.default_rng(len(lens) + page)
    table, ref = private_pool(lens, page, 1)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    parents = [random_parents(rng, c, 0.5) for c in counts]
    last = [int(rng.integers(-1, c)) if c else -1 for c in counts]
    cut = [T.accept(n, p, a) for n, p, a in zip(lens, parents, last)]
    new_len = np.array([c[0] for c in cut])
    moves = {r: c[1] for r, c in enumerate(cut)}
    planes = token_planes(len(ref), page, 1)
    want = [moved(p, table, moves, page) for p in planes]
    ld = table.shape[1]
    t_out, l_out, r_out = filled(len(lens), ld), filled(len(lens)), filled(len(ref))
    positions = ints(rng.integers(0, 1000, (len(lens), ld * page - 1)).tolist())
    want_pos = positions.cpu().numpy().copy()
    for r, some in moves.items():
        old = want_pos[r].copy()
        for to, at in some:
            want_pos[r, to] = old[at]
    ws = qb.keep_workspace(len(lens))
    flat = ints([p for row in parents for p in row] + [0, 0])
    args = (page, ints(off), flat, ints(last), ints(table.tolist()), ints(lens), ints(ref.tolist()))
    qb.qsa_accept_drafts(*args, t_out, l_out, r_out, planes, ws, positions)
    assert status(ws) == (0, 0)
    want_t, want_r = T.release(table, ref, lens, new_len, page)
    assert np.array_equal(l_out.cpu().numpy(), new_len) and np.array_equal(t_out.cpu().numpy(), want_t)
    assert np.array_equal(r_out.cpu().numpy(), want_r) and np.array_equal(positions.cpu().numpy(), want_pos)
    for got, w in zip(planes, want):
        assert torch.equal(got, w)
    r_out.fill_(77)
    qb.qsa_accept_drafts(*args, t_out, l_out, r_out, [], ws)               # no planes, no positions
    assert np.array_equal(r_out.cpu().numpy(), want_r)


@pytest.mark.parametrize("lens,counts", ACCEPT_ROWS)
@pytest.mark.parametrize("cut", [0, 5])
def test_accept_moves_weights_along(cuda_lib, lens, counts, cut):
    """Weights and positions follow the accepted path and are cleared where tokens are dropped, in arrays of all places and in
    shorter ones; the rest of the call is qsa_accept_drafts."""
    page, rng = 4, np.random.default_rng(len(lens) + cut)
    table, ref = private_pool(lens, page, 1)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    parents = [random_parents(rng, c, 0.5) for c in counts]
    last = [int(rng.integers(-1, c)) if c else -1 for c in counts]
    held = list(lens)
    if len(lens) > 3:                                     # a row out of range keeps what it has
        last[4] = counts[4]
    places = max(1, max(lens) - cut)
    positions = rng.integers(0, 1000, (len(lens), places)).astype(np.int32)
    weights = rng.random((len(lens), places)).astype(np.float32)
    want_p, want_w, moves, new_len = positions.copy(), weights.copy(), {}, []
    for r, (n, p, a) in enumerate(zip(lens, parents, last)):
        new, moves[r] = T.accept(n, p, a) if a < len(p) else (n, [])
        new_len.append(new)
        for to, at in moves[r]:
            if at < places:
                want_p[r, to], want_w[r, to] = positions[r, at], weights[r, at]
        want_p[r, new:n], want_w[r, new:n] = -1, 0
    planes = token_planes(len(ref), page, 1)
    want = [moved(p, table, moves, page) for p in planes]
    t_out, l_out, r_out = filled(*table.shape), filled(len(lens)), filled(len(ref))
    ws = qb.keep_workspace(len(lens))
    pos, w = ints(positions.tolist()), torch.from_numpy(weights).to(DEV)
    qb.qsa_accept_drafts_weights(page, ints(off), ints([p for row in parents for p in row] + [0]), ints(last), w, pos,
                                 ints(table.tolist()), ints(held), ints(ref.tolist()), t_out, l_out, r_out, planes, ws)
    assert status(ws) == ((qb.QSA_ERR_DEVICE_BOUNDS, 4) if len(lens) > 3 else (0, 0))
    fine = np.array([r for r in range(len(lens)) if last[r] < counts[r] or last[r] < 0])
    want_t, want_r = T.release(table[fine], ref, np.array(lens)[fine], np.array(new_len)[fine], page)
    assert l_out.tolist() == new_len and np.array_equal(t_out.cpu().numpy()[fine], want_t)
    assert np.array_equal(r_out.cpu().numpy(), want_r)
    for r in range(len(lens)):                            # what of a moved token lies behind the arrays is nothing to compare
        sure = [j for j in range(places) if not any(to == j and at >= places for to, at in moves[r])]
        assert np.array_equal(pos[r].cpu().numpy()[sure], want_p[r, sure]), r
        assert np.array_equal(w[r].cpu().numpy()[sure], want_w[r, sure]), r
    for got, x in zip(planes, want):
        assert torch.equal(got, x)


@pytest.mark.parametrize("what", ["length", "long", "drafts", "offset", "parent", "accepted"])
def test_accept_leaves_rows_out_of_range_as_they_are(cuda_lib, what):
    page, lens, off, parents, last = 4, [10, 12, 9], [0, 4, 8, 12], [[-1, 0, 1, 2]] * 3, [1, 3, 2]
    table, ref = private_pool(lens, page, 1)
    held = [10, 12, 9]
    parents = [list(p) for p in parents]
    if what == "length":
        held[1] = -1
    elif what == "long":
        held[1] = 10 ** 6
    elif what == "drafts":
        held[1] = 3
    elif what == "offset":
        off = [0, 4, 8, 99]
    elif what == "parent":
        parents[1][2] = 2
    else:
        last[1] = 4
    bad = 2 if what == "offset" else 1
    planes = token_planes(len(ref), page, 1)
    cut = [T.accept(n, [-1, 0, 1, 2], a) if r != bad else (held[r], []) for r, (n, a) in enumerate(zip(lens, last))]
    want = [moved(p, table, {r: c[1] for r, c in enumerate(cut)}, page) for p in planes]
    t_out, l_out, r_out = filled(3, table.shape[1]), filled(3), filled(len(ref))
    ws = qb.keep_workspace(3)
    qb.qsa_accept_drafts(page, ints(off), ints(sum(parents, [])), ints(last), ints(table.tolist()), ints(held),
                         ints(ref.tolist()), t_out, l_out, r_out, planes, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, bad)
    fine = [r for r in range(3) if r != bad]
    new_len = [c[0] for c in cut]
    assert l_out.tolist() == new_len
    want_t, want_r = T.release(table[fine], ref, [lens[r] for r in fine], [new_len[r] for r in fine], page)
    assert np.array_equal(t_out.cpu().numpy()[fine], want_t) and np.array_equal(t_out[bad].cpu().numpy(), table[bad])
    assert np.array_equal(r_out.cpu().numpy(), want_r)
    for got, w in zip(planes, want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("parent,last", [([-1, 0, 2, 1], 1), ([-1, 0, -2, 1], 3), ([-1, 0, 1, 7], -1), ([0, -1, 1, -1], 3)])
def test_accept_leaves_rows_with_any_parent_out_of_range(cuda_lib, parent, last):
    """A parent out of range that the accepted path does not meet; the row beside it is cut."""
    page, lens, off = 4, [10, 12], [0, 4, 8]
    table, ref = private_pool(lens, page, 1)
    planes = token_planes(len(ref), page, 1)
    want = [p.clone() for p in planes]
    t_out, l_out, r_out, ws = filled(2, table.shape[1]), filled(2), filled(len(ref)), qb.keep_workspace(2)
    positions = ints(np.arange(24).reshape(2, 12).tolist())
    qb.qsa_accept_drafts(page, ints(off), ints(parent + [-1, 0, 1, 2]), ints([last, 1]), ints(table.tolist()), ints(lens),
                         ints(ref.tolist()), t_out, l_out, r_out, planes, ws, positions)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0) and l_out.tolist() == [10, 10]
    want_t, want_r = T.release(table, ref, lens, [10, 10], page)
    assert np.array_equal(t_out.cpu().numpy(), want_t) and np.array_equal(r_out.cpu().numpy(), want_r)
    assert positions.flatten().tolist() == list(range(24)) and all(torch.equal(a, b) for a, b in zip(planes, want))


# ------------------------------------------------------------------------------------------ evicting
def run_evict(page, budget, first, recent, weights, positions, table, lens, ref, planes, ws=None):
    S, places = weights.shape
    w_out, p_out = torch.full_like(weights, 77.0), torch.full_like(positions, 77)
    t_out, l_out, r_out = filled(*table.shape), filled(S), filled(len(ref))
    ws = qb.keep_workspace(S, places) if ws is None else ws
    qb.qsa_evict_tokens(page, ints(budget), first, recent, weights, positions, ints(table.tolist()), ints(list(lens)),
                        ints(ref.tolist()), w_out, p_out, t_out, l_out, r_out, planes, ws)
    return w_out, p_out, t_out, l_out, r_out, ws


def check_evict(page, budget, first, recent, weights, positions, table, lens, ref, planes, result, before):
    w_out, p_out, t_out, l_out, r_out, ws = result
    w, p = weights.cpu().numpy(), positions.cpu().numpy()
    new_len, moves = [], {}
    want_w, want_p = np.zeros_like(w), np.full_like(p, -1)
    for r, n in enumerate(lens):
        shared = [ref[table[r, j // page]] > 1 for j in range(n)]
        keep, moves[r] = T.evict(w[r, :n], p[r, :n], shared, budget[r], first, recent)
        new_len.append(keep)
        want_w[r, :keep], want_p[r, :keep] = w[r, :keep], p[r, :keep]
        for to, at in moves[r]:
            want_w[r, to], want_p[r, to] = w[r, at], p[r, at]
    want_t, want_r = T.release(table, ref, lens, new_len, page)
    assert l_out.tolist() == new_len
    assert np.array_equal(t_out.cpu().numpy(), want_t) and np.array_equal(r_out.cpu().numpy(), want_r)
    assert np.array_equal(p_out.cpu().numpy(), want_p)
    assert np.array_equal(w_out.cpu().numpy().view(np.int32), want_w.view(np.int32))      # NaN and all
    for got, old in zip(planes, before):
        assert torch.equal(got, moved(old, table, moves, page))
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("lens,budget,first,recent,page,shared", [
    ([10], 4, 0, 0, 4, 0), ([10], 0, 0, 0, 4, 0), ([1, 0, 2, 30, 31, 33], 16, 2, 5, 4, 2), ([500, 20, 700], 100, 4, 32, 16, 0),
    ([500, 20, 700], 100, 4, 200, 16, 0), ([9000, 5000, 100], 1000, 16, 100, 64, 3), ([64] * 300, 60, 1, 8, 8, 0),
    ([3000], 2999, 0, 1, 1, 0), ([40000], 20000, 64, 512, 24, 0)])
@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "odd"])
def test_evict(cuda_lib, lens, budget, first, recent, page, shared, kind):
    rng = np.random.default_rng(len(lens) + page)
    table, ref = private_pool(lens, page, 2, shared=shared)
    places = table.shape[1] * page
    S = len(lens)
    w = {"spread": np.exp(2 * rng.standard_normal((S, places))), "ties": rng.integers(0, 3, (S, places)) * 0.5,
         "zeros": np.zeros((S, places)), "odd": rng.standard_normal((S, places))}[kind].astype(np.float32)
    if kind == "odd":                                     # NaN, infinities, both zeros, subnormals
        w.flat[::7], w.flat[1::11], w.flat[2::13] = np.nan, np.inf, -0.0
        w.flat[3::17], w.flat[4::19], w.flat[5::23] = 0.0, -np.inf, 1e-41
    pos = np.stack([rng.permutation(3 * places)[:places] for _ in range(S)])
    weights, positions = torch.from_numpy(w).to(DEV), ints(pos.tolist())
    planes = token_planes(len(ref), page, 3)
    before = [p.clone() for p in planes]
    budgets = [budget] * S
    if S > 2:
        budgets[1] = -1                                   # any number of tokens
    result = run_evict(page, budgets, first, recent, weights, positions, table, lens, ref, planes)
    check_evict(page, budgets, first, recent, weights, positions, table, lens, ref, planes, result, before)


def test_evict_of_a_row_of_all_the_tokens_there_can_be(cuda_lib):
    """2^31 - 2 tokens, the most that a pool has: three light ones go, the last three take their places."""
    page, n_pages = 42966, 49981
    n = page * n_pages
    assert n == 2 ** 31 - 2
    weights = torch.ones(1, n, device=DEV)
    positions = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    light = [5, 2 ** 30, 2 ** 31 - 10]
    weights[0, light] = 0.5
    w_out, p_out = torch.empty_like(weights), torch.empty_like(positions)
    table, ref = torch.arange(n_pages, dtype=torch.int32, device=DEV)[None], torch.ones(n_pages, dtype=torch.int32, device=DEV)
    t_out, l_out, r_out = filled(1, n_pages), filled(1), filled(n_pages)
    ws = qb.keep_workspace(1, n)
    qb.qsa_evict_tokens(page, ints([n - 3]), 4, 0, weights, positions, table, ints([n]), ref, w_out, p_out, t_out, l_out, r_out, [], ws)
    assert status(ws) == (0, 0) and l_out.tolist() == [n - 3]
    assert torch.equal(t_out, table) and torch.equal(r_out, ref)
    positions[0, light] = ints([n - 3, n - 2, n - 1])
    positions[0, n - 3:] = -1
    assert torch.equal(p_out, positions)
    assert bool((w_out[0, :n - 3] == 1).all()) and not bool(w_out[0, n - 3:].any())
    del weights, positions, w_out, p_out, ws              # 60 GB that later tests need not work around
    torch.cuda.empty_cache()


def test_evict_rows_out_of_range_are_left(cuda_lib):
    page, lens = 4, [30, 20, 25]
    table, ref = private_pool(lens, page, 2)
    places = table.shape[1] * page
    g = torch.Generator().manual_seed(1)
    weights, positions = torch.rand(3, places, generator=g).to(DEV), ints(np.arange(3 * places).reshape(3, -1).tolist())
    for bad in (-1, places + 1, 2 ** 31 - 1):
        planes = token_planes(len(ref), page, 3)
        before = [p.clone() for p in planes]
        w_out, p_out, t_out, l_out, r_out, ws = run_evict(page, [8] * 3, 1, 2, weights, positions, table, [30, bad, 25], ref, planes)
        assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1) and l_out.tolist() == [8, bad, 8]
        assert torch.equal(w_out[1], weights[1]) and torch.equal(p_out[1], positions[1])
        assert np.array_equal(t_out[1].cpu().numpy(), table[1])
        mine = table[1][table[1] >= 0].tolist()
        assert all(torch.equal(a[:, mine], b[:, mine]) for a, b in zip(planes, before))
        assert bool((r_out[mine] == 1).all())


def wide_pool(lens, page, seed, shared=0):
    """private_pool with room for more than 16,384 tokens a row."""
    table, ref = private_pool(lens, page, seed, shared=shared)
    wide = np.full((len(lens), max(table.shape[1], 17000 // page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    return wide, ref


@pytest.mark.parametrize("lens,budget,first,recent,page,shared", [
    ([10], 0, 0, 0, 4, 0), ([1, 0, 2, 30, 31, 33], 16, 2, 5, 4, 2), ([9000, 5000, 100], 1000, 16, 100, 64, 3),
    ([64] * 40, 60, 1, 8, 8, 0), ([17000, 40, 20000, 16384, 16385], 12000, 4, 64, 16, 2), ([4080] * 3, 4079, 4, 32, 16, 0)])
@pytest.mark.parametrize("kind", ["ties", "odd"])
def test_evict_in_wide_tables(cuda_lib, lens, budget, first, recent, page, shared, kind):
    """Rows of any length in tables with room for more tokens than one CTA holds in registers."""
    rng = np.random.default_rng(len(lens) + page)
    table, ref = wide_pool(lens, page, 2, shared)
    S, places = len(lens), table.shape[1] * page
    assert places > 16384
    w = (rng.integers(0, 3, (S, places)) * 0.5 if kind == "ties" else rng.standard_normal((S, places))).astype(np.float32)
    if kind == "odd":
        w.flat[::7], w.flat[1::11], w.flat[2::13], w.flat[4::19] = np.nan, np.inf, -0.0, -np.inf
    pos = np.stack([rng.permutation(3 * places)[:places] for _ in range(S)])
    weights, positions = torch.from_numpy(w).to(DEV), ints(pos.tolist())
    planes = token_planes(len(ref), page, 3)
    before = [p.clone() for p in planes]
    budgets = [budget] * S
    if S > 2:
        budgets[1] = -1
    result = run_evict(page, budgets, first, recent, weights, positions, table, lens, ref, planes)
    check_evict(page, budgets, first, recent, weights, positions, table, lens, ref, planes, result, before)


def test_evict_in_wide_tables_leaves_rows_out_of_range_and_bad_pages(cuda_lib):
    page, lens = 4, [30, 20, 25]
    table, ref = wide_pool(lens, page, 2)
    places = table.shape[1] * page
    weights = torch.rand(3, places, generator=torch.Generator().manual_seed(1)).to(DEV)
    positions = ints(np.arange(3 * places).reshape(3, -1).tolist())
    for bad in (-1, places + 1, 2 ** 31 - 1):
        planes = token_planes(len(ref), page, 3)
        before = [p.clone() for p in planes]
        w_out, p_out, t_out, l_out, r_out, ws = run_evict(page, [8] * 3, 1, 2, weights, positions, table, [30, bad, 25], ref, planes)
        assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1) and l_out.tolist() == [8, bad, 8]
        assert torch.equal(w_out[1], weights[1]) and torch.equal(p_out[1], positions[1])
        assert np.array_equal(t_out[1].cpu().numpy(), table[1])
        mine = table[1][table[1] >= 0].tolist()
        assert all(torch.equal(a[:, mine], b[:, mine]) for a, b in zip(planes, before)) and bool((r_out[mine] == 1).all())
    broken = table.copy()
    broken[0, 1], broken[0, 6] = -1, 2 ** 30
    weights = torch.arange(places, device=DEV, dtype=torch.float32).repeat(3, 1)
    positions = ints(np.tile(np.arange(places), (3, 1)).tolist())
    _, p_out, _, l_out, _, ws = run_evict(page, [10] * 3, 0, 0, weights, positions, broken, lens, ref, token_planes(len(ref), page, 3))
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0) and l_out.tolist() == [10] * 3
    for r, n in enumerate(lens):
        assert sorted(p_out[r, :10].tolist()) == list(range(n - 10, n))


def test_accept_moves_nothing_into_shared_pages(cuda_lib):
    """A row forked with its drafts in full pages that both rows name: what would move into them stays, in this row alone;
    a path that is in place already may be kept."""
    page, lens, off, parents = 4, [12, 12, 12], [0, 6, 12, 18], [-1, 0, 1, 0, -1, 4]
    table, ref = private_pool(lens, page, 1)
    ref[table[0, 1]] += 1
    ref[table[1, 1]] += 1
    last = [5, 1, 5]                                      # rows 0 and 2 move two tokens, row 1's first two are in place
    planes = token_planes(len(ref), page, 1)
    cut = [(12, []), T.accept(12, parents, 1), T.accept(12, parents, 5)]
    want = [moved(p, table, {r: c[1] for r, c in enumerate(cut)}, page) for p in planes]
    t_out, l_out, r_out = filled(3, table.shape[1]), filled(3), filled(len(ref))
    positions = ints(np.arange(3 * 12).reshape(3, 12).tolist())
    ws = qb.keep_workspace(3)
    qb.qsa_accept_drafts(page, ints(off), ints(parents * 3), ints(last), ints(table.tolist()), ints(lens), ints(ref.tolist()),
                         t_out, l_out, r_out, planes, ws, positions)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 0)
    want_t, want_r = T.release(table, ref, lens, [c[0] for c in cut], page)
    assert l_out.tolist() == [12, 8, 8]
    assert np.array_equal(t_out.cpu().numpy(), want_t) and np.array_equal(r_out.cpu().numpy(), want_r)
    assert positions[:2].tolist() == np.arange(24).reshape(2, 12).tolist() and positions[2, 6:8].tolist() == [34, 35]
    for got, w in zip(planes, want):
        assert torch.equal(got, w)


def test_evict_leaves_out_and_records_bad_pages(cuda_lib):
    """A page out of range: its tokens' contents do not move, and nothing outside the pool is touched."""
    page, lens = 4, [30]
    table, ref = private_pool(lens, page, 2)
    places = table.shape[1] * page
    weights = torch.arange(places, device=DEV, dtype=torch.float32)[None].contiguous()
    positions = ints([list(range(places))])
    broken = table.copy()
    broken[0, 1], broken[0, 6] = -1, 2 ** 30
    planes = token_planes(len(ref), page, 3)
    w_out, p_out, t_out, l_out, r_out, ws = run_evict(page, [10], 0, 0, weights, positions, broken, lens, ref, planes)
    assert status(ws)[0] == qb.QSA_ERR_DEVICE_BOUNDS and l_out.tolist() == [10]
    assert sorted(p_out[0, :10].tolist()) == list(range(20, 30))


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_speculative_steps_equal_plain_decoding(cuda_lib, fp8):
    """Rows that draft trees and accept a path hold, after every step, the K and V bytes of rows that appended the accepted
    tokens one by one; their attention agrees, as does the freed pages' bookkeeping."""
    Hq, Hkv, D, page, S, layers = 8, 2, 128, 8, 3, 2
    rope = qb.rope_table(D, base=1e5)
    make = dict(n_layers=layers, n_pages=60, page_size=page, n_rows=S, max_pages=12, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D,
                fp8=fp8)
    spec, plain = PagedCache(**make, max_draft=16), PagedCache(**make)
    prompt = [13, 1, 30]
    x = randn((layers, sum(prompt), Hq + 2 * Hkv, D), 1)
    seq, pos = ints(sum(([r] * n for r, n in enumerate(prompt)), [])), ints(sum((list(range(n)) for n in prompt), []))
    for cache in (spec, plain):
        cache.fork(ints([-1] * S), ints(prompt))
        for layer in range(layers):
            cache.append(layer, rope, None, x[layer, :, Hq:Hq + Hkv], x[layer, :, Hq + Hkv:], pos, seq)
    rng = np.random.default_rng(0)
    lens = list(prompt)
    for step in range(6):
        counts = [int(c) for c in rng.integers(1, 12, S)]
        if step == 3:
            counts[1] = 0
        parents = [random_parents(rng, c) for c in counts]
        last = [int(rng.integers(-1, c)) if c else -1 for c in counts]
        off = np.concatenate([[0], np.cumsum(counts)]).tolist()
        n = off[-1]
        depth = [len(line) for p in parents for line in T.lines(p)]
        seq = sum(([r] * c for r, c in enumerate(counts)), [])
        place = [lens[r] + i for r, c in enumerate(counts) for i in range(c)]
        where = [lens[r] + d - 1 for r, d in zip(seq, depth)]
        x = randn((layers, n, Hq + 2 * Hkv, D), 10 + step)
        parent = ints(sum(parents, []))
        spec.extend(ints(counts))
        outs = []
        for layer in range(layers):
            q = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV)
            spec.append(layer, rope, x[layer, :, :Hq], x[layer, :, Hq:Hq + Hkv], x[layer, :, Hq + Hkv:], ints(where), ints(seq), q,
                        place=ints(place))
            out, lse = torch.empty_like(q), torch.empty(n, Hq, device=DEV)
            spec.attend_tree(layer, q, ints(off), parent, out, lse)
            outs.append((q, out, lse))
        spec.accept(ints(off), parent, ints(last))
        # the accepted tokens one by one
        paths = [[off[r] + i for i in T.lines(p)[a]] if a >= 0 else [] for r, (p, a) in enumerate(zip(parents, last))]
        for k in range(max(map(len, paths))):
            rows = [r for r in range(S) if k < len(paths[r])]
            plain.extend(ints([int(k < len(p)) for p in paths]))
            pick = [paths[r][k] for r in rows]
            for layer in range(layers):
                y = x[layer, pick]
                q = torch.zeros(S, Hq, D, dtype=torch.bfloat16, device=DEV)
                turned = torch.empty(len(rows), Hq, D, dtype=torch.bfloat16, device=DEV)
                plain.append(layer, rope, y[:, :Hq].contiguous(), y[:, Hq:Hq + Hkv].contiguous(), y[:, Hq + Hkv:].contiguous(),
                             ints([lens[r] + k for r in rows]), ints(rows), turned)
                q[rows] = turned
                out, lse = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(S, Hq, device=DEV)
                plain.attend(layer, q, out, lse)
                tq, tout, tlse = outs[layer]
                assert torch.equal(turned, tq[pick])
                # |V| is below 5: both operators' roundings
                assert bool(((out[rows] - tout[pick]).abs().float() <= 2.0 ** -7 * out[rows].abs().float() + 2.0 ** -8 * 5).all())
                assert bool(((lse[rows] - tlse[pick]).abs() <= 1e-4).all())
        lens = [n_ + len(p) for n_, p in zip(lens, paths)]
        assert spec.seq_len.tolist() == lens == plain.seq_len.tolist()
        assert int((spec.ref > 0).sum()) == sum(-(-n_ // page) for n_ in lens) == int((plain.ref > 0).sum())
        for r in range(S):
            for a, b in zip(spec.planes, plain.planes):
                u, w = (c.table[r].cpu().numpy() for c in (spec, plain))
                s1, s2 = P.slots_of(u, lens[r], page), P.slots_of(w, lens[r], page)
                assert torch.equal(a.flatten(1, 2)[:, s1], b.flatten(1, 2)[:, s2])
    assert spec.status() == ((0, 0), (0, 0)) and spec.more_status() == ((0, 0), (0, 0))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_loop_under_a_budget(cuda_lib, fp8):
    """Decoding with eviction every few steps, beams forked in between: rows hold the bytes and positions that a host model
    of the policy says, and the attention is that over exactly those tokens."""
    Hq, Hkv, D, page, S = 8, 2, 128, 4, 4
    rope = qb.rope_table(D, base=1e5)
    cache = PagedCache(1, 80, page, S, 20, Hq, Hkv, D, fp8=fp8, evictable=True, max_draft=4)
    n0 = 30
    x = randn((S, n0, Hq + 2 * Hkv, D), 1)
    cache.fork(ints([-1] * S), ints([n0] * S))
    flat = x.flatten(0, 1)
    cache.append(0, rope, None, flat[:, Hq:Hq + Hkv], flat[:, Hq + Hkv:], ints(list(range(n0)) * S),
                 ints(sum(([r] * n0 for r in range(S)), [])), place=ints(list(range(n0)) * S))
    where = [n0] * S                                      # the next position of each row
    rows = [list(range(n0)) for _ in range(S)]            # positions at each place
    weights = [np.zeros(n0) for _ in range(S)]
    rng = np.random.default_rng(1)
    for step in range(12):
        cache.extend()
        y = randn((S, Hq + 2 * Hkv, D), 50 + step)
        q = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV)
        cache.append(0, rope, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], ints(where), None, q, place=ints([len(r) for r in rows]))
        out, lse = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(S, Hq, device=DEV)
        cache.attend(0, q, out, lse, weigh=True)
        table = cache.table.cpu().numpy()
        for r in range(S):
            rows[r].append(where[r])
            weights[r] = np.append(weights[r], 0.0)
            where[r] += 1
        if fp8:
            values = [f64(c.view(torch.float8_e4m3fn).float())[0] * np.repeat(f64(s)[0], 128, -1)
                      for c, s in (cache.planes[:2], cache.planes[2:])]
        else:
            values = [f64(p)[0] for p in cache.planes]
        check_decode(out, lse, q, values, table, [len(r) for r in rows], page, 0, D ** -0.5, fp8)
        got = cache.weights.cpu().numpy()
        for r in range(S):
            K = values[0].reshape(-1, Hkv, D)[P.slots_of(table[r], len(rows[r]), page)]
            weights[r] += T.token_weights(f64(q[r]), K, 0, D ** -0.5)
            assert np.allclose(got[r, :len(rows[r])], weights[r], rtol=1e-4, atol=0) and not got[r, len(rows[r]):].any()
            assert cache.positions[r, :len(rows[r])].tolist() == rows[r]
        if step % 3 == 2:
            shared = [[bool(v) for v in (cache.ref[cache.table[r].long().clamp(min=0)] > 1).repeat_interleave(page)[:len(rows[r])]]
                      for r in range(S)]
            held = cache.weights.cpu().numpy()
            cache.evict(ints([24] * S), 2, 6)
            for r in range(S):
                keep, moves = T.evict(held[r, :len(rows[r])], rows[r], shared[r], 24, 2, 6)
                for to, at in moves:
                    rows[r][to], weights[r][to] = rows[r][at], weights[r][at]
                rows[r], weights[r] = rows[r][:keep], weights[r][:keep]
            assert cache.seq_len.tolist() == [len(r) for r in rows]
            assert [cache.positions[r, :len(rows[r])].tolist() for r in range(S)] == rows
        if step in (4, 7):                                # a beam step: two rows continue row 1
            parent = [1, 1, 2, 3] if step == 4 else [0, 3, 2, 3]
            cache.fork(ints(parent), ints([0] * S))
            rows, weights = [list(rows[p]) for p in parent], [weights[p].copy() for p in parent]
            where = [where[p] for p in parent]
            cache.compact()
    assert cache.status() == ((0, 0), (0, 0)) and cache.more_status() == ((0, 0),) * 3


@pytest.mark.parametrize("fp8", [False, True])
def test_drafting_under_a_budget(cuda_lib, fp8):
    """Drafts that are weighed while they are in their rows, then accepted or not, then cut by weight: what each token has
    received stays with it, and a token at a dropped one's place starts with nothing."""
    Hq, Hkv, D, page, S = 8, 2, 128, 4, 3
    rope = qb.rope_table(D, base=1e5)
    cache = PagedCache(1, 60, page, S, 20, Hq, Hkv, D, fp8=fp8, evictable=True, max_draft=8)
    n0 = 26
    x = randn((S * n0, 2 * Hkv, D), 1)
    cache.fork(ints([-1] * S), ints([n0] * S))
    cache.append(0, rope, None, x[:, :Hkv], x[:, Hkv:], ints(list(range(n0)) * S), ints(sum(([r] * n0 for r in range(S)), [])))
    rows, weights, newest = [list(range(n0)) for _ in range(S)], [np.zeros(n0) for _ in range(S)], [n0] * S
    parents, lasts = [-1, 0, 0, 2, 1, 3], [5, -1, 3]
    off, depth = [0, 6, 12, 18], [len(line) - 1 for line in T.lines(parents)]
    for step in range(6):
        cache.extend(ints([6] * S))
        y = randn((S * 6, Hq + 2 * Hkv, D), 20 + step)
        where = [newest[r] + d for r in range(S) for d in depth]
        place = [len(rows[r]) + i for r in range(S) for i in range(6)]
        q = torch.empty(S * 6, Hq, D, dtype=torch.bfloat16, device=DEV)
        cache.append(0, rope, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], ints(where), ints(sum(([r] * 6 for r in range(S)), [])),
                     q, place=ints(place))
        before = cache.weights.cpu().numpy()
        for r in range(S):
            rows[r] += where[6 * r:6 * r + 6]
            assert not before[r, len(weights[r]):].any()
            weights[r] = np.append(weights[r], np.zeros(6))
        out = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV)
        cache.attend(0, q[5::6], out, weigh=True)         # the newest token's queries, over drafts and all
        held = cache.weights.cpu().numpy()
        for r in range(S):
            weights[r] = held[r, :len(rows[r])].copy()
            assert (weights[r][-6:] > 0).all()
        cache.accept(ints(off), ints(parents * S), ints(lasts))
        for r in range(S):
            n, moves = T.accept(len(rows[r]), parents, lasts[r])
            newest[r] += n - (len(rows[r]) - 6)
            old_p, old_w = list(rows[r]), weights[r].copy()
            for to, at in moves:
                rows[r][to], weights[r][to] = old_p[at], old_w[at]
            rows[r], weights[r] = rows[r][:n], weights[r][:n]
        check = cache.weights.cpu().numpy(), cache.positions.cpu().numpy()
        for r in range(S):
            n = len(rows[r])
            assert np.array_equal(check[0][r, :n], weights[r].astype(np.float32)) and not check[0][r, n:].any()
            assert check[1][r, :n].tolist() == rows[r] and (check[1][r, n:] == -1).all()
        if step % 2:
            cache.evict(ints([24] * S), 2, 4)
            for r in range(S):
                keep, moves = T.evict(weights[r], rows[r], [False] * len(rows[r]), 24, 2, 4)
                for to, at in moves:
                    rows[r][to], weights[r][to] = rows[r][at], weights[r][at]
                rows[r], weights[r] = rows[r][:keep], weights[r][:keep]
            assert [cache.positions[r, :len(rows[r])].tolist() for r in range(S)] == rows
    assert cache.status() == ((0, 0), (0, 0)) and cache.more_status() == ((0, 0),) * 3


@pytest.mark.parametrize("fp8", [False, True])
def test_beams_over_a_shared_prompt_are_all_weighed(cuda_lib, fp8):
    """Rows that share a prompt attend more tokens together than the pool holds: each step adds Hq to every row's weights (each
    weight off by less than 2^-17, n sums of it in fp32)."""
    Hq, Hkv, D, page, S, n = 8, 2, 128, 16, 12, 800
    cache = PagedCache(1, n // page + S, page, S, n // page + 2, Hq, Hkv, D, fp8=fp8, evictable=True)
    rope = qb.rope_table(D)
    x = randn((n, 2 * Hkv, D), 1)
    cache.fork(ints([-1] * S), ints([n] + [0] * (S - 1)))
    cache.append(0, rope, None, x[:, :Hkv], x[:, Hkv:], ints(list(range(n))), ints([0] * n))
    cache.fork(ints([0] * S), ints([0] * S))
    for step in range(2):
        cache.extend()
        y = randn((S, Hq + 2 * Hkv, D), 5 + step)
        q = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV)
        cache.append(0, rope, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], ints([n + step] * S), None, q)
        cache.attend(0, q, torch.empty_like(q), weigh=True)
        assert cache.status() == ((0, 0), (0, 0)) and cache.more_status() == ((0, 0), (0, 0))
        assert np.allclose(f64(cache.weights).sum(1), Hq * (step + 1), rtol=2.0 ** -17 + 2 * 2.0 ** -24, atol=0)
        assert bool((cache.weights[:, :n + step + 1] > 0).all()) and not bool(cache.weights[:, n + step + 1:].any())


def test_an_evictable_cache_keeps_its_own_records(cuda_lib):
    """Tokens appended by position alone have their positions recorded; rows that a fork empties have received nothing."""
    Hq, Hkv, D, page, S = 4, 1, 64, 4, 2
    rope = qb.rope_table(D)
    cache = PagedCache(2, 6, page, S, 6, Hq, Hkv, D, evictable=True)
    cache.fork(ints([-1] * S), ints([6, 5]))
    x = randn((11, 2 * Hkv, D), 1)
    seq, pos = ints([0] * 6 + [1] * 5), ints(list(range(6)) + list(range(5)))
    for layer in range(2):
        cache.append(layer, rope, None, x[:, :Hkv], x[:, Hkv:], pos, seq)
    assert cache.positions[0, :6].tolist() == list(range(6)) and cache.positions[1, :5].tolist() == list(range(5))
    q = randn((S, Hq, D), 2)
    cache.attend(0, q, torch.empty_like(q), weigh=True)
    assert bool((cache.weights[0, :6] > 0).all()) and bool((cache.weights[1, :5] > 0).all())
    cache.evict(ints([3, -1]), 0, 1)
    assert cache.seq_len.tolist() == [3, 5] and cache.positions[0, :3].max() == 5
    assert cache.status() == ((0, 0), (0, 0)) and cache.more_status() == ((0, 0), (0, 0))
    cache.fork(ints([0, 1]), ints([0, 100]))              # row 1 is out of pages, and empty
    assert cache.status()[1] == (qb.QSA_ERR_DEVICE_BOUNDS, 1) and cache.seq_len.tolist() == [3, 0]
    assert not cache.weights[1].any() and bool((cache.positions[1] == -1).all()) and bool((cache.weights[0, :3] > 0).all())


def test_captured_speculative_steps_replay(cuda_lib):
    """Two steps (drafts, attention, acceptance) in one graph, replayed: the lengths grow by the accepted tokens each time."""
    Hq, Hkv, D, page, S = 8, 2, 128, 8, 2
    rope = qb.rope_table(D)
    cache = PagedCache(1, 64, page, S, 24, Hq, Hkv, D, max_draft=4)
    cache.fork(ints([-1] * S), ints([5, 9]))
    x = randn((8, Hq + 2 * Hkv, D), 3)
    off, parent, last, count = ints([0, 4, 8]), ints([-1, 0, 0, 2, -1, 0, 1, -1]), ints([3, 2]), ints([4, 4])
    step, depth, seq = ints([0, 1, 2, 3] * 2), ints([0, 1, 1, 2, 0, 1, 2, 0]), ints([0] * 4 + [1] * 4)
    q = torch.empty(8, Hq, D, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(8, Hq, device=DEV)

    def steps():
        for _ in range(2):
            base = cache.seq_len[seq.long()]
            cache.extend(count)
            cache.append(0, rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], base + depth, seq, q, place=base + step)
            cache.attend_tree(0, q, off, parent, out, lse)
            cache.accept(off, parent, last)

    steps()                                               # before the capture
    cache.extend(ints([0, 0]))                            # and an even number of changes again
    cache.extend(ints([0, 0]))
    assert cache.seq_len.tolist() == [11, 15]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        steps()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert cache.seq_len.tolist() == [17 + 6 * i, 21 + 6 * i]
    assert int((cache.ref > 0).sum()) == 4 + 5 and cache.status() == ((0, 0), (0, 0)) and cache.more_status() == ((0, 0),) * 2


# ------------------------------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("Hq,Hkv,D,fp8", [(16, 2, 256, False), (8, 2, 128, False), (4, 1, 64, False), (16, 2, 256, True), (8, 2, 128, True)])
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_tree_odd_values_of_a_draft_reach_its_family_alone(cuda_lib, Hq, Hkv, D, fp8, page, value):
    """K and V of one drafted token that are not finite: the tokens that attend it get what their sums give (the value in its
    dim, or NaN), its other relatives and siblings stay as they were."""
    lens, counts = [150, 40, 9], [12, 7, 9]
    q, planes, values, tab, table, off, _ = tree_inputs(lens, counts, Hq, Hkv, D, page, fp8, seed=4, spare_rows=0)
    parents = [[-1, 0, 0, 1, 1, 2, 2, -1, 7, 8, 3, 3], [-1, 0, 1, -1, 3, 4, 5], [-1, 0, 0, 0, 1, 2, 3, -1, -1]]
    cfg = qb.make_paged_config(Hq, Hkv, D, page)
    ws = qb.tree_workspace(cfg, 12)
    good, good_lse = run_tree(cfg, q, planes, tab, lens, off, parents, 12, ws)
    odd = 2                                               # the third draft of each row, dim 5 of KV head 0
    for r, n in enumerate(lens):
        slot = int(P.slots_of(table[r], n, page)[n - counts[r] + odd])
        if fp8:
            planes[2].flatten(0, 1)[slot, 0, 5] = 0x7F    # E4M3 has no infinity
        else:
            planes[1].flatten(0, 1)[slot, 0, 5] = value
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 12, ws)
    assert status(ws) == (0, 0) and torch.equal(lse, good_lse)
    G = Hq // Hkv
    want = good.clone()
    for r in range(3):
        for i, line in enumerate(T.lines(parents[r])):
            if odd in line:
                want[off[r] + i, :G, 5] = float("nan") if fp8 else value
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out, 0.0), torch.nan_to_num(want, 0.0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [32, 3])
def test_tree_odd_values_at_the_windows_edge(cuda_lib, fp8, page):
    """Tokens that some drafts see and others, deeper ones, do not: what is not finite in them reaches those that do."""
    Hq, Hkv, D, n, window = 8, 2, 128, 300, 90
    parents = [[-1, 0, 1, 2, 3, -1]]
    q, planes, values, tab, table, off, _ = tree_inputs([n], [6], Hq, Hkv, D, page, fp8, seed=4, spare_rows=0)
    cfg = qb.make_paged_config(Hq, Hkv, D, page, window=window)
    ws = qb.tree_workspace(cfg, 6)
    good, _ = run_tree(cfg, q, planes, tab, [n], off, parents, 6, ws)
    place = n - 6 + 1 - window + 2                        # positions above own - window: seen at depths 1, 2 and 3
    slot = int(P.slots_of(table[0], n, page)[place])
    gone = int(P.slots_of(table[0], n, page)[place - 4])  # seen by none
    if fp8:
        planes[2].flatten(0, 1)[slot, 1, 3] = 0xFF
        planes[3].flatten(0, 1)[gone] = float("nan")
    else:
        planes[1].flatten(0, 1)[slot, 1, 3] = float("nan")
        planes[1].flatten(0, 1)[gone] = float("inf")
    out, _ = run_tree(cfg, q, planes, tab, [n], off, parents, 6, ws)
    seen = [place in places for places in T.attended(n, parents[0], window)]
    assert seen == [True, True, True, False, False, True]
    for i in range(6):
        spoiled = torch.isnan(out[i])
        assert bool(spoiled[4:, 3].all()) == seen[i] and int(spoiled.sum()) == (4 if seen[i] else 0)
        assert torch.equal(out[i][~spoiled], good[i][~spoiled])


@pytest.mark.parametrize("Hq,D", [(8, 256), (8, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["history", "draft"])
def test_tree_value_scale_that_is_not_finite(cuda_lib, Hq, D, value, where):
    """An infinite or undefined V scale makes NaN of its 128 dims for the tokens that attend it, and of nothing else."""
    page, n, counts = 16, 500, [8]
    q, planes, values, tab, table, off, parents = tree_inputs([n], counts, Hq, 1, D, page, True, seed=4, spare_rows=0, chain=0.3)
    cfg = qb.make_paged_config(Hq, 1, D, page)
    ws = qb.tree_workspace(cfg, 8)
    good, good_lse = run_tree(cfg, q, planes, tab, [n], off, parents, 8, ws)
    at = 100 if where == "history" else n - 8 + 1
    planes[3].flatten(0, 1)[int(P.slots_of(table[0], n, page)[at]), 0, -1] = value
    out, lse = run_tree(cfg, q, planes, tab, [n], off, parents, 8, ws)
    assert torch.equal(lse, good_lse)
    for i, places in enumerate(T.attended(n, parents[0])):
        if at in places:
            assert bool(torch.isnan(out[i, :, -128:]).all())
            assert torch.equal(out[i, :, :-128], good[i, :, :-128])
        else:
            assert torch.equal(out[i], good[i])


@pytest.mark.parametrize("D", [256, 128])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("n,window,place", [
    (20, 0, 3), (20, 0, 11), (500, 0, 491), (500, 0, 448), (500, 0, 447), (500, 0, 492), (500, 0, 499),
    # the drafts' positions reach 8 deep: places below 492 + 8 - 90 = 410 are not for all of them, those below 403 for none
    (500, 90, 402), (500, 90, 403), (500, 90, 409), (500, 90, 410), (500, 90, 447), (500, 90, 448)])
def test_tree_value_scale_that_is_not_finite_in_a_masked_tile(cuda_lib, D, value, n, window, place):
    """Such a scale in a tile that holds drafts, or the window's edge: of a token that all, some or none of the drafts attend."""
    Hq, page, T_ = 8, 16, 8
    q, planes, values, tab, table, off, _ = tree_inputs([n], [T_], Hq, 1, D, page, True, seed=4, spare_rows=0)
    for parents in ([list(range(-1, 7))], [[-1, 0, 0, 1, 2, 2, -1, 6]]):
        cfg = qb.make_paged_config(Hq, 1, D, page, window=window)
        ws = qb.tree_workspace(cfg, T_)
        good, good_lse = run_tree(cfg, q, planes, tab, [n], off, parents, T_, ws)
        spoiled = [p.clone() for p in planes]
        spoiled[3].flatten(0, 1)[int(P.slots_of(table[0], n, page)[place]), 0, -1] = value
        out, lse = run_tree(cfg, q, spoiled, tab, [n], off, parents, T_, ws)
        assert torch.equal(lse, good_lse) and status(ws) == (0, 0)
        for i, places in enumerate(T.attended(n, parents[0], window)):
            odd = torch.isnan(out[i])
            assert bool(odd[:, -128:].all()) if place in places else not bool(odd.any()), i
            assert torch.equal(out[i][~odd], good[i][~odd])


@pytest.mark.parametrize("D", [256, 128])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("n,place", [(20, 0), (20, 18), (20, 19), (300, 256), (300, 298), (300, 255)])
def test_one_token_meets_value_scales_as_the_decode_does(cuda_lib, D, value, n, place):
    q, planes, values, tab, table, off, parents = tree_inputs([n], [1], 8, 1, D, 16, True, seed=4, spare_rows=0)
    planes[3].flatten(0, 1)[int(P.slots_of(table[0], n, 16)[place]), 0, 0] = value
    cfg = qb.make_paged_config(8, 1, D, 16)
    out, _ = run_tree(cfg, q, planes, tab, [n], off, parents, 1, qb.tree_workspace(cfg, 1))
    want, _ = run_decode(cfg, q, planes, tab, ints([n]), qb.paged_workspace(cfg))
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and bool(torch.isnan(out[..., :128]).all())


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq,D,fp8", [(8, 256, True), (8, 128, True), (8, 256, False), (4, 64, False)])
def test_tree_query_that_is_not_finite_spoils_its_head_alone(cuda_lib, Hq, D, fp8, value):
    lens, counts = [300, 70], [5, 3]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, 1, D, 16, fp8, seed=4, spare_rows=0)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.tree_workspace(cfg, 5)
    good, good_lse = run_tree(cfg, q, planes, tab, lens, off, parents, 5, ws)
    q[6, 1, 7] = value
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 5, ws)
    assert bool(torch.isnan(out[6, 1]).all())
    out[6, 1], lse[6, 1] = good[6, 1], good_lse[6, 1]
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_tree_odd_keys_of_masked_tokens_change_nothing(cuda_lib, value):
    lens, counts = [90], [6]
    q, planes, values, tab, table, off, _ = tree_inputs(lens, counts, 8, 2, 128, 8, False, seed=4, spare_rows=0)
    parents = [[-1, 0, 1, -1, 3, 4]]
    cfg = qb.make_paged_config(8, 2, 128, 8)
    ws = qb.tree_workspace(cfg, 6)
    good, _ = run_tree(cfg, q, planes, tab, lens, off, parents, 6, ws)
    planes[0].flatten(0, 1)[int(P.slots_of(table[0], 90, 8)[84 + 1])] = value         # draft 1: seen by 1 and 2
    out, _ = run_tree(cfg, q, planes, tab, lens, off, parents, 6, ws)
    assert torch.equal(out[[0, 3, 4, 5]], good[[0, 3, 4, 5]])


@pytest.mark.parametrize("D", [256, 128])
@pytest.mark.parametrize("page", [8, 3])
@pytest.mark.parametrize("what", ["code", "inf", "nan"])
def test_tree_odd_keys_of_masked_tokens_change_nothing_over_fp8_rows(cuda_lib, D, page, what):
    """A draft's K code or K scale that is not finite, and those of tokens that lie before every window or behind the row's end."""
    n, T_, Hq, window = 200, 6, 8, 70
    q, planes, values, tab, table, off, _ = tree_inputs([n], [T_], Hq, 1, D, page, True, seed=4, spare_rows=0)
    parents = [[-1, 0, 1, -1, 3, 4]]
    cfg = qb.make_paged_config(Hq, 1, D, page, window=window)
    ws = qb.tree_workspace(cfg, T_)
    good, good_lse = run_tree(cfg, q, planes, tab, [n], off, parents, T_, ws)
    slots = P.slots_of(table[0], n, page)
    places = [n - T_ + 1, n - T_ - window, 3] + [n] * (n % page != 0)
    for place in places:
        slot = int(slots[place]) if place < n else int(slots[n - 1]) + 1
        if what == "code":
            planes[0].flatten(0, 1)[slot, 0, D - 1] = 0x7F
        else:
            planes[1].flatten(0, 1)[slot, 0, 0] = float(what)
    out, lse = run_tree(cfg, q, planes, tab, [n], off, parents, T_, ws)
    seen = [bool(set(places) & set(at)) for at in T.attended(n, parents[0], window)]
    assert seen == [False, True, True, False, False, False] and status(ws) == (0, 0)
    for i in range(T_):
        if seen[i]:
            assert bool(torch.isnan(out[i]).any())
        else:
            assert torch.equal(out[i], good[i]) and torch.equal(lse[i], good_lse[i])


@pytest.mark.parametrize("Hq,D,fp8", [(8, 256, True), (8, 128, True), (8, 256, False), (4, 64, False)])
@pytest.mark.parametrize("scale", [0.0, 1e-9, 1e-38])
def test_tree_queries_of_zeros_take_the_mean(cuda_lib, Hq, D, fp8, scale):
    """Every score is zero, whatever the scale: masked tokens stay masked beside them."""
    lens, counts = [150, 70], [5, 3]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, 1, D, 16, fp8, seed=4)
    q[:, 1].zero_()
    q[3].zero_()
    cfg = qb.make_paged_config(Hq, 1, D, 16, softmax_scale=scale)
    ws = qb.tree_workspace(cfg, 5)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, 5, ws)
    check_tree(out, lse, q, values, table, lens, off, parents, 16, float(np.float32(scale)) or D ** -0.5, 0, fp8)


# ------------------------------------------------------------------------------------------ limits
@pytest.mark.parametrize("Hq,Hkv,D,drafts", [(160, 160, 64, 3), (16, 1, 256, 128), (64, 4, 128, 100), (620, 310, 64, 2)])
def test_tree_of_many_heads_and_drafts(cuda_lib, Hq, Hkv, D, drafts):
    """More CTAs than one wave, and sixteen tiles of query rows."""
    lens = [drafts + 300, drafts + 1, 64]
    counts = [drafts, drafts, min(drafts, 64)]
    q, planes, values, tab, table, off, parents = tree_inputs(lens, counts, Hq, Hkv, D, 16, False, seed=3)
    cfg = qb.make_paged_config(Hq, Hkv, D, 16)
    ws = qb.tree_workspace(cfg, drafts)
    out, lse = run_tree(cfg, q, planes, tab, lens, off, parents, drafts, ws)
    assert status(ws) == (0, 0)
    pick = [0, drafts // 2, drafts - 1]                   # a few tokens of each row against the oracle
    for r in range(3):
        keep = [i for i in pick if i < counts[r]]
        slots = P.slots_of(table[r], lens[r], 16)
        K, V = (x.reshape(-1, *x.shape[2:])[slots] for x in values)
        for i in keep:
            at = T.attended(lens[r], parents[r])[i]
            want, want_lse, mass, terms = P.decode(f64(q[off[r] + i]), K[at], V[at], 0, D ** -0.5)
            ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1)
            sums = len(at) / 8 * 2.0 ** -24 + 2.0 ** -15
            tol = 2.0 ** -8 * np.abs(want) + (2 * ds[:, None] + sums + 2.0 ** -8) * mass
            assert np.all(np.abs(f64(out[off[r] + i]) - want) <= tol)
            assert np.all(np.abs(f64(lse[off[r] + i]) - want_lse) <= ds + sums + 2.0 ** -22 * np.abs(want_lse))
    assert bool((out[off[-1]:] == 8).all())


@pytest.mark.parametrize("Hq,D", [(8, 256), (8, 128)])
@pytest.mark.parametrize("spread", [4, 16])
def test_tree_queries_and_scales_of_a_wide_range_over_fp8_rows(cuda_lib, Hq, D, spread):
    """Queries whose values span 2^spread within a head: what lies below 2^-10 of a head's largest value is off by at most 2^-17
    of that. V scales that span 2^spread over the tokens: each weight times its scale is off by 2^-11 of it and 2^-31 of
    the largest weight (2^8 of the lazy maximum's) times the largest scale."""
    n, count, page = 700, 9, 16
    q, planes, values, tab, table, off, parents = tree_inputs([n], [count], Hq, 1, D, page, True, seed=2, spare_rows=0)
    g = torch.Generator().manual_seed(5)
    q *= torch.exp2(-spread * torch.rand(q.shape, generator=g)).to(DEV)
    factor = torch.exp2(-spread * torch.rand(planes[3].shape, generator=g)).to(DEV)
    planes[3].mul_(factor)
    values = (values[0], values[1] * np.repeat(f64(factor), 128, -1))
    cfg = qb.make_paged_config(Hq, 1, D, page)
    ws = qb.tree_workspace(cfg, count)
    out, lse = run_tree(cfg, q, planes, tab, [n], off, parents, count, ws)
    slots = P.slots_of(table[0], n, page)
    K, V = (x.reshape(-1, *x.shape[2:])[slots] for x in values)
    for i, at in enumerate(T.attended(n, parents[0])):
        qi = f64(q[i])
        want, want_lse, mass, terms = P.decode(qi, K[at], V[at], 0, D ** -0.5)
        ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1) + 2.0 ** -17 * np.abs(qi).max(1) * np.abs(K[at]).sum(2).max() * D ** -0.5
        sums = len(at) / 8 * 2.0 ** -24 + 2.0 ** -15
        tol = 2.0 ** -8 * np.abs(want) + (2 * ds[:, None] + sums + 2.0 ** -11) * mass + len(at) * 2.0 ** -31 * 2.0 ** 8 * np.abs(V[at]).max()
        assert np.all(np.abs(f64(out[i]) - want) <= tol)
        assert np.all(np.abs(f64(lse[i]) - want_lse) <= ds + sums + 2.0 ** -22 * np.abs(want_lse))
