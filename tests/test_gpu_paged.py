"""The paged-cache operators on the GPU against a plain 64-bit implementation: rotary positions, appending
(bf16 and FP8 rows), attention of one new token over a page table, forking, compacting and copying pages,
and a run of them together.

Tolerances. A result rounded once to bf16 is off by at most half a step, 2^-8 of its value. Before that:
- a turned value u cos - w sin: the angle is a 32-bit fraction of a turn (2 pi 2^-32) converted to fp32 (at
  most pi 2^-24 off), sin and cos within 2^-22, two products and a sum rounded to fp32: below
  (|u| + |w|) x 2^-20;
- a score: D products summed in fp32 in any order, off by at most D 2^-24 times the sum of their
  magnitudes (`terms`), and 2^-21 of itself for the scale, the FP8 scale and the exponential's argument. A weight
  is then off by twice that relative to the others (its own and the maximum's), plus 2^-15 for the
  exponential and the second product's operands, plus the fp32 sums over n tokens, taken 8 at a time:
  n 2^-27 ... n 2^-24 / 8; all of it relative to the weighted mean of |V| (`mass`);
- over FP8 rows a weight (times V's scale, relative to the largest) is rounded once to f16: half a step of its 11
  bits is 2^-11 of it, and 2^-25 of the largest below f16's normal range. The largest weight times its row's
  largest |V| is at most the largest of `mass` over the dims, so n tokens add at most n 2^-25 of that."""

import numpy as np
import pytest
import torch

from indexer_driven_sparse_gb300 import binding as qb
from indexer_driven_sparse_gb300.pipeline import DecodeBatch, PagedCache
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def status(ws):
    return qb.qsa_read_device_status(ws)


# ------------------------------------------------------------------------------------------ rotary positions
SCALINGS = {"none": {}, "linear": dict(factor=8.0), "ntk": dict(factor=4.0),
            "by_parts": dict(factor=16.0, original_len=8192)}


def rope_want(x, pos, dim, rot, begin, inter, base, scaling):
    freq, amp = P.rope_frequencies(rot, base, scaling, **SCALINGS[scaling])
    want = P.rope(f64(x), pos, freq, amp, begin, inter)
    mag = np.abs(f64(x))
    pair = mag.copy()                                     # |u| + |w| of each turned dim
    half = rot // 2
    a = begin + (2 * np.arange(half) if inter else np.arange(half))
    b = a + (1 if inter else half)
    pair[..., a] = pair[..., b] = mag[..., a] + mag[..., b]
    return want, amp * pair * 2.0 ** -20


def check_rope(got, want, slack):
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack), np.abs(got - want).max()


@pytest.mark.parametrize("dim,rot,begin,inter,scaling", [
    (256, 256, 0, False, "none"), (256, 64, 0, False, "by_parts"), (128, 128, 0, True, "linear"),
    (128, 96, 16, False, "ntk"), (576, 64, 512, True, "none"), (64, 32, 8, True, "by_parts"), (16, 16, 0, False, "none"),
    (48, 0, 0, False, "none")])
@pytest.mark.parametrize("n,heads", [(1, 1), (5, 7), (301, 16)])
def test_rope(cuda_lib, dim, rot, begin, inter, scaling, n, heads):
    x = randn((n, heads, dim), seed=n + dim)
    pos = np.random.default_rng(n).integers(0, 3_145_728, n)
    pos[0] = 3_145_727
    if n > 3:
        pos[1], pos[2], pos[3] = 0, -5000, 2 ** 31 - 1
    rope = qb.rope_table(dim, rot, begin, inter, base=5e5, scaling=scaling, **SCALINGS[scaling])
    out = torch.full_like(x, 7.0)
    qb.qsa_rope(rope, x, ints(pos.tolist()), out)
    want, slack = rope_want(x, pos, dim, rot, begin, inter, 5e5, scaling)
    check_rope(f64(out), want, slack)
    # in place, the same bits
    qb.qsa_rope(rope, x, ints(pos.tolist()), x)
    assert torch.equal(x, out)


def test_rope_strided_rows_and_untouched_neighbours(cuda_lib):
    fused = randn((33, 5, 128), seed=1)                   # q: 3 heads, k: 1, v: 1 of one projection
    before = fused.clone()
    rope = qb.rope_table(128)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    q = fused[:, :3]
    want = torch.empty(33, 3, 128, dtype=torch.bfloat16, device=DEV)
    qb.qsa_rope(rope, q, pos, want)
    qb.qsa_rope(rope, q, pos, q)
    assert torch.equal(fused[:, :3], want) and torch.equal(fused[:, 3:], before[:, 3:])
    wide = torch.full((33, 9, 128), -3.0, dtype=torch.bfloat16, device=DEV)
    qb.qsa_rope(rope, before[:, :3], pos, wide[:, 4:7])
    assert torch.equal(wide[:, 4:7], want) and bool((wide[:, :4] == -3).all()) and bool((wide[:, 7:] == -3).all())


def test_rope_is_undone_by_negative_positions(cuda_lib):
    # two roundings to bf16: 2^-8 of the turned value (at most |u| + |w|) and 2^-8 of the result
    x = randn((64, 4, 256), seed=2)
    pos = torch.randint(0, 3_000_000, (64,), dtype=torch.int32, device=DEV)
    rope = qb.rope_table(256, base=1e6)
    y = torch.empty_like(x)
    qb.qsa_rope(rope, x, pos, y)
    qb.qsa_rope(rope, y, -pos, y)
    a, b = f64(x), f64(y)
    pair = np.abs(a[..., :128]) + np.abs(a[..., 128:])
    assert np.all(np.abs(a - b) <= 2.0 ** -8 * (2.0 * np.concatenate([pair, pair], -1) + np.abs(a)) + 1e-5)


# ------------------------------------------------------------------------------------------ appending
def quantise64(x):
    """fp32 scales of x [..., D] per 128 dims (from 64-bit values)."""
    g = np.abs(x.reshape(*x.shape[:-1], -1, 128)).max(-1)
    return g / 448.0


def e4m3(t):
    return f64(t.view(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("dim,q_heads,kv_heads,rot,inter,page,fp8", [
    (256, 16, 2, 256, False, 64, False), (128, 7, 1, 64, True, 24, False), (64, 8, 8, 64, False, 1, False),
    (256, 16, 2, 128, True, 16, True), (128, 8, 8, 128, False, 5, True), (128, 4, 2, 0, False, 4, True)])
@pytest.mark.parametrize("n", [1, 37, 700])
def test_append(cuda_lib, dim, q_heads, kv_heads, rot, inter, page, fp8, n):
    rows = 9
    room = n // page + 3
    n_pages = rows * room + 2
    rng = np.random.default_rng(n + dim)
    table = rng.permutation(n_pages)[:rows * room].reshape(rows, room)
    # distinct (row, position) pairs; some tokens are padding
    flat = rng.permutation(rows * room * page)[:n]
    seq, pos = flat // (room * page), flat % (room * page)
    seq = np.where(rng.random(n) < 0.2, -1, seq) if n > 1 else seq
    cfg = qb.make_paged_config(q_heads, kv_heads, dim, page)
    ws = qb.paged_workspace(cfg)
    rope = qb.rope_table(dim, rot, 0, inter, base=1e6)
    fused = randn((n, q_heads + 2 * kv_heads, dim), seed=n)
    q, k, v = fused[:, :q_heads], fused[:, q_heads:q_heads + kv_heads], fused[:, q_heads + kv_heads:]
    q_out = torch.full((n, q_heads, dim), 9.0, dtype=torch.bfloat16, device=DEV)
    shape = (n_pages, page, kv_heads, dim)
    freq, amp = P.rope_frequencies(rot, 1e6) if rot else (np.zeros(0), 1.0)
    args = (cfg, rope, q, k, v, ints(pos.tolist()), ints(seq.tolist()), q_out)
    live = seq >= 0
    slot = table[np.maximum(seq, 0), pos // page] * page + pos % page
    want_q, slack_q = rope_want(q, pos, dim, rot, 0, inter, 1e6, "none") if rot else (f64(q), 0 * f64(q))
    want_k, slack_k = rope_want(k, pos, dim, rot, 0, inter, 1e6, "none") if rot else (f64(k), 0 * f64(k))
    tab = ints(table.tolist())
    if not fp8:
        kc, vc = torch.full(shape, 5.0, dtype=torch.bfloat16, device=DEV), torch.full(shape, 6.0, dtype=torch.bfloat16,
                                                                                      device=DEV)
        qb.qsa_rope_append(*args, kc, vc, tab, ws)
        kf, vf = kc.flatten(0, 1), vc.flatten(0, 1)
        check_rope(f64(kf)[slot[live]], want_k[live], slack_k[live])
        assert torch.equal(vf[slot[live]], v[torch.from_numpy(live).to(DEV)])
        rest = np.setdiff1d(np.arange(n_pages * page), slot[live])
        assert bool((kf[rest] == 5).all()) and bool((vf[rest] == 6).all())
    else:
        codes = dict(dtype=torch.uint8, device=DEV)
        kv8 = [torch.full(shape, 17, **codes), torch.full(shape[:3] + (dim // 128,), 2.0, device=DEV),
               torch.full(shape, 18, **codes), torch.full(shape[:3] + (dim // 128,), 3.0, device=DEV)]
        qb.qsa_rope_append_fp8kv(*args, kv8, tab, ws)
        rest = np.setdiff1d(np.arange(n_pages * page), slot[live])
        for plane, fill in zip(kv8, (17, 2, 18, 3)):
            assert bool((plane.flatten(0, 1)[rest] == fill).all())
        for (c, s), want, slack in ((kv8[:2], want_k, slack_k), (kv8[2:], f64(v), 0 * f64(v))):
            got_s = f64(s.flatten(0, 1))[slot[live]]
            got = e4m3(c.flatten(0, 1))[slot[live]] * np.repeat(got_s, 128, -1)
            want_s = quantise64(want)[live]
            tol_s = quantise64(slack)[live] + 2.0 ** -23 * want_s
            assert np.all(np.abs(got_s - want_s) <= tol_s)
            # half an E4M3 step: 2^-4 of the value, 2^-10 scales below the normal range (values under 2^-6 scales)
            step = np.maximum(2.0 ** -4 * np.abs(want[live]), 2.0 ** -10 * np.repeat(want_s, 128, -1))
            assert np.all(np.abs(got - want[live]) <= 1.001 * step + 2 * slack[live])
        # V, not turned: the same bits as the quantiser of flat caches (rows of 256 dims)
        if dim == 256:
            c, s = torch.empty(n, kv_heads, 256, **codes), torch.empty(n, kv_heads, 2, device=DEV)
            qb.qsa_quantize_kv_fp8(v.contiguous(), c, s)
            at = torch.from_numpy(live).to(DEV)
            assert torch.equal(kv8[2].flatten(0, 1)[slot[live]], c[at])
            assert torch.equal(kv8[3].flatten(0, 1)[slot[live]], s[at])
    check_rope(f64(q_out)[live], want_q[live], slack_q[live])
    assert bool((q_out[torch.from_numpy(~live).to(DEV)] == 9).all())
    assert status(ws) == (0, 0)


def test_append_without_queries_and_in_place(cuda_lib):
    cfg = qb.make_paged_config(4, 2, 128, 8)
    ws, rope = qb.paged_workspace(cfg), qb.rope_table(128)
    fused = randn((6, 8, 128), seed=3)
    pos, table = ints([0, 1, 2, 3, 4, 5]), ints([[1], [0], [3], [2], [5], [4]])
    a = [torch.zeros(6, 8, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    q_out = torch.empty(6, 4, 128, dtype=torch.bfloat16, device=DEV)
    qb.qsa_rope_append(cfg, rope, fused[:, :4], fused[:, 4:6], fused[:, 6:], pos, None, q_out, a[0], a[1], table, ws)
    qb.qsa_rope_append(cfg, rope, None, fused[:, 4:6], fused[:, 6:], pos, None, None, a[2], a[3], table, ws)
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])
    qb.qsa_rope_append(cfg, rope, fused[:, :4], fused[:, 4:6], fused[:, 6:], pos, None, fused[:, :4], a[2], a[3], table,
                       ws)
    assert torch.equal(fused[:, :4], q_out)
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("seq,pos,page", [(3, 0, 0), (0, -1, 0), (0, 16, 0), (0, 3, -1), (0, 3, 4)])
def test_append_skips_and_records_bad_targets(cuda_lib, seq, pos, page):
    cfg = qb.make_paged_config(4, 2, 128, 8)
    ws, rope = qb.paged_workspace(cfg), qb.rope_table(128)
    fused = randn((2, 8, 128), seed=4)
    table = ints([[1, 2], [0, 3], [page, page]])
    table[0] = table[2] if page not in (0,) else table[0]
    kc = torch.full((4, 8, 2, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    q_out = torch.empty(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    qb.qsa_rope_append(cfg, rope, fused[:, :4], fused[:, 4:6], fused[:, 6:], ints([7, pos]), ints([1, seq]), q_out, kc,
                       vc, table, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1)
    assert torch.equal(vc[0, 7], fused[0, 6:])            # the good token is stored
    vc[0, 7] = 5.0
    kc[0, 7] = 5.0
    assert bool((vc == 5).all()) and bool((kc == 5).all())


# ------------------------------------------------------------------------------------------ attention
def paged_inputs(lens, Hq, Hkv, D, page, fp8, seed, spare=3, scale=1.0, fill=float("nan")):
    """Pages in random order; what no token lies in is NaN (bf16) or NaN codes."""
    rng = np.random.default_rng(seed)
    count = [-(-n // page) for n in lens]
    n_pages, ld = sum(count) + spare, max(count + [1]) + 1
    order = rng.permutation(n_pages)
    table = np.full((len(lens), ld), -1)
    at = 0
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        at += c
    k, v = (randn((n_pages, page, Hkv, D), seed + i, scale) for i in (1, 2))
    used = torch.zeros(n_pages * page, dtype=torch.bool, device=DEV)
    for r, n in enumerate(lens):
        used[P.slots_of(table[r], n, page)] = True
    q = randn((len(lens), Hq, D), seed + 3)
    if not fp8:
        for t in (k, v):
            t.flatten(0, 1)[~used] = fill
        return q, (k, v), (f64(k), f64(v)), ints(table.tolist()), table
    planes, values = [], []
    for t in (k, v):
        x = t.float().reshape(n_pages, page, Hkv, D // 128, 128)
        s = x.abs().amax(-1) / 448.0
        c = (x / s[..., None]).to(torch.float8_e4m3fn)
        values.append(f64(c.float()).reshape(t.shape) * np.repeat(f64(s), 128, -1))
        c = c.view(torch.uint8).reshape(t.shape)
        c.flatten(0, 1)[~used] = 0x7F
        s.flatten(0, 1)[~used] = float("nan")
        planes += [c, s]
    return q, tuple(planes), tuple(values), ints(table.tolist()), table


def run_decode(cfg, q, planes, table, lens, ws, out=None, lse=None, stream=None):
    B = q.shape[0]
    out = torch.full((B, cfg.n_q_heads, cfg.head_dim), 8.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((B, cfg.n_q_heads), 8.0, device=DEV) if lse is None else lse
    if len(planes) == 2:
        qb.qsa_paged_decode(cfg, q, *planes, table, lens, out, lse, ws, stream)
    else:
        qb.qsa_paged_decode_fp8kv(cfg, q, planes, table, lens, out, lse, ws, stream)
    return out, lse


def check_decode(out, lse, q, values, table, lens, page, window, scale, fp8=False, q_step=0.0):
    out, lse, q = f64(out), f64(lse), f64(q)
    for r, n in enumerate(lens):
        slots = P.slots_of(table[r], n, page)
        K, V = (x.reshape(-1, *x.shape[2:])[slots] for x in values)
        lo = max(0, n - window) if window else 0
        want, want_lse, mass, terms = P.decode(q[r], K, V, lo, scale)
        D = q.shape[-1]
        ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1)
        if q_step and n:                                  # q off by q_step of its head's largest
            ds = ds + q_step * np.abs(q[r]).max(1) * np.abs(K[lo:]).sum(2).max() * scale
        if n == 0:
            assert np.all(out[r] == 0) and np.all(np.isneginf(lse[r]))
            continue
        sums = n / 8 * 2.0 ** -24 + 2.0 ** -15
        tol = 2.0 ** -8 * np.abs(want) + (2 * ds[:, None] + sums) * mass
        if fp8:
            tol += 2.0 ** -11 * mass + n * 2.0 ** -25 * mass.max(1, keepdims=True)
        assert np.all(np.abs(out[r] - want) <= tol), (r, n, np.abs(out[r] - want).max(), tol.min())
        assert np.all(np.abs(lse[r] - want_lse) <= ds + sums + 2.0 ** -22 * np.abs(want_lse)), (r, n)


DECODE_GEOMETRY = [(16, 2, 256, 64, False), (8, 2, 256, 16, False), (7, 1, 128, 24, False), (8, 8, 64, 100, False),
                   (32, 2, 64, 4, False), (3, 3, 128, 1, False), (12, 1, 256, 7, False),
                   (16, 2, 256, 64, True), (8, 2, 256, 3, True), (32, 8, 128, 24, True), (15, 1, 128, 256, True)]


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", DECODE_GEOMETRY)
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 0, 127, 129], [3000], [5, 0, 1500, 700, 64, 0]])
@pytest.mark.parametrize("window", [0, 50])
def test_decode(cuda_lib, Hq, Hkv, D, page, fp8, lens, window):
    q, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, page, fp8, seed=Hq + D + len(lens))
    cfg = qb.make_paged_config(Hq, Hkv, D, page, window=window)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    check_decode(out, lse, q, values, table, lens, page, window, D ** -0.5, fp8)
    assert status(ws) == (0, 0)
    again, lse2 = run_decode(cfg, q, planes, tab, ints(lens), ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # without lse
    third = torch.empty_like(out)
    if fp8:
        qb.qsa_paged_decode_fp8kv(cfg, q, planes, tab, ints(lens), third, None, ws)
    else:
        qb.qsa_paged_decode(cfg, q, *planes, tab, ints(lens), third, None, ws)
    assert torch.equal(out, third)


@pytest.mark.parametrize("Hq,Hkv,D,page,fp8", [(16, 2, 256, 64, False), (4, 4, 64, 16, False), (16, 2, 256, 48, True)])
def test_decode_long_and_many(cuda_lib, Hq, Hkv, D, page, fp8):
    rng = np.random.default_rng(5)
    lens = [20000] + rng.integers(0, 300, 600).tolist() + [9999, 1]
    q, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, page, fp8, seed=9)
    cfg = qb.make_paged_config(Hq, Hkv, D, page, softmax_scale=0.11)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    check_decode(out, lse, q, values, table, lens, page, 0, float(np.float32(0.11)), fp8)
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_sharp_scores_and_wide_value_scales(cuda_lib, fp8):
    """Scores of a few hundred (one token takes nearly all) and V rows from 2^-20 to 2^20: tokens that matter
    are not lost beside larger ones that do not."""
    lens = [700, 130]
    q, planes, values, tab, table = paged_inputs(lens, 16, 2, 256, 16, fp8, seed=21, scale=8.0)
    factor = 2.0 ** torch.randint(-20, 21, planes[0].shape[:3], generator=torch.Generator().manual_seed(1)).to(DEV)
    if fp8:
        planes[3].mul_(factor[..., None])
    else:
        planes[1].mul_(factor[..., None].to(torch.bfloat16))
    values = (values[0], values[1] * f64(factor)[..., None])
    cfg = qb.make_paged_config(16, 2, 256, 16)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws := qb.paged_workspace(cfg))
    check_decode(out, lse, q, values, table, lens, 16, 0, 1 / 16, fp8)
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (5, 1, 256), (12, 1, 256), (8, 2, 128)])
def test_decode_queries_of_a_wide_range_over_fp8_rows(cuda_lib, Hq, Hkv, D):
    """Values of one head from 2^-20 to 1 of its largest, heads from 2^-30 to 8 and zero: over FP8 rows a query value may be
    rounded by 2^-22 of its head's largest (two E4M3 parts, the second with steps of 2^-21 of it)."""
    lens = [300, 40]
    q, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, 16, True, seed=61)
    g = torch.Generator().manual_seed(2)
    q = (q * (2.0 ** torch.randint(-20, 1, q.shape, generator=g).to(DEV))).to(torch.bfloat16)
    heads = 2.0 ** torch.randint(-30, 1, (2, Hq, 1), generator=g).to(DEV)
    heads[0, 0], heads[1, Hq - 1] = 8.0, 0.0                  # few tokens matter; all count alike
    q = (q * heads).to(torch.bfloat16).contiguous()
    cfg = qb.make_paged_config(Hq, Hkv, D, 16)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    check_decode(out, lse, q, values, table, lens, 16, 0, D ** -0.5, True, q_step=2.0 ** -22)
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq,D,fp8", [(8, 256, True), (16, 256, True), (8, 128, True), (8, 256, False)])
def test_decode_query_that_is_not_finite_spoils_its_head_alone(cuda_lib, Hq, D, fp8, value):
    lens = [70, 50]
    q, planes, values, tab, table = paged_inputs(lens, Hq, 1, D, 16, fp8, seed=71)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    want, want_lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    bad = q.clone()
    bad[0, 3, 5] = value
    out, lse = run_decode(cfg, bad, planes, tab, ints(lens), ws)
    assert bool(torch.isnan(out[0, 3]).all())
    keep = torch.ones(2, Hq, dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("Hq,D", [(8, 256), (16, 256), (8, 128), (16, 128)])
@pytest.mark.parametrize("plane", [1, 3])
def test_decode_scale_that_is_not_a_number_spoils_its_row_alone(cuda_lib, Hq, D, plane):
    lens = [70, 50]
    q, planes, values, tab, table = paged_inputs(lens, Hq, 1, D, 16, True, seed=73)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    want, _ = run_decode(cfg, q, planes, tab, ints(lens), ws)
    page = int(table[0][1])
    planes[plane][page, 3, 0, 0] = float("nan")                # token 19 of row 0, its first 128 dims
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    assert bool(torch.isnan(out[0, :, :128]).all()) and torch.equal(out[1], want[1])
    if plane == 1:
        assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())


def test_decode_strided_queries(cuda_lib):
    lens = [40, 300, 7]
    q, planes, values, tab, table = paged_inputs(lens, 8, 2, 128, 16, False, seed=31)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    fused = torch.full((3, 12, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[:, 2:10] = q
    again, _ = run_decode(cfg, fused[:, 2:10], planes, tab, ints(lens), ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_leaves_out_and_records_bad_pages(cuda_lib, fp8):
    lens = [200, 100, 90]
    q, planes, values, tab, table = paged_inputs(lens, 8, 2, 128, 16, fp8, seed=41)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    ws = qb.paged_workspace(cfg)
    bad = tab.clone()
    bad[1, 3] = planes[0].shape[0]                        # one past the pool: tokens 48..63 of row 1
    out, lse = run_decode(cfg, q, planes, bad, ints(lens), ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1)
    # the other rows are right, and row 1 attends its other tokens
    rows = [0, 2]
    check_decode(out[rows], lse[rows], q[rows], values, table[rows], [200, 90], 16, 0, 128 ** -0.5, fp8)
    slots = P.slots_of(table[1], 100, 16)
    slots = np.concatenate([slots[:48], slots[64:]])
    flat = [x.reshape(-1, *x.shape[2:])[slots] for x in values]
    want = P.decode(f64(q[1]), *flat, 0, 128 ** -0.5)[0]
    assert np.abs(f64(out[1]) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    # a length past the table, or negative, counts as empty
    for n in (tab.shape[1] * 16 + 1, -1):
        ws = qb.paged_workspace(cfg)
        out, lse = run_decode(cfg, q, planes, tab, ints([200, n, 90]), ws)
        assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1)
        assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
        check_decode(out[rows], lse[rows], q[rows], values, table[rows], [200, 90], 16, 0, 128 ** -0.5, fp8)


def test_decode_agrees_with_the_sparse_decode_on_short_contexts(cuda_lib):
    """Up to 2051 tokens the sparse path attends everything: the paged decode over the same flat cache (identity
    pages) gives its result. Both round once to bf16: off by 2^-7 of the value, and the scores' fp32 sums."""
    ctx = [3, 700, 2050]
    b = DecodeBatch(16, 2, ctx)
    T = b.n_tokens
    k, v, q = randn((T, 2, 256), 1), randn((T, 2, 256), 2), randn((3, 16, 256), 3)
    nb = [p // 4 for p in ctx]
    blocks = torch.full((3, 512), -1, dtype=torch.int32)
    for r, n in enumerate(nb):
        blocks[r, :n] = torch.arange(n)
    b.attend(q, k, v, blocks.to(DEV), ints(nb))
    cfg = qb.make_paged_config(16, 2, 256, 1)
    table = torch.full((3, 2051), -1, dtype=torch.int32)
    for r, p in enumerate(ctx):
        table[r, :p + 1] = torch.arange(p + 1) + int(b.tok_off[r])
    out, lse = run_decode(cfg, q, (k.view(T, 1, 2, 256), v.view(T, 1, 2, 256)), table.to(DEV), ints([p + 1 for p in ctx]),
                          qb.paged_workspace(cfg))
    scale = np.abs(f64(b.out))
    assert np.all(np.abs(f64(out) - f64(b.out)) <= 2.0 ** -7 * scale + 2e-4)
    assert np.abs(f64(lse) - f64(b.lse)).max() <= 2e-5


def test_decode_from_pinned_host_memory(cuda_lib):
    lens = [333, 20]
    q, planes, values, tab, table = paged_inputs(lens, 8, 2, 128, 16, False, seed=51)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    ws = qb.paged_workspace(cfg)
    out, _ = run_decode(cfg, q, planes, tab, ints(lens), ws)
    host = tuple(p.cpu().pin_memory() for p in planes)
    again, _ = run_decode(cfg, q, host, tab, ints(lens), ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def test_decode_captured_replays_with_new_lengths_on_another_stream(cuda_lib):
    """A captured step reads lengths, tables and caches anew at each replay; two batches of other sizes share the
    workspace in between."""
    page = 16
    lens = [500, 0, 64]
    q, planes, values, tab, table = paged_inputs([700] * 3, 16, 2, 128, page, False, seed=61)
    cfg = qb.make_paged_config(16, 2, 128, page)
    ws = qb.paged_workspace(cfg)
    dev_lens = ints(lens)
    out, lse = torch.empty_like(q), torch.empty(3, 16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_decode(cfg, q, planes, tab, dev_lens, ws, out, lse)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run_decode(cfg, q, planes, tab, dev_lens, ws, out, lse)
    for now in ([500, 0, 64], [1, 700, 333], [700, 700, 700], [0, 0, 0]):
        dev_lens.copy_(ints(now))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        check_decode(out, lse, q, values, table, now, page, 0, 128 ** -0.5)
        one, one_lse = run_decode(cfg, q[:1], planes, tab[:1], ints([650]), ws)
        check_decode(one, one_lse, q[:1], values, table[:1], [650], page, 0, 128 ** -0.5)
    assert status(ws) == (0, 0)


# ------------------------------------------------------------------------------------------ pages
def random_pool(S, page, high, spare, seed, shared=True):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, high + 1, S)
    ld = -(-high // page) + 3
    count = -(-lens // page)
    n_pages = int(count.sum()) + spare
    order = rng.permutation(n_pages)
    table, ref, at = np.full((S, ld), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        at += c
    if shared and S > 1:                                  # the last row starts with row 0's full pages
        both = min(lens[0], lens[-1]) // page
        table[-1, :both] = table[0, :both]
    for r, c in enumerate(count):
        np.add.at(ref, table[r, :c], 1)
    return table, lens.astype(np.int32), ref


def planes_of(n_pages, page, seed):
    """A wide plane group (16-byte words), and one of 4-byte words."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-2 ** 15, 2 ** 15, (3, n_pages, page, 8), dtype=torch.int16, generator=g).to(DEV),
            torch.randn((2, n_pages, page, 1), generator=g).to(DEV)]


def copied(plane, copies, page):
    want = plane.clone()
    row = plane[0, 0].numel() // page * plane.element_size()
    word = 16 if row * page % 16 == 0 else 4
    for src, dst, used in copies:
        part = -(-used * row // word) * word // plane.element_size()
        want[:, dst].flatten(1)[:, :part] = plane[:, src].flatten(1)[:, :part]
    return want


@pytest.mark.parametrize("S,page,high,spare", [(1, 4, 9, 5), (8, 16, 100, 30), (300, 8, 60, 1500), (70, 1, 5, 400),
                                               (5, 1000, 3000, 12), (1030, 4, 20, 4000), (20, 2, 90, 17000),
                                               (600, 1, 120, 3000)])
@pytest.mark.parametrize("kind", ["beams", "extend", "any", "free"])
def test_fork(cuda_lib, S, page, high, spare, kind):
    table, lens, ref = random_pool(S, page, high, spare, seed=S + page)
    rng = np.random.default_rng(S)
    n_out = S if kind != "any" else S + 7
    parent = {"beams": np.arange(S) // 4 * 4 % S, "extend": np.arange(S), "free": np.full(S, -1),
              "any": rng.integers(-1, S, n_out)}[kind]
    add = np.zeros(S, int) if kind == "free" else rng.integers(0, 3, n_out)
    if kind == "any":
        ref[table[0, 0]] += int(lens[0] > 0)              # another holder keeps row 0's first page
    planes = planes_of(len(ref), page, 1)
    want_planes = None
    want = P.fork(table, lens, ref, parent.tolist(), add.tolist(), page)
    want_planes = [copied(p, want[3], page) for p in planes]
    ws = qb.pages_workspace(max(S, n_out), len(ref))
    t_out = torch.full((n_out, table.shape[1]), 77, dtype=torch.int32, device=DEV)
    l_out, r_out = torch.full((n_out,), 77, dtype=torch.int32, device=DEV), torch.full((len(ref),), 77, dtype=torch.int32,
                                                                                      device=DEV)
    args = (page, ints(parent.tolist()), ints(add.tolist()), ints(table.tolist()), ints(lens.tolist()))
    ref_dev = ints(ref.tolist())
    qb.qsa_fork_pages(*args, ref_dev, t_out, l_out, r_out, planes, ws)
    assert np.array_equal(t_out.cpu().numpy(), want[0])
    assert np.array_equal(l_out.cpu().numpy(), want[1])
    assert np.array_equal(r_out.cpu().numpy(), want[2])
    for got, w in zip(planes, want_planes):
        assert torch.equal(got, w)
    assert want[4] == [] and status(ws) == (0, 0)
    r_out.fill_(77)
    qb.qsa_fork_pages(*args, ref_dev, t_out, l_out, r_out, [], ws)            # no planes: bookkeeping alone
    assert np.array_equal(r_out.cpu().numpy(), want[2]) and np.array_equal(t_out.cpu().numpy(), want[0])


def test_fork_rows_that_find_no_page_become_empty(cuda_lib):
    page = 4
    table, lens, ref = random_pool(6, page, 30, 3, seed=3)
    parent, add = [0, 1, 2, 3, 4, 5, 6, -2], [12, 0, 24, 30, 0, 1, 0, 0]
    want = P.fork(table, lens, ref, parent, add, page)
    assert want[4] == [3, 5, 6, 7]                        # rows 3 and 5 find no page; row 4 needs none
    ws = qb.pages_workspace(8, len(ref))
    t_out, l_out = torch.zeros((8, table.shape[1]), dtype=torch.int32, device=DEV), ints([0] * 8)
    r_out, planes = ints([0] * len(ref)), planes_of(len(ref), page, 2)
    want_planes = [copied(p, want[3], page) for p in planes]
    qb.qsa_fork_pages(page, ints(parent), ints(add), ints(table.tolist()), ints(lens.tolist()), ints(ref.tolist()), t_out,
                      l_out, r_out, planes, ws)
    assert np.array_equal(t_out.cpu().numpy(), want[0]) and np.array_equal(l_out.cpu().numpy(), want[1])
    assert np.array_equal(r_out.cpu().numpy(), want[2])
    assert all(torch.equal(a, b) for a, b in zip(planes, want_planes))
    st, row = status(ws)
    assert st == qb.QSA_ERR_DEVICE_BOUNDS and row in want[4]


@pytest.mark.parametrize("S,page,high,spare", [(1, 4, 9, 5), (8, 16, 100, 30), (300, 8, 60, 1500), (0, 4, 8, 9),
                                               (40, 2, 700, 9000), (40, 2, 700, 9), (16, 4, 90, 30000), (1500, 4, 40, 11)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(cuda_lib, S, page, high, spare, in_place):
    table, lens, ref = random_pool(S, page, high, spare, seed=S + 1)
    want_t, want_r, moves = P.compact(table, lens, ref, page)
    planes = planes_of(len(ref), page, 4)
    want_planes = []
    for p in planes:
        w = p.clone()
        for old, new in moves.items():
            w[:, new] = p[:, old]
        want_planes.append(w)
    ws = qb.pages_workspace(max(S, 1), len(ref))
    t, r = ints(table.tolist()).reshape(table.shape), ints(ref.tolist())
    t_out, r_out = t if in_place else torch.full_like(t, 77), torch.full_like(r, 77)
    qb.qsa_compact_pages(page, t, ints(lens.tolist()), r, t_out, r_out, planes, ws)
    assert np.array_equal(t_out.cpu().numpy(), want_t) and np.array_equal(r_out.cpu().numpy(), want_r)
    assert all(torch.equal(a, b) for a, b in zip(planes, want_planes))
    assert status(ws) == (0, 0)
    # a compact pool stays as it is
    again = torch.full_like(r, 77)
    qb.qsa_compact_pages(page, t_out, ints(lens.tolist()), r_out, t_out, again, planes, ws)
    assert torch.equal(again, r_out)
    assert np.array_equal(t_out.cpu().numpy(), want_t) and all(torch.equal(a, b) for a, b in zip(planes, want_planes))


def test_compact_records_entries_without_a_live_page(cuda_lib):
    ws = qb.pages_workspace(2, 6)
    table, ref = ints([[4, 9], [2, 1]]), ints([0, 1, 0, 0, 1, 0])      # row 0's page 9 is outside, row 1's page 2 is free
    t_out, r_out = torch.zeros_like(table), torch.zeros_like(ref)
    qb.qsa_compact_pages(4, table, ints([3, 8]), ref, t_out, r_out, [], ws)
    assert t_out.tolist() == [[0, -1], [-1, 1]] and r_out.tolist() == [1, 1, 0, 0, 0, 0]
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1)


def test_copy_pages_out_to_the_host_and_back(cuda_lib):
    planes = planes_of(20, 4, 5)
    keep = [p.clone() for p in planes]
    host = [torch.zeros((p.shape[0], 6) + p.shape[2:], dtype=p.dtype).pin_memory() for p in planes]
    ws = qb.pages_workspace(1, 20)
    qb.qsa_copy_pages(ints([3, 19, -1, 0]), ints([5, 0, 1, 2]), planes, ws, dst_planes=host)
    torch.cuda.synchronize()
    for h, p in zip(host, keep):
        assert torch.equal(h[:, 5], p[:, 3].cpu()) and torch.equal(h[:, 0], p[:, 19].cpu())
        assert torch.equal(h[:, 2], p[:, 0].cpu()) and not h[:, [1, 3, 4]].any()
    for p in planes:
        p.zero_()
    qb.qsa_copy_pages(ints([5, 0, 2]), ints([3, 19, 0]), host, ws, dst_planes=planes)
    for p, k in zip(planes, keep):
        assert torch.equal(p[:, [3, 19, 0]], k[:, [3, 19, 0]]) and not p[:, 1:3].any()
    qb.qsa_copy_pages(ints([3, 3]), ints([7, 8]), planes, ws)
    for p, k in zip(planes, keep):
        assert torch.equal(p[:, 7], k[:, 3]) and torch.equal(p[:, 8], k[:, 3])
    assert status(ws) == (0, 0)
    qb.qsa_copy_pages(ints([3, 20]), ints([9, 10]), planes, ws)
    assert status(ws) == (qb.QSA_ERR_DEVICE_BOUNDS, 1) and torch.equal(planes[0][:, 9], keep[0][:, 3])


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_loop_with_beams_and_compaction(cuda_lib, fp8):
    """A prompt and five decode steps of four beams that fork, over two layers; every step's attention against
    the tokens each beam has seen, and the same bits after compaction."""
    L, page, Hq, Hkv, D, rows = 2, 8, 8, 2, 128, 4
    cache = PagedCache(L, 60, page, rows, 8, Hq, Hkv, D, fp8=fp8)
    rope = qb.rope_table(D, base=1e4)
    rng = np.random.default_rng(0)

    def tokens(n, seed):
        return [randn((n, Hq + 2 * Hkv, D), 1000 * seed + l) for l in range(L)]

    prompt = 19
    cache.fork(ints([-1] * rows), ints([prompt, 0, 0, 0]))
    pos = torch.arange(prompt, dtype=torch.int32, device=DEV)
    fused = tokens(prompt, 1)
    for l in range(L):
        q_out = torch.empty(prompt, Hq, D, dtype=torch.bfloat16, device=DEV)
        cache.append(l, rope, fused[l][:, :Hq], fused[l][:, Hq:Hq + Hkv], fused[l][:, Hq + Hkv:], pos,
                     torch.zeros(prompt, dtype=torch.int32, device=DEV), q_out)
    # hist[r][l]: the projection rows of the tokens that row r has seen in layer l
    hist = [[[fused[l][t] for t in range(prompt)] for l in range(L)] for _ in range(rows)]
    parent = [0, 0, 0, 0]
    for step in range(5):
        cache.fork(ints(parent), ints([1] * rows))
        lens = cache.seq_len.tolist()
        assert lens == [prompt + step + 1] * rows
        new = tokens(rows, step + 2)
        hist = [[list(hist[p][l]) + [new[l][r]] for l in range(L)] for r, p in enumerate(parent)]
        for l in range(L):
            q_out = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=DEV)
            cache.append(l, rope, new[l][:, :Hq], new[l][:, Hq:Hq + Hkv], new[l][:, Hq + Hkv:], cache.seq_len - 1, None,
                         q_out)
            out, lse = torch.empty_like(q_out), torch.empty(rows, Hq, device=DEV)
            cache.attend(l, q_out, out, lse)
            for r in range(rows):
                n = lens[r]
                seen = f64(torch.stack(hist[r][l]))
                freq, amp = P.rope_frequencies(D, 1e4)
                K = P.rope(seen[:, Hq:Hq + Hkv], np.arange(n), freq, amp, 0, False)
                want = P.decode(f64(q_out[r]), K, seen[:, Hq + Hkv:], 0, D ** -0.5)[0]
                # K rounded to bf16 (2^-8) or E4M3 (2^-4), V to E4M3: scores off by a few hundredths at most
                assert np.abs(f64(out[r]) - want).max() <= (0.25 if fp8 else 0.03), (step, l, r)
            if step == 3:
                keep = (out.clone(), lse.clone())
                if l == L - 1:
                    cache.compact()
                    live = cache.ref > 0
                    assert bool(live[: int(live.sum())].all())
                    cache.attend(l, q_out, out, lse)
                    assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1])
        parent = rng.integers(0, rows, rows).tolist()
    cache.fork(ints([-1] * rows), ints([0] * rows))
    assert not cache.ref.any() and cache.seq_len.tolist() == [0] * rows
    assert cache.status() == ((0, 0), (0, 0))


def test_captured_decode_steps_replay(cuda_lib):
    """Two decode steps (the bookkeeping alternates between two sets of arrays) captured with their forks, appends
    and attention; replays continue the sequences as eager steps do. Another stream, and a kernel of another
    kind right before and behind."""
    page, Hq, Hkv, D, rows = 4, 4, 2, 64, 3
    rope = qb.rope_table(D)

    def build():
        c = PagedCache(1, 40, page, rows, 8, Hq, Hkv, D)
        c.fork(ints([-1] * rows), ints([3, 0, 9]))
        return c

    fused = torch.empty(rows, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    q_out = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q_out)
    source = randn((rows, Hq + 2 * Hkv, D), 5)
    grow = torch.ones(1, dtype=torch.bfloat16, device=DEV)
    parents = [ints([0, 0, 2]), ints([1, 1, 2])]

    def step(c, parent):
        torch.mul(source, grow, out=fused)                # what the attention input's producer would be
        grow.mul_(1.5)
        c.fork(parent, ints_one)
        c.append(0, rope, fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:], last(c), None, q_out)
        c.attend(0, q_out, out)
        return out

    ints_one = ints([1] * rows)
    pos = torch.empty(rows, dtype=torch.int32, device=DEV)

    def last(c):
        torch.sub(c.seq_len, 1, out=pos)
        return pos

    eager = build()
    want = []
    for i in range(8):
        want.append(step(eager, parents[i % 2]).clone())
    grow.fill_(1.0)
    cache = build()
    keep = torch.zeros(2, *out.shape, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for i in range(2):
            keep[i].copy_(step(cache, parents[i]))
    for i in range(4):
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert torch.equal(keep[0], want[2 * i]) and torch.equal(keep[1], want[2 * i + 1]), i
    assert torch.equal(cache.table, eager.table) and torch.equal(cache.ref, eager.ref)
    assert torch.equal(cache.seq_len, eager.seq_len) and cache.status() == ((0, 0), (0, 0))


def test_calls_take_a_stream(cuda_lib):
    side = torch.cuda.Stream()
    x = randn((5, 2, 128), 1)
    pos = ints([1, 2, 3, 4, 5])
    rope = qb.rope_table(128)
    a, b = torch.empty_like(x), torch.empty_like(x)
    qb.qsa_rope(rope, x, pos, a)
    torch.cuda.synchronize()
    qb.qsa_rope(rope, x, pos, b, stream=side)
    qb.qsa_rope(rope, b, -pos, b, stream=side.cuda_stream)
    side.synchronize()
    again = torch.empty_like(x)
    qb.qsa_rope(rope, a, -pos, again)
    assert torch.equal(b, again)
    q, planes, values, tab, table = paged_inputs([70, 3], 8, 2, 128, 16, False, seed=3)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    ws = qb.paged_workspace(cfg)
    torch.cuda.synchronize()
    out, lse = torch.empty_like(q), torch.empty(2, 8, device=DEV)
    lens = ints([70, 3])
    torch.cuda.synchronize()
    run_decode(cfg, q, planes, tab, lens, ws, out, lse, stream=side)
    side.synchronize()
    check_decode(out, lse, q, values, table, [70, 3], 16, 0, 128 ** -0.5)


@pytest.mark.parametrize("Hq,D,fp8", [(8, 64, False), (8, 256, False), (8, 128, True), (16, 256, True)])
def test_decode_of_the_longest_sequence(cuda_lib, Hq, D, fp8):
    """2^31 - 1 tokens, all pages the same one, and a window over the last 100: the last tile reaches past 2^31."""
    page, n, window = 1 << 20, (1 << 31) - 1, 100
    groups = D // 128
    if fp8:
        planes = [torch.full((1, page, 1, D), 0x7F, dtype=torch.uint8, device=DEV),
                  torch.full((1, page, 1, groups), float("nan"), device=DEV)]
        planes += [p.clone() for p in planes]
    else:
        planes = [torch.full((1, page, 1, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q, small, values, _, _ = paged_inputs([window], Hq, 1, D, 128, fp8, seed=91, spare=0)
    at = slice(page - 1 - window, page - 1)               # token n - 1 lies in slot page - 2 of page 2047
    order = slice(0, window)
    for p, x in zip(planes, small):
        p[0, at] = x[0, order]
    cfg = qb.make_paged_config(Hq, 1, D, page, 0.0, window)
    ws = qb.paged_workspace(cfg)
    table = torch.zeros(1, 2048, dtype=torch.int32, device=DEV)
    out, lse = run_decode(cfg, q, tuple(planes), table, ints([n]), ws)
    assert status(ws) == (0, 0)
    check_decode(out, lse, q, values, np.zeros((1, 1), dtype=np.int64), [window], 128, 0, D ** -0.5, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_slots_of_a_large_cache(cuda_lib, fp8):
    """Rows whose byte offsets pass 2^32 (and 2^33 with bf16 rows): appended, attended, copied and compacted."""
    page, Hkv, D = 64, 8, 128
    row = D if fp8 else 2 * D
    n_pages = (5 << 30) // (page * Hkv * row)             # 5 GB a plane
    shape = (n_pages, page, Hkv, D)
    if fp8:
        pool = [torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty(shape[:3] + (1,), device=DEV),
                torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty(shape[:3] + (1,), device=DEV)]
    else:
        pool = [torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    cfg = qb.make_paged_config(16, Hkv, D, page)
    ws = qb.paged_workspace(cfg)
    n = 3 * page - 5
    table = ints([[n_pages - 1, n_pages // 2 + 7, n_pages - 3]])
    fused = randn((n, 16 + 2 * Hkv, D), 8)
    q_out = torch.empty(n, 16, D, dtype=torch.bfloat16, device=DEV)
    rope = qb.rope_table(D)
    args = (cfg, rope, fused[:, :16], fused[:, 16:16 + Hkv], fused[:, 16 + Hkv:],
            torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV), q_out)
    q = q_out[-1:]

    def attend(planes, tab):
        return run_decode(cfg, q, planes, tab, ints([n]), ws)

    if fp8:
        qb.qsa_rope_append_fp8kv(*args, pool, table, ws)
        small = [p[table[0].long()].contiguous() for p in pool]
    else:
        qb.qsa_rope_append(*args, *pool, table, ws)
        small = [p[table[0].long()].contiguous() for p in pool]
    out, lse = attend(pool, table)
    near, near_lse = attend(small, ints([[0, 1, 2]]))
    assert torch.equal(out, near) and torch.equal(lse, near_lse)
    freq, amp = P.rope_frequencies(D, 1e4)
    K = P.rope(f64(fused[:, 16:16 + Hkv]), np.arange(n), freq, amp, 0, False)
    want = P.decode(f64(q[0]), K, f64(fused[:, 16 + Hkv:]), 0, D ** -0.5)[0]
    assert np.abs(f64(out[0]) - want).max() <= (0.25 if fp8 else 0.03)
    # the page calls over the same planes
    planes = [p[None] for p in pool]
    pws = qb.pages_workspace(2, n_pages)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    ref[table[0].long()] = 1
    t2, r2 = torch.empty_like(table), torch.empty_like(ref)
    qb.qsa_compact_pages(page, table, ints([n]), ref, t2, r2, planes, pws)
    assert t2.tolist() == [[2, 0, 1]]
    out, lse = attend(pool, t2)
    assert torch.equal(out, near)
    t3, l3, r3 = torch.empty(2, 3, dtype=torch.int32, device=DEV), ints([0, 0]), torch.empty_like(ref)
    qb.qsa_fork_pages(page, ints([0, 0]), ints([0, 0]), t2, ints([n]), r2, t3, l3, r3, planes, pws)
    assert t3.tolist() == [[2, 0, 1], [2, 0, 3]]
    out, lse = attend(pool, t3[1:])
    assert torch.equal(out, near)
    qb.qsa_copy_pages(t3[1], ints([n_pages - 2, 5, n_pages - 9]), planes, pws)
    out, lse = attend(pool, ints([[n_pages - 2, 5, n_pages - 9]]))
    assert torch.equal(out, near)
    assert status(ws) == (0, 0) and status(pws) == (0, 0)


def test_host_checks_reach_python(cuda_lib):
    """A refused call raises with the library's text and launches nothing: misaligned rows, host memory that the
    GPU cannot read, a workspace that is too small, arrays that must differ."""
    rope = qb.rope_table(64)
    x = torch.zeros(3 * 2 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    pos = ints([0, 1, 2])

    def refused(text, fn, *args, **kw):
        with pytest.raises(qb.QsaError, match=text) as e:
            fn(*args, **kw)
        assert e.value.status in (qb.QSA_ERR_INVALID_ARGUMENT, qb.QSA_ERR_WORKSPACE_TOO_SMALL)

    off = x[4:4 + 384].view(3, 2, 64)
    refused("x must be 16-byte aligned", qb.qsa_rope, rope, off, pos, x[:384].view(3, 2, 64))
    q, planes, values, tab, table = paged_inputs([30, 3], 8, 2, 128, 16, False, seed=2)
    cfg = qb.make_paged_config(8, 2, 128, 16)
    ws = qb.paged_workspace(cfg)
    out = torch.empty_like(q)
    pageable = [p.cpu() for p in planes]
    lens = ints([30, 3])
    refused("pinned", qb.qsa_paged_decode, cfg, q, *pageable, tab, lens, out, None, ws)
    refused("workspace", qb.qsa_paged_decode, cfg, q, *planes, tab, lens, out, None, ws[:256])
    r128 = qb.rope_table(128)
    kv = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    refused("pinned", qb.qsa_rope_append, cfg, r128, None, kv[:, :2], kv[:, 2:], ints([0, 1]), None, None, *pageable, tab, ws)
    refused("head_dim", qb.qsa_rope_append, cfg, rope, None, kv[:, :2], kv[:, 2:], ints([0, 1]), None, None, *planes, tab, ws)
    n = planes[0].shape[0]
    pws = qb.pages_workspace(2, n)
    ref, out_ref, t2, l2 = ints([1] * n), ints([0] * n), torch.zeros_like(tab), ints([0, 0])
    host = [pageable[0][None]]
    refused("pinned", qb.qsa_fork_pages, 16, ints([0, 1]), ints([1, 1]), tab, lens, ref, t2, l2, out_ref, host, pws)
    refused("another array", qb.qsa_fork_pages, 16, ints([0, 1]), ints([1, 1]), tab, lens, ref, tab, l2, out_ref, [], pws)
    refused("another array", qb.qsa_compact_pages, 16, tab, lens, ref, t2, ref, [], pws)
    refused("pinned", qb.qsa_compact_pages, 16, tab, lens, ref, t2, out_ref, host, pws)
    refused("pinned", qb.qsa_copy_pages, ints([0]), ints([1]), host, pws)
    with pytest.raises(ValueError, match="current CUDA device"):
        qb.qsa_rope(rope, x[:384].view(3, 2, 64), pos.cpu(), x[:384].view(3, 2, 64))


@pytest.mark.parametrize("Hq,Hkv,D", [(160, 160, 256), (620, 310, 128), (700, 700, 64)])
def test_decode_with_more_kv_heads_than_one_wave(cuda_lib, Hq, Hkv, D):
    lens = [70, 0, 5, 129]
    q, planes, values, tab, table = paged_inputs(lens, Hq, Hkv, D, 16, False, seed=13)
    cfg = qb.make_paged_config(Hq, Hkv, D, 16)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    check_decode(out, lse, q, values, table, lens, 16, 0, D ** -0.5)


def test_workspace_shared_by_other_geometries(cuda_lib):
    """One allocation, large enough for all, used in turn by batches of other sizes, heads and row types, with other
    calls of the library writing over it in between: nothing of a call is left for the next."""
    big = max((qb.paged_workspace(qb.make_paged_config(h, k, d, 16)) for h, k, d in
               ((16, 2, 256), (32, 8, 128), (8, 8, 64))), key=lambda t: t.numel())
    cases = []
    for seed, (Hq, Hkv, D, fp8, lens) in enumerate([(16, 2, 256, False, [3000, 5, 0]), (32, 8, 128, True, [40] * 70),
                                                    (8, 8, 64, False, [9000]), (16, 2, 256, True, [1, 2, 3, 700])]):
        cases.append((Hq, Hkv, D, fp8, lens, *paged_inputs(lens, Hq, Hkv, D, 16, fp8, seed=70 + seed)))
    for turn in range(2):
        for Hq, Hkv, D, fp8, lens, q, planes, values, tab, table in cases:
            big[256:].fill_(0xFF if turn else 0x7F)       # what another operator's scratch may look like
            cfg = qb.make_paged_config(Hq, Hkv, D, 16)
            out, lse = run_decode(cfg, q, planes, tab, ints(lens), big)
            check_decode(out, lse, q, values, table, lens, 16, 0, D ** -0.5, fp8)
    pws = qb.pages_workspace(300, 2000)
    for S, spare in ((300, 900), (8, 30), (40, 200)):
        pws[256:].fill_(0xFF)
        table, lens, ref = random_pool(S, 8, 30, spare, seed=S)
        want = P.fork(table, lens, ref, list(range(S)), [1] * S, 8)
        t2, l2, r2 = torch.zeros(table.shape, dtype=torch.int32, device=DEV), ints([0] * S), ints([0] * len(ref))
        qb.qsa_fork_pages(8, ints(list(range(S))), ints([1] * S), ints(table.tolist()), ints(lens.tolist()),
                          ints(ref.tolist()), t2, l2, r2, [], pws)
        assert np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(r2.cpu().numpy(), want[2])
    assert status(big) == (0, 0) and status(pws) == (0, 0)


# ------------------------------------------------------------------------------------------ limits of the small plan
@pytest.mark.parametrize("n_in,n_out,n_pages,ld", [
    (1024, 1024, 16384, 64), (1025, 1024, 16384, 63), (1024, 1025, 16384, 64), (1024, 1024, 16385, 64),
    (1024, 1024, 16384, 65), (994, 994, 16384, 64), (1024, 1024, 16211, 64), (1, 1024, 16384, 65536), (1024, 1, 16384, 64),
    (1024, 1024, 8192, 8), (1025, 1024, 8192, 7), (1024, 1025, 8192, 8), (1024, 1024, 8193, 8), (1024, 1024, 8192, 9),
    (1, 1024, 8192, 8192), (1, 1, 8192, 8193), (1024, 1, 8192, 8)])
def test_fork_at_the_limits_of_the_single_kernel(cuda_lib, n_in, n_out, n_pages, ld):
    """The largest tables and pools that one kernel plans, and one row, page or entry more."""
    page, rng = 4, np.random.default_rng(n_in + n_pages)
    most = min(ld, n_pages // (2 * max(n_in, n_out))) * page          # half the pool at most, so that every row finds pages
    lens = rng.integers(0, most + 1, n_in).astype(np.int32)
    count, order = -(-lens // page), rng.permutation(n_pages)
    table, ref, at = np.full((n_in, ld), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        ref[order[at:at + c]] = 1
        at += c
    parent, add = rng.integers(-1, n_in, n_out), rng.integers(0, 3, n_out)
    planes = planes_of(n_pages, page, 3)
    want = P.fork(table, lens, ref, parent.tolist(), add.tolist(), page)
    assert want[4] == []
    want_planes = [copied(p, want[3], page) for p in planes]
    ws = qb.pages_workspace(max(n_in, n_out), n_pages)
    t_out = torch.full((n_out, ld), 77, dtype=torch.int32, device=DEV)
    l_out, r_out = torch.full((n_out,), 77, dtype=torch.int32, device=DEV), torch.full((n_pages,), 77, dtype=torch.int32,
                                                                                      device=DEV)
    qb.qsa_fork_pages(page, ints(parent), ints(add), ints(table), ints(lens), ints(ref), t_out, l_out, r_out, planes, ws)
    assert np.array_equal(t_out.cpu().numpy(), want[0]) and np.array_equal(l_out.cpu().numpy(), want[1])
    assert np.array_equal(r_out.cpu().numpy(), want[2])
    assert all(torch.equal(a, b) for a, b in zip(planes, want_planes))
    assert status(ws) == (0, 0)


# ------------------------------------------------------------------------------------------ light tokens
@pytest.mark.parametrize("Hq,D", [(8, 256), (16, 256), (8, 128), (16, 128)])
@pytest.mark.parametrize("nats", [12.0, 15.0, 18.0, 22.0])
@pytest.mark.parametrize("n", [100, 20000])
def test_light_tokens_beside_a_heavy_one_over_fp8_rows(cuda_lib, Hq, D, nats, n):
    """One token `nats` above the others, whose V is zero in a quarter of the dims: there the others alone make the output.
    A weight x V scale is rounded to f16 relative to the largest, which is 2^15: half a step is 2^-11 of it, and below f16's
    normal range 2^-25, which is 2^-40 of the largest. The largest times 448 is at most the largest of `mass` in its 128
    dims, since every row has a code of 448 there, so n tokens add at most n 2^-40 of that."""
    q, planes, values, tab, table = paged_inputs([n], Hq, 1, D, 16, True, seed=81)
    g = torch.Generator().manual_seed(4)
    base = torch.randn(D, generator=g)
    q.copy_((base + 0.05 * torch.randn(1, Hq, D, generator=g)).to(torch.bfloat16))
    slot = P.slots_of(table[0], n, 16)[n // 2]
    heavy = base * (nats / (D ** -0.5 * float(base @ base)))
    scale = heavy.view(-1, 128).abs().amax(-1) / 448.0
    codes = (heavy.view(-1, 128) / scale[:, None]).to(torch.float8_e4m3fn)
    planes[0].flatten(0, 1)[slot, 0] = codes.view(torch.uint8).flatten().to(DEV)
    planes[1].flatten(0, 1)[slot, 0] = scale.to(DEV)
    values[0].reshape(-1, D)[slot] = (codes.float().double() * scale.double()[:, None]).flatten().numpy()
    planes[2].bitwise_and_(0x7F)                          # V is not negative: nothing cancels
    np.abs(values[1], out=values[1])
    planes[2].flatten(0, 1)[slot, 0].view(-1, 128)[:, :33] = torch.tensor([0] * 32 + [0x7E], dtype=torch.uint8, device=DEV)
    values[1].reshape(-1, D // 128, 128)[slot, :, :32] = 0
    values[1].reshape(-1, D // 128, 128)[slot, :, 32] = 448 * f64(planes[3].flatten(0, 1)[slot, 0])
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    out, lse = run_decode(cfg, q, planes, tab, ints([n]), ws)
    at = P.slots_of(table[0], n, 16)
    K, V = (x.reshape(-1, 1, D)[at] for x in values)
    want, want_lse, mass, terms = P.decode(f64(q[0]), K, V, 0, D ** -0.5)
    ds = D * 2.0 ** -24 * terms + 2.0 ** -21 * (terms + 1)
    if D == 256 and Hq <= 8:                              # queries as two E4M3 values: 2^-22 of the head's largest
        ds = ds + 2.0 ** -22 * np.abs(f64(q[0])).max(1) * np.abs(K).sum(2).max() * D ** -0.5
    sums = n / 8 * 2.0 ** -24 + 2.0 ** -15
    most = np.repeat(mass.reshape(Hq, -1, 128).max(-1), 128, -1)
    tol = 2.0 ** -8 * np.abs(want) + (2 * ds[:, None] + sums + 2.0 ** -11) * mass + n * 2.0 ** -40 * most
    assert np.all(np.abs(f64(out[0]) - want) <= tol), np.abs((f64(out[0]) - want) / tol).max()
    assert np.all(np.abs(f64(lse[0]) - want_lse) <= ds + sums + 2.0 ** -22 * np.abs(want_lse))
    assert status(ws) == (0, 0)


# ------------------------------------------------------------------------------------------ attention right behind the page calls
@pytest.mark.parametrize("rows,fp8", [(3, False), (40, False), (3, True)])
def test_attention_reads_what_a_fork_right_before_it_wrote(cuda_lib, rows, fp8):
    """Fork, then attention, many times without a wait in between: each call sees the lengths and pages of its own fork,
    which swaps rows of different lengths, and of the compaction behind it."""
    D, page = 128, 8
    cache = PagedCache(1, 40 * rows, page, rows, 30, 4, 1, D, fp8=fp8)
    lens = [5 + (37 * r) % 150 for r in range(rows)]
    cache.fork(ints([-1] * rows), ints(lens))
    rope = qb.rope_table(D)
    for r, n in enumerate(lens):
        x = randn((n, 2, D), seed=200 + r)
        cache.append(0, rope, None, x[:, :1], x[:, 1:], torch.arange(n, dtype=torch.int32, device=DEV),
                     torch.full((n,), r, dtype=torch.int32, device=DEV))
    q = randn((1, 4, D), seed=5).expand(rows, 4, D).contiguous()
    first = torch.empty_like(q)
    cache.attend(0, q, first)
    turn, none = ints([(r + 1) % rows for r in range(rows)]), ints([0] * rows)
    outs = [torch.empty_like(q) for _ in range(24)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        cache.fork(turn, none)
        if i % 5 == 4:
            cache.compact()
        cache.attend(0, q, out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, first.roll(-(i + 1), 0)), i
    assert cache.status() == ((0, 0), (0, 0))


# ------------------------------------------------------------------------------------------ infinite V
@pytest.mark.parametrize("Hq,D", [(8, 256), (16, 256), (7, 128), (16, 64), (8, 64)])
@pytest.mark.parametrize("n", [1, 70, 5000])
def test_decode_infinite_values_stay_infinite(cuda_lib, Hq, D, n):
    """V infinite in a dim: the output is that infinity there, and the same bits as before elsewhere; infinities of both
    signs, or a NaN, give NaN."""
    q, planes, values, tab, table = paged_inputs([n, 60], Hq, 1, D, 16, False, seed=83)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    want, want_lse = run_decode(cfg, q, planes, tab, ints([n, 60]), ws)
    logit = torch.from_numpy(values[0].reshape(-1, D)[P.slots_of(table[0], n, 16)]).float() @ q[0].float().cpu().T
    slots = P.slots_of(table[0], n, 16)
    heaviest, lightest = int(slots[int(logit[:, 0].argmax())]), int(slots[int(logit[:, 0].argmin())])
    flat = planes[1].flatten(0, 1)
    flat[heaviest, 0, 3], flat[lightest, 0, D - 2] = float("inf"), float("-inf")
    flat[int(slots[n // 2]), 0, 9] = float("nan")
    if n > 1:
        flat[int(slots[0]), 0, 20], flat[int(slots[n - 1]), 0, 20] = float("inf"), float("-inf")
    out, lse = run_decode(cfg, q, planes, tab, ints([n, 60]), ws)
    assert bool((out[0, :, 3] == float("inf")).all()) and bool((out[0, :, D - 2] == float("-inf")).all())
    assert bool(torch.isnan(out[0, :, 9]).all()) and (n == 1 or bool(torch.isnan(out[0, :, 20]).all()))
    keep = torch.ones(D, dtype=torch.bool, device=DEV)
    keep[[3, D - 2, 9, 20]] = False
    assert torch.equal(out[0][:, keep], want[0][:, keep]) and torch.equal(out[1], want[1]) and torch.equal(lse, want_lse)
    assert status(ws) == (0, 0)


# ------------------------------------------------------------------------------------------ NaN in an FP8 append
@pytest.mark.parametrize("D,rot", [(256, 0), (128, 0), (256, 256), (128, 64)])
def test_append_keeps_what_is_not_a_number(cuda_lib, D, rot):
    """A group of 128 dims that is NaN throughout, or NaN and zeros, is stored with NaN codes, not as zeros; beside other
    values a NaN spoils its own code alone (and its pair's, where K turns); attention over it is NaN."""
    cfg = qb.make_paged_config(2, 1, D, 4)
    ws, rope = qb.paged_workspace(cfg), qb.rope_table(D, rot)
    x = randn((4, 2, D), seed=85)
    x[0, :, :128] = float("nan")                          # a group
    x[1, :, :128], x[1, :, 5] = 0.0, float("nan")         # NaN among zeros
    x[2, :, 7] = float("nan")                             # NaN among others
    x[3, :, :128] = 0.0
    x[3, :, 1] = -0.0
    shape = (1, 4, 1, D)
    kv8 = [torch.full(shape, 17, dtype=torch.uint8, device=DEV), torch.full(shape[:3] + (D // 128,), 2.0, device=DEV),
           torch.full(shape, 18, dtype=torch.uint8, device=DEV), torch.full(shape[:3] + (D // 128,), 3.0, device=DEV)]
    qb.qsa_rope_append_fp8kv(cfg, rope, None, x[:, :1], x[:, 1:], ints([0, 1, 2, 3]), ints([0] * 4), None, kv8, ints([[0]]), ws)
    k, v = (torch.isnan(c[0, :, 0].view(torch.float8_e4m3fn).float()) for c in (kv8[0], kv8[2]))
    assert bool(v[0, :128].all()) and not v[0, 128:].any()
    assert v[1].nonzero().flatten().tolist() == [5] and v[2].nonzero().flatten().tolist() == [7] and not v[3].any()
    assert bool(k[0, :128].all())
    pair = lambda d: sorted({d, (d + rot // 2) % rot}) if rot and d < rot else [d]  # noqa: E731
    assert k[1].nonzero().flatten().tolist() == pair(5) and k[2].nonzero().flatten().tolist() == pair(7)
    assert not kv8[2][0, 3, 0, :128].any() and float(kv8[3][0, 3, 0, 0]) == 0.0        # zeros: zero codes, scale 0
    q = randn((1, 2, D), seed=86)
    out, _ = run_decode(cfg, q, kv8, ints([[0]]), ints([1]), ws)
    assert bool(torch.isnan(out).all())
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("Hq,D", [(8, 256), (16, 256), (8, 128), (16, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("n", [70, 3000])
def test_decode_value_scale_that_is_not_finite_spoils_its_dims_alone(cuda_lib, Hq, D, value, n):
    lens = [n, 50]
    q, planes, values, tab, table = paged_inputs(lens, Hq, 1, D, 16, True, seed=75)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    want, want_lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
    for group in range(D // 128):
        keep = planes[3].clone()
        planes[3][int(table[0][1]), 3, 0, group] = value   # token 19 of row 0
        out, lse = run_decode(cfg, q, planes, tab, ints(lens), ws)
        planes[3].copy_(keep)
        dims = torch.arange(D, device=DEV) // 128 == group
        assert bool(torch.isnan(out[0][:, dims]).all()) and torch.equal(out[1], want[1])
        # weights are relative to the largest, which this token's may have been: each side rounds them to f16 (2^-11 of a
        # sum of at most max |V|) and its result to bf16 (2^-8); the sums' fp32 rounding is far below
        a, b = f64(out[0][:, ~dims]), f64(want[0][:, ~dims])
        assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2.0 ** -10 * np.nanmax(np.abs(values[1])))
        assert np.abs(f64(lse) - f64(want_lse)).max() <= 2.0 ** -20 * (1 + np.abs(f64(want_lse)).max())
    assert status(ws) == (0, 0)


# ------------------------------------------------------------------------------------------ rows that nobody uses
@pytest.mark.parametrize("kind", ["none", "stream", "pointer", "zero"])
def test_extend_leaves_empty_rows_empty(cuda_lib, kind):
    own = torch.cuda.Stream()
    side = {"none": None, "stream": own, "pointer": own.cuda_stream, "zero": 0}[kind]
    cache = PagedCache(1, 12, 4, 5, 6, 4, 2, 64)
    cache.fork(ints([-1] * 5), ints([3, 0, 8, 1, 0]))
    cache.fork(ints([0, 1, 2, -1, 4]), ints([0] * 5))     # row 3 is given back
    torch.cuda.synchronize()
    for step in range(1, 10):
        cache.extend(stream=side)
        torch.cuda.synchronize()
        assert cache.seq_len.tolist() == [3 + step, 0, 8 + step, 0, 0]
    assert int((cache.ref > 0).sum()) == 3 + 5 and cache.status() == ((0, 0), (0, 0))
    assert cache.table[[1, 3, 4]].eq(-1).all()
    cache.extend(ints([0, 2, 0, 0, 1]))                   # by name: any row
    assert cache.seq_len.tolist() == [12, 2, 17, 0, 1]


def test_captured_extends_grow_the_rows_in_use(cuda_lib):
    cache = PagedCache(1, 20, 4, 3, 6, 4, 2, 64)
    cache.fork(ints([-1] * 3), ints([3, 0, 8]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cache.extend()
        cache.extend()
    for i in range(3):
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert cache.seq_len.tolist() == [5 + 2 * i, 0, 10 + 2 * i]
    assert cache.status() == ((0, 0), (0, 0))


@pytest.mark.parametrize("n_pages,ld", [(3000, 900), (8192, 1024), (8193, 1024)])
def test_fork_starts_long_rows_beside_short_ones(cuda_lib, n_pages, ld):
    """Prompts of hundreds of pages start in some rows while others go on, end, find no page or share a last page."""
    page, rng = 4, np.random.default_rng(n_pages)
    lens = np.array([9, 0, 31, 4, 700, 2, 12], np.int32)
    table, ref, at = np.full((7, ld), -1, np.int32), np.zeros(n_pages, np.int32), 0
    order = rng.permutation(n_pages)
    for r, n in enumerate(lens):
        c = -(-int(n) // page)
        table[r, :c] = order[at:at + c]
        ref[order[at:at + c]] = 1
        at += c
    parent = [-1, 0, 0, -1, 2, -1, 4, 5, 4, -1]
    add = [4 * 800 - 3, 1, 2500, 4 * 8, 0, 4 * 9 + 1, 300, 1, 0, 4 * (ld if n_pages == 3000 else 9)]
    if n_pages == 3000:
        parent, add = parent + [-1] * 3, add + [4 * 700] * 3     # the last finds too few pages
    want = P.fork(table, lens, ref, parent, add, page)
    assert (want[4] == []) == (n_pages != 3000)
    planes = planes_of(n_pages, page, 6)
    want_planes = [copied(p, want[3], page) for p in planes]
    ws = qb.pages_workspace(len(parent), n_pages)
    t_out = torch.full((len(parent), ld), 77, dtype=torch.int32, device=DEV)
    l_out, r_out = ints([77] * len(parent)), ints([77] * n_pages)
    qb.qsa_fork_pages(page, ints(parent), ints(add), ints(table), ints(lens), ints(ref), t_out, l_out, r_out, planes, ws)
    assert np.array_equal(t_out.cpu().numpy(), want[0]) and np.array_equal(l_out.cpu().numpy(), want[1])
    assert np.array_equal(r_out.cpu().numpy(), want[2])
    assert all(torch.equal(a, b) for a, b in zip(planes, want_planes))
    st, row = status(ws)
    assert (st, row) == (0, 0) if not want[4] else st == qb.QSA_ERR_DEVICE_BOUNDS and row in want[4]


@pytest.mark.parametrize("Hq,D", [(8, 256), (16, 256), (8, 128), (16, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 0.0, 2.0 ** -110])
@pytest.mark.parametrize("n,bad", [(1, 1), (70, 70), (400, 128), (400, 300), (3000, 2900)])
def test_decode_value_scales_of_whole_tiles_leave_the_rest(cuda_lib, Hq, D, value, n, bad):
    """The first `bad` tokens' V scales of a group are infinite, NaN, zero or tiny: the group's dims are NaN, or what the
    other tokens give; other dims and the log-sum-exp are as they would be."""
    q, planes, values, tab, table = paged_inputs([n], Hq, 1, D, 16, True, seed=76)
    cfg = qb.make_paged_config(Hq, 1, D, 16)
    ws = qb.paged_workspace(cfg)
    slots = P.slots_of(table[0], n, 16)
    keep = planes[3].clone()
    for group in range(D // 128):
        planes[3].copy_(keep).flatten(0, 1)[slots[:bad], 0, group] = value
        out, lse = run_decode(cfg, q, planes, tab, ints([n]), ws)
        small = value == value and value < 1
        dims = torch.arange(D, device=DEV) // 128 == group
        if small:
            V, of_group = values[1].copy(), slice(group * 128, group * 128 + 128)
            V.reshape(-1, 1, D)[slots[:bad], :, of_group] = value * e4m3(planes[2]).reshape(-1, 1, D)[slots[:bad], :, of_group]
            check_decode(out, lse, q, (values[0], V), table, [n], 16, 0, D ** -0.5, True,
                         q_step=2.0 ** -22 if D == 256 and Hq <= 8 else 0.0)
            continue
        assert bool(torch.isnan(out[0][:, dims]).all()) and not torch.isnan(out[0][:, ~dims]).any()
        got = torch.where(dims, 0.0, out.float()).to(torch.bfloat16)              # the NaN dims compared as zeros
        zeroed = values[1].copy()
        zeroed.reshape(-1, 1, D)[slots, :, group * 128:group * 128 + 128] = 0.0
        check_decode(got, lse, q, (values[0], zeroed), table, [n], 16, 0, D ** -0.5, True,
                     q_step=2.0 ** -22 if D == 256 and Hq <= 8 else 0.0)
    assert status(ws) == (0, 0)
