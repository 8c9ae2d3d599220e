"""Cases of the paged-cache operators: rotary positions, appending to a paged K/V cache, attention of
one new token over it, and forking and compacting its pages.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` their inputs on the GPU,
``run(state)`` one pass: elementary torch operations where ``own`` is false, the library's calls
where it is true. ``exact(case, seed)`` computes the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False
DEV = "cuda"
E4M3_MAX = 448.0


def listed():
    return [
        # The indexer queries of a decode batch of 32 (one 128-dim head each): the smallest call, one per layer.
        dict(name="rope_decode_index", op="rope", n=32, heads=1, dim=128, rot=128, begin=0, pairs="interleaved",
             scaling="none", first=65503),
        # The query heads of a prefill chunk behind 262,144 tokens; a quarter of each head turns, frequencies
        # rescaled by parts for contexts 8 times the trained one.
        dict(name="rope_prefill_query", op="rope", n=4096, heads=16, dim=256, rot=64, begin=0, pairs="half",
             scaling="by_parts", first=262144),
        # One decode step's new tokens of a batch of 32 (lengths up to 65,536 in service; the pages around the
        # new tokens suffice here): q turned, K turned and stored, V stored.
        dict(name="append_decode", op="append", n=32, rows=32, q_heads=16, kv_heads=2, dim=256, rot=256,
             pairs="half", scaling="none", page=64, pages=8, fp8=False),
        # A prefill chunk of 4,096 tokens of one sequence appended to an FP8 cache.
        dict(name="append_prefill_fp8", op="append", n=4096, rows=1, q_heads=16, kv_heads=2, dim=256, rot=128,
             pairs="half", scaling="linear", page=256, pages=24, fp8=True),
        # The tiny decode: one sequence of 4,096 tokens, 8 query heads; latency counts.
        dict(name="attend_short", op="attend", rows=1, low=4096, high=4096, q_heads=8, kv_heads=2, dim=256,
             page=64, window=0, fp8=False),
        # A ragged decode batch, lengths in [4096, 65536].
        dict(name="attend_ragged", op="attend", rows=32, low=4096, high=65536, q_heads=16, kv_heads=2, dim=256,
             page=64, window=0, fp8=False),
        # One sequence of a million tokens: the longest cache.
        dict(name="attend_million", op="attend", rows=1, low=1048321, high=1048321, q_heads=16, kv_heads=2,
             dim=256, page=256, window=0, fp8=False),
        # Many short and empty rows over FP8 rows with small pages that end inside any tile.
        dict(name="attend_many_fp8", op="attend", rows=128, low=0, high=5000, q_heads=32, kv_heads=8, dim=128,
             page=24, window=0, fp8=True),
        # Eight beams of one prompt after a step of beam search: one layer's K and V.
        dict(name="fork_beams", op="fork", rows=8, low=1000, high=1100, ld=24, page=64, layers=1, width=512,
             spare=64),
        # 64 requests of four beams each, every layer's K and V.
        dict(name="fork_batch", op="fork", rows=256, low=100, high=1000, ld=20, page=64, layers=12, width=512,
             spare=512),
        # A small pool, a few pages to move, one layer.
        dict(name="compact_small", op="compact", rows=16, low=1, high=600, ld=40, page=16, layers=1, width=512,
             spare=0),
        # A 12-layer pool of which close to half is free.
        dict(name="compact_pool", op="compact", rows=100, low=200, high=2000, ld=40, page=64, layers=12, width=512,
             spare=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "fork", "compact"])
    if op == "rope":
        dim, rot, begin = rng.choice([(128, 128, 0), (256, 64, 0), (256, 256, 0), (64, 64, 0), (576, 64, 512),
                                      (128, 96, 16), (256, 128, 128)])
        heads = rng.choice([1, 2, 7, 16, 64])
        n = min(_log(rng, 1, 8192), 16777216 // (heads * dim))
        return dict(op="rope", n=n, heads=heads, dim=dim, rot=rot, begin=begin, pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]), first=rng.randrange(3000000))
    if op == "append":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 8])
        rows = rng.choice([1, 1, 3, 32, 100])
        n = _log(rng, 1, 4096) if rows == 1 else rows
        page = rng.choice([4, 16, 24, 64, 256])
        return dict(op="append", n=n, rows=rows, q_heads=kv * rng.choice([1, 2, 7, 8]), kv_heads=kv, dim=dim,
                    rot=rng.choice([32, 64, dim]), pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "ntk", "by_parts"]), page=page, pages=n // page + 3,
                    fp8=dim >= 128 and rng.random() < 0.5)
    if op == "attend":
        fp8 = rng.random() < 0.5
        dim = rng.choice([128, 256] if fp8 else [64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        rows = _log(rng, 1, 256)
        high = max(1, min(_log(rng, 1, 500000), (1 << 29) // (rows * kv * dim)))
        return dict(op="attend", rows=rows, low=rng.choice([0, high // 16, high]), high=high,
                    q_heads=kv * rng.choice([1, 2, 3, 4, 8, 12, 16]), kv_heads=kv, dim=dim,
                    page=rng.choice([1, 4, 16, 24, 64, 100, 256]), window=rng.choice([0, 0, 0, 1 + high // 3]),
                    fp8=fp8)
    rows = _log(rng, 1, 200)
    page = rng.choice([4, 16, 24, 64])
    high = _log(rng, page, 1200)
    return dict(op=op, rows=rows, low=rng.choice([0, high // 2]), high=high, ld=high // page + 4, page=page,
                layers=rng.choice([1, 2, 5, 12]), width=rng.choice([64, 128, 512]), spare=3 * rows + _log(rng, 1, 500))


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _quantised(shape, g):
    """FP8 rows of N(0, 1) values: E4M3 codes and an fp32 scale for each 128 dims."""
    x = torch.randn(shape, generator=g, device=DEV).reshape(*shape[:-1], shape[-1] // 128, 128)
    scale = x.abs().amax(-1) / E4M3_MAX
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape)
    return codes, scale


ROPE_BASE, ROPE_FACTOR, ROPE_TRAINED = 1e6, 8.0, 32768
BETA_FAST, BETA_SLOW = 32.0, 1.0


def _rope_kw(c):
    return dict(head_dim=c["dim"], rot_dim=c["rot"], rot_begin=c.get("begin", 0), interleaved=c["pairs"] == "interleaved",
                base=ROPE_BASE, scaling=c["scaling"], factor=ROPE_FACTOR, original_len=ROPE_TRAINED,
                beta_fast=BETA_FAST, beta_slow=BETA_SLOW)


def _frequencies(c):
    """Radians per token of each pair, and the factor on cos and sin, in 64 bits."""
    half = c["rot"] // 2
    i = np.arange(half, dtype=np.float64)
    plain = ROPE_BASE ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return plain / ROPE_FACTOR, 1.0
    if c["scaling"] == "ntk":
        base = ROPE_BASE * ROPE_FACTOR ** (c["rot"] / (c["rot"] - 2.0))
        return base ** (-2.0 * i / c["rot"]), 1.0
    if c["scaling"] == "by_parts":
        # pairs that turn more than BETA_FAST times over the trained length keep their frequency, those that
        # turn less than BETA_SLOW times are slowed by the factor, and a ramp in the pair's index joins them
        at = [half * math.log(ROPE_TRAINED / (b * 2.0 * math.pi)) / math.log(ROPE_BASE) for b in (BETA_FAST, BETA_SLOW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), half - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return plain * (1.0 - ramp) + plain / ROPE_FACTOR * ramp, 0.1 * math.log(ROPE_FACTOR) + 1.0
    return plain, 1.0


def _pool_pages(c):
    return c["rows"] * -(-c["high"] // c["page"]) + c["spare"]


def _prepare_table(c, g):
    """A pool's page table: rows of lengths in [low, high] over pages in random order; the last rows share
    their first pages with row 0 (a common prompt)."""
    S, ps = c["rows"], c["page"]
    length = torch.randint(c["low"], c["high"] + 1, (S,), generator=g, device=DEV)
    count = (length + ps - 1) // ps
    n_pages = _pool_pages(c)
    order = torch.randperm(n_pages, generator=g, device=DEV)
    j = torch.arange(c["ld"], device=DEV)
    start = torch.cumsum(count, 0) - count
    used = j[None, :] < count[:, None]
    table = torch.where(used, order[(start[:, None] + j).clamp(max=n_pages - 1)], -1)
    if S > 2:  # share the full pages that both rows have
        shared = torch.minimum(length[0], length[S - 2:].min()) // ps // 2
        table[S - 2:] = torch.where(j[None, :] < shared, table[:1], table[S - 2:])
    ref = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
    ref.scatter_add_(0, table.clamp(min=0).reshape(-1), used.reshape(-1).long())
    return table.int(), length.int(), ref.int(), n_pages


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "rope":
        s["x"] = _randn((c["n"], c["heads"], c["dim"]), g)
        s["pos"] = c["first"] + torch.arange(c["n"], device=DEV, dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
        s["freq"], s["amp"] = torch.from_numpy(_frequencies(c)[0]).to(DEV), _frequencies(c)[1]
    elif c["op"] == "append":
        N, Hq, Hkv, D, ps = c["n"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = _randn((N, Hq + 2 * Hkv, D), g)               # one projection's rows: q, k and v side by side
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        n_pages = c["rows"] * c["pages"]
        s["table"] = torch.randperm(n_pages, generator=g, device=DEV).int().reshape(c["rows"], c["pages"])
        room = c["pages"] * ps
        if c["rows"] == 1:
            s["seq"] = torch.zeros(N, dtype=torch.int32, device=DEV)
            s["pos"] = torch.arange(N, device=DEV, dtype=torch.int32) + min(ps // 2 + 1, room - N)
        else:
            s["seq"] = torch.arange(N, device=DEV, dtype=torch.int32)
            s["pos"] = torch.randint(0, room, (N,), generator=g, device=DEV, dtype=torch.int32)
        s["q_out"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device=DEV)
        shape = (n_pages, ps, Hkv, D)
        if c["fp8"]:
            s["kv8"] = _quantised(shape, g) + _quantised(shape, g)
        else:
            s["k_cache"], s["v_cache"] = _randn(shape, g), _randn(shape, g)
        s["freq"], s["amp"] = torch.from_numpy(_frequencies(c)[0]).to(DEV), _frequencies(c)[1]
    elif c["op"] == "attend":
        B, Hq, Hkv, D, ps = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        length = torch.randint(c["low"], c["high"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        ld = (c["high"] + ps - 1) // ps
        count = (length + ps - 1) // ps
        n_pages = int(count.sum()) + 1
        order = torch.randperm(n_pages, generator=g, device=DEV).int()
        j = torch.arange(ld, device=DEV)
        at = (torch.cumsum(count, 0) - count)[:, None] + j
        s["table"] = torch.where(j < count[:, None], order[at.clamp(max=n_pages - 1)], -1)
        s["seq_len"] = length
        s["q"] = _randn((B, Hq, D), g)
        shape = (n_pages, ps, Hkv, D)
        if c["fp8"]:
            s["kv8"] = _quantised(shape, g) + _quantised(shape, g)
        else:
            s["k_cache"], s["v_cache"] = _randn(shape, g), _randn(shape, g)
        s["out"] = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device=DEV)
    else:
        s["table"], s["seq_len"], s["ref"], n_pages = _prepare_table(c, g)
        s["pool"] = _randn((2 * c["layers"], n_pages, c["page"], c["width"]), g)
        s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
        if c["op"] == "fork":
            # a step of beam search: each row continues one of its group's four rows and gets a token or two;
            # a group in sixteen has ended and gives its pages back
            i = torch.arange(c["rows"], device=DEV)
            parent = (i // 4 * 4 + torch.randint(0, 4, (c["rows"],), generator=g, device=DEV)).clamp(max=c["rows"] - 1)
            s["parent"] = torch.where(i // 4 % 16 == 15, -1, parent).int()
            s["add"] = torch.where(s["parent"] >= 0, torch.randint(1, 3, (c["rows"],), generator=g, device=DEV), 0).int()
            s["len_out"] = torch.empty_like(s["seq_len"])
    if own:
        from indexer_driven_sparse_gb300 import binding as qb
        if c["op"] in ("rope", "append"):
            s["rope"] = qb.rope_table(device=DEV, **_rope_kw(c))
        if c["op"] in ("append", "attend"):
            s["cfg"] = qb.make_paged_config(c["q_heads"], c["kv_heads"], c["dim"], c["page"], window=c.get("window", 0))
            s["ws"] = qb.paged_workspace(s["cfg"], device=DEV)
        if c["op"] in ("fork", "compact"):
            s["ws"] = qb.pages_workspace(c["rows"], n_pages, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ one pass
def _turn(x, pos, freq, amp, rot, begin, pairs):
    """x [N, H, D] -> fp32 with dims [begin, begin + rot) turned by pos x freq; angles in 64 bits."""
    angle = pos.double()[:, None] * freq
    cos, sin = (angle.cos() * amp).float()[:, None], (angle.sin() * amp).float()[:, None]
    y = x.float()
    part = y[..., begin:begin + rot]
    if pairs == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y[..., :begin], turned, y[..., begin + rot:]], -1)


def _to_fp8(x):
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 128, 128)
    scale = y.abs().amax(-1) / E4M3_MAX
    codes = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).reshape(x.shape), scale


def _rows_fp32(s, name, slots):
    """K or V rows of `slots` as fp32."""
    c = s["case"]
    if not c["fp8"]:
        return s[name + "_cache"].flatten(0, 1)[slots].float()
    codes, scales = s["kv8"][:2] if name == "k" else s["kv8"][2:]
    values = codes.flatten(0, 1)[slots].view(torch.float8_e4m3fn).float()
    return values * scales.flatten(0, 1)[slots].repeat_interleave(128, -1)


def _plain_append(s):
    c = s["case"]
    ps = c["page"]
    s["q_out"].copy_(_turn(s["q"], s["pos"], s["freq"], s["amp"], c["rot"], 0, c["pairs"]).to(torch.bfloat16))
    k = _turn(s["k"], s["pos"], s["freq"], s["amp"], c["rot"], 0, c["pairs"])
    pos = s["pos"].long()
    slot = s["table"][s["seq"].long(), pos // ps].long() * ps + pos % ps
    if not c["fp8"]:
        s["k_cache"].flatten(0, 1)[slot] = k.to(torch.bfloat16)
        s["v_cache"].flatten(0, 1)[slot] = s["v"]
        return
    kc, ks = _to_fp8(k)
    vc, vs = _to_fp8(s["v"].float())
    k_codes, k_scales, v_codes, v_scales = (plane.flatten(0, 1) for plane in s["kv8"])
    k_codes[slot], k_scales[slot], v_codes[slot], v_scales[slot] = kc, ks, vc, vs


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D, ps = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    j = torch.arange(s["table"].shape[1] * ps, device=DEV)
    length = s["seq_len"][:, None]
    seen = j < length
    if c["window"]:
        seen = seen & (j >= length - c["window"])
    slots = s["table"].long().clamp(min=0)[:, j // ps] * ps + j % ps
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    logit = torch.matmul(q, _rows_fp32(s, "k", slots).permute(0, 2, 3, 1)) / math.sqrt(D)
    logit = torch.where(seen[:, None, None], logit, -torch.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = torch.exp(logit - top)
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight, _rows_fp32(s, "v", slots).permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    s["out"].copy_(out.reshape(B, Hq, D))
    s["lse"].copy_((top + torch.log(total)).reshape(B, Hq))


def _free_first(ref):
    """Page ids with the free ones first, both parts ascending."""
    return torch.argsort((ref != 0).int(), stable=True)


def _plain_fork(s):
    c = s["case"]
    ps, S = c["page"], c["rows"]
    table, length, ref = s["table"].long(), s["seq_len"].long(), s["ref"].long()
    row = torch.arange(S, device=DEV)
    j = torch.arange(c["ld"], device=DEV)
    goes_on, parent = s["parent"] >= 0, s["parent"].long().clamp(min=0)
    base = torch.where(goes_on, length[parent], 0)
    total = base + s["add"]
    full, used = base // ps, base % ps
    first = torch.full((S,), S, device=DEV).scatter_reduce(0, parent, torch.where(goes_on, row, S), "amin")
    partial = table[parent, full.clamp(max=c["ld"] - 1)]
    keeps = (used > 0) & (first[parent] == row) & (ref[partial.clamp(min=0)] == 1)
    copies = (used > 0) & ~keeps
    kept = full + keeps.long()
    pages = (total + ps - 1) // ps
    start = torch.cumsum(pages - kept, 0) - (pages - kept)
    fresh = _free_first(ref)
    new = fresh[(start[:, None] + j - kept[:, None]).clamp(0, ref.numel() - 1)]
    table_out = torch.where(j < kept[:, None], table[parent], torch.where(j < pages[:, None], new, -1))
    count = (length + ps - 1) // ps
    ref_out = ref.scatter_add(0, table.clamp(min=0).reshape(-1), -(j < count[:, None]).reshape(-1).long())
    ref_out.scatter_add_(0, table_out.clamp(min=0).reshape(-1), (j < pages[:, None]).reshape(-1).long())
    at = torch.nonzero(copies).squeeze(1)
    src, dst = partial[at], table_out[at, full[at]]
    part = (torch.arange(ps, device=DEV) < used[at][:, None])[None, :, :, None]
    s["pool"][:, dst] = torch.where(part, s["pool"][:, src], s["pool"][:, dst])
    s["table_out"].copy_(table_out)
    s["len_out"].copy_(total)
    s["ref_out"].copy_(ref_out)


def _plain_compact(s):
    c = s["case"]
    table, ref = s["table"].long(), s["ref"]
    page = torch.arange(ref.numel(), device=DEV)
    live = ref > 0
    n_live = live.sum()
    moves, holes = live & (page >= n_live), ~live & (page < n_live)
    src, dst = torch.nonzero(moves).squeeze(1), torch.nonzero(holes).squeeze(1)
    goes_to = page.index_put((src,), dst)
    s["pool"][:, dst] = s["pool"][:, src]
    s["table_out"].copy_(torch.where(table >= 0, goes_to[table.clamp(min=0)], -1))
    s["ref_out"].copy_(torch.where(page < n_live, ref, 0).index_put((dst,), ref[src]))


def run(state):
    s = state
    c = s["case"]
    if own:
        from indexer_driven_sparse_gb300 import binding as qb
    if c["op"] == "rope":
        if own:
            qb.qsa_rope(s["rope"], s["x"], s["pos"], s["out"])
        else:
            s["out"].copy_(_turn(s["x"], s["pos"], s["freq"], s["amp"], c["rot"], c["begin"], c["pairs"]))
        return {"out": s["out"]}
    if c["op"] == "append":
        if not own:
            _plain_append(s)
        elif c["fp8"]:
            qb.qsa_rope_append_fp8kv(s["cfg"], s["rope"], s["q"], s["k"], s["v"], s["pos"], s["seq"], s["q_out"],
                                     s["kv8"], s["table"], s["ws"])
        else:
            qb.qsa_rope_append(s["cfg"], s["rope"], s["q"], s["k"], s["v"], s["pos"], s["seq"], s["q_out"],
                               s["k_cache"], s["v_cache"], s["table"], s["ws"])
        if c["fp8"]:
            kc, ks, vc, vs = s["kv8"]
            return {"q": s["q_out"], "k": kc.view(torch.float8_e4m3fn), "k_scales": ks,
                    "v": vc.view(torch.float8_e4m3fn), "v_scales": vs}
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "attend":
        if not own:
            _plain_attend(s)
        elif c["fp8"]:
            qb.qsa_paged_decode_fp8kv(s["cfg"], s["q"], s["kv8"], s["table"], s["seq_len"], s["out"], s["lse"], s["ws"])
        else:
            qb.qsa_paged_decode(s["cfg"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_len"], s["out"],
                                s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "fork":
        if own:
            qb.qsa_fork_pages(c["page"], s["parent"], s["add"], s["table"], s["seq_len"], s["ref"], s["table_out"],
                              s["len_out"], s["ref_out"], [s["pool"]], s["ws"])
        else:
            _plain_fork(s)
        return {"table": s["table_out"], "seq_len": s["len_out"], "ref": s["ref_out"], "pool": s["pool"]}
    if own:
        qb.qsa_compact_pages(c["page"], s["table"], s["seq_len"], s["ref"], s["table_out"], s["ref_out"], [s["pool"]],
                             s["ws"])
    else:
        _plain_compact(s)
    return {"table": s["table_out"], "ref": s["ref_out"], "pool": s["pool"]}


# ------------------------------------------------------------------------------------------ work
def work(case):
    """Bytes and operations of one pass, each input read once and each output written once. Lengths are drawn
    uniformly in [low, high]: their mean stands for them."""
    c = case
    if c["op"] == "rope":
        return {"bytes": c["n"] * (4 * c["heads"] * c["dim"] + 4), "flops": 3 * c["n"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        D, Hq, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
        row = D + D // 128 * 4 if c["fp8"] else 2 * D
        return {"bytes": c["n"] * (4 * D * Hq + 2 * Hkv * (2 * D + row) + 8),
                "flops": 3 * c["n"] * (Hq + Hkv) * c["rot"]}
    mean = (c["low"] + c["high"]) / 2
    if c["op"] == "attend":
        if c["window"]:
            mean = min(mean, c["window"])
        D, Hq, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
        row = D + D // 128 * 4 if c["fp8"] else 2 * D
        tokens = c["rows"] * mean
        return {"bytes": tokens * 2 * Hkv * row + c["rows"] * (4 * Hq * D + 4 * Hq) + tokens / c["page"] * 4,
                "flops": 4 * tokens * Hq * D}
    plane = 2 * c["layers"] * c["width"] * 2                # bytes of one token in every plane
    pages = c["rows"] * (mean / c["page"] + 0.5)
    tables = 8 * c["rows"] * c["ld"] + 8 * _pool_pages(c)
    if c["op"] == "fork":                                   # about a third of the rows copy half a page
        return {"bytes": tables + c["rows"] / 3 * c["page"] / 2 * plane * 2, "flops": 0}
    moved = pages * max(0.0, 1 - pages / _pool_pages(c))
    return {"bytes": tables + moved * c["page"] * plane * 2, "flops": 0}


# ------------------------------------------------------------------------------------------ 64 bits
def _exact_turn(x, pos, c):
    freq, amp = _frequencies(c)
    begin, rot = c.get("begin", 0), c["rot"]
    angle = pos.double()[:, None] * torch.from_numpy(freq).to(DEV)
    y = x.double().clone()
    for i in range(rot // 2):
        a, b = (begin + i, begin + i + rot // 2) if c["pairs"] == "half" else (begin + 2 * i, begin + 2 * i + 1)
        co, si = torch.cos(angle[:, i:i + 1]) * amp, torch.sin(angle[:, i:i + 1]) * amp
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * co - w * si, w * co + u * si
    return y


def _exact_fp8(x):
    y = x.reshape(*x.shape[:-1], -1, 128)
    scale = y.abs().amax(-1) / E4M3_MAX
    return (y / scale[..., None]).reshape(x.shape), scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    ps = c.get("page", 1)
    if c["op"] == "rope":
        return {"out": _exact_turn(s["x"], s["pos"], c)}
    if c["op"] == "append":
        q, k, v = _exact_turn(s["q"], s["pos"], c), _exact_turn(s["k"], s["pos"], c), s["v"].double()
        if c["fp8"]:
            planes = [p.view(torch.float8_e4m3fn).double() if p.dtype == torch.uint8 else p.double() for p in s["kv8"]]
            new = _exact_fp8(k) + _exact_fp8(v)
        else:
            planes, new = [s["k_cache"].double(), s["v_cache"].double()], (k, v)
        table, pos = s["table"].tolist(), s["pos"].tolist()
        for i, r in enumerate(s["seq"].tolist()):
            page, at = table[r][pos[i] // ps], pos[i] % ps
            for plane, rows in zip(planes, new):
                plane[page, at] = rows[i]
        names = ("k", "k_scales", "v", "v_scales") if c["fp8"] else ("k", "v")
        return {"q": q, **dict(zip(names, planes))}
    if c["op"] == "attend":
        Hkv, G, D = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
        out = torch.zeros(c["rows"], c["q_heads"], D, dtype=torch.float64, device=DEV)
        lse = torch.full((c["rows"], c["q_heads"]), -torch.inf, dtype=torch.float64, device=DEV)
        for r, n in enumerate(s["seq_len"].tolist()):
            lo = max(0, n - c["window"]) if c["window"] else 0
            if n == 0:
                continue
            pages = s["table"][r, lo // ps:(n + ps - 1) // ps].long()
            cut = slice(lo - lo // ps * ps, n - lo // ps * ps)

            def rows64(name):
                if not c["fp8"]:
                    return s[name + "_cache"][pages].flatten(0, 1)[cut].double()
                codes, scales = s["kv8"][:2] if name == "k" else s["kv8"][2:]
                y = codes[pages].flatten(0, 1)[cut].view(torch.float8_e4m3fn).double()
                z = scales[pages].flatten(0, 1)[cut].double()
                return (y.reshape(*z.shape, 128) * z[..., None]).reshape(y.shape)

            K, V = rows64("k"), rows64("v")
            for h in range(Hkv):
                t = s["q"][r, h * G:(h + 1) * G].double() @ K[:, h].T * D ** -0.5
                l = torch.logsumexp(t, 1)
                lse[r, h * G:(h + 1) * G] = l
                out[r, h * G:(h + 1) * G] = torch.exp(t - l[:, None]) @ V[:, h]
        return {"out": out, "lse": lse}
    # pages: whole numbers by hand on the host, pages' contents as they were copied
    table, ref, pool = s["table"].tolist(), s["ref"].tolist(), s["pool"].clone()
    length = s["seq_len"].tolist()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if c["op"] == "compact":
        live = [p for p in range(len(ref)) if ref[p]]
        free = [p for p in range(len(live)) if not ref[p]]
        to, new_ref = {}, ref[:len(live)] + [0] * (len(ref) - len(live))
        for p in live:
            if p >= len(live):
                to[p] = free[len(to)]
                new_ref[to[p]] = ref[p]
        if to:
            pool[:, list(to.values())] = s["pool"][:, list(to)]
        return {"table": ints([[to.get(p, p) for p in r] for r in table]), "ref": ints(new_ref), "pool": pool}
    free = iter([p for p in range(len(ref)) if not ref[p]])
    new_table, new_len, seen = [], [], set()
    for p, more in zip(s["parent"].tolist(), s["add"].tolist()):
        n, pages = (length[p], table[p][:(length[p] + ps - 1) // ps]) if p >= 0 else (0, [])
        if n % ps and (p in seen or ref[pages[-1]] != 1):
            old, pages = pages[-1], pages[:-1] + [next(free)]
            pool[:, pages[-1], :n % ps] = s["pool"][:, old, :n % ps]
        seen.add(p)
        while len(pages) * ps < n + more:
            pages = pages + [next(free)]
        new_table.append(pages + [-1] * (c["ld"] - len(pages)))
        new_len.append(n + more)
    new_ref = list(ref)
    for rows, sign, lens in ((table, -1, length), (new_table, 1, new_len)):
        for r, n in zip(rows, lens):
            for p in r[:(n + ps - 1) // ps]:
                new_ref[p] += sign
    return {"table": ints(new_table), "seq_len": ints(new_len), "ref": ints(new_ref), "pool": pool}
