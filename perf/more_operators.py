"""Cases of the paged cache's operators for drafted tokens and for eviction: attention of a tree of drafted tokens,
keeping the accepted ones, attention that accumulates each cached token's weight, and evicting the lightest tokens.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` their inputs on the GPU,
``run(state)`` one pass: elementary torch operations where ``own`` is false, the library's calls
where it is true. ``exact(case, seed)`` computes the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False
DEV = "cuda"
E4M3_MAX = 448.0


def listed():
    return [
        # The tiny verification: a chain of four drafted tokens of one sequence of 4,096, 8 query heads; latency counts.
        dict(name="tree_chain", op="tree", rows=1, low=4096, high=4096, drafts_low=4, drafts=4, q_heads=8, kv_heads=2,
             dim=256, page=64, window=0, fp8=False),
        # A ragged batch, lengths in [4096, 65536], sixteen drafted tokens each.
        dict(name="tree_batch", op="tree", rows=32, low=4096, high=65536, drafts_low=16, drafts=16, q_heads=16,
             kv_heads=2, dim=256, page=64, window=0, fp8=False),
        # Wide trees of 64 tokens: every cached row serves 512 query rows, so the products count.
        dict(name="tree_wide", op="tree", rows=8, low=16384, high=65536, drafts_low=64, drafts=64, q_heads=16,
             kv_heads=2, dim=256, page=64, window=0, fp8=False),
        # Many short and empty rows over FP8 rows with small pages, up to 24 drafted tokens each, some none.
        dict(name="tree_many_fp8", op="tree", rows=64, low=64, high=5000, drafts_low=0, drafts=24, q_heads=32,
             kv_heads=8, dim=128, page=24, window=0, fp8=True),
        # Long FP8 histories, 16 drafted tokens.
        dict(name="tree_long_fp8", op="tree", rows=4, low=100000, high=262144, drafts_low=16, drafts=16, q_heads=16,
             kv_heads=2, dim=256, page=256, window=0, fp8=True),
        # After the verification of 8 rows: one layer's K and V, up to 8 drafted tokens.
        dict(name="accept_few", op="accept", rows=8, low=1000, high=1100, drafts_low=8, drafts=8, page=64, layers=1,
             width=512, fp8=False),
        # 128 rows, up to 32 drafted tokens, every layer's K and V.
        dict(name="accept_batch", op="accept", rows=128, low=100, high=400, drafts_low=4, drafts=32, page=16, layers=12,
             width=512, fp8=False),
        # One sequence of 4,096 tokens whose weights are accumulated; latency counts.
        dict(name="weights_short", op="weights", rows=1, low=4096, high=4096, q_heads=8, kv_heads=2, dim=256, page=64,
             window=0, fp8=False),
        # A ragged decode batch.
        dict(name="weights_ragged", op="weights", rows=32, low=4096, high=32768, q_heads=16, kv_heads=2, dim=256, page=64,
             window=0, fp8=False),
        # Many short and empty rows over FP8 rows.
        dict(name="weights_many_fp8", op="weights", rows=128, low=0, high=5000, q_heads=32, kv_heads=8, dim=128,
             page=24, window=0, fp8=True),
        # A decode batch over its budget by up to a page each: few rows of each cache move.
        dict(name="evict_step", op="evict", rows=32, low=4000, high=4160, budget=4096, first=4, recent=256, page=64,
             layers=4, width=512, shared=0, fp8=False),
        # Prompts of 16 sequences cut down to an eighth.
        dict(name="evict_prompt", op="evict", rows=16, low=12000, high=16384, budget=2048, first=16, recent=512,
             page=64, layers=2, width=512, shared=2, fp8=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "weights", "evict"])
    page = rng.choice([1, 4, 16, 24, 64, 100, 256])
    if op in ("tree", "weights"):
        fp8 = rng.random() < 0.5
        dim = rng.choice([128, 256] if fp8 else [64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8, 12, 16])
        c = dict(op=op, rows=_log(rng, 1, 128), q_heads=heads, kv_heads=kv, dim=dim, page=page, fp8=fp8)
        drafts = 1
        if op == "tree":
            drafts = _log(rng, 1, 128)
            c.update(drafts=drafts, drafts_low=rng.choice([0, drafts, drafts]))
        # at most the cache of the largest listed case of its kind, and the tree's products
        most = min((1 << 28) // (c["rows"] * kv * dim), (1 << 32) // (c["rows"] * drafts * heads * max(dim, 128) // 16))
        high = max(drafts + 1, min(_log(rng, 1, 300000), most))
        c.update(low=max(drafts if op == "tree" else 0, rng.choice([0, high // 16, high])), high=high,
                 window=rng.choice([0, 0, 0, 1 + high // 3]))
        return c
    rows, fp8 = _log(rng, 1, 128), rng.random() < 0.3
    page = rng.choice([4, 16, 24, 64])
    width, layers = rng.choice([128, 256, 512]), rng.choice([1, 2, 5])
    if op == "accept":
        drafts = _log(rng, 1, 128)
        high = drafts + _log(rng, 1, 500)
        return dict(op="accept", rows=rows, low=drafts, high=high, drafts_low=rng.choice([0, 1, drafts]), drafts=drafts,
                    page=page, layers=layers, width=width, fp8=fp8)
    high = min(_log(rng, 20, 16384), (1 << 28) // (rows * layers * width))
    budget = max(1, int(high * rng.uniform(0.05, 1.0)))
    return dict(op="evict", rows=rows, low=rng.choice([0, high // 2, high]), high=high, budget=budget,
                first=rng.choice([0, 1, 4, 64]), recent=rng.choice([0, 1, budget // 8, budget // 2]), page=page,
                layers=layers, width=width, shared=rng.choice([0, 0, 1]), fp8=fp8)


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=g)


def _quantised(shape, g):
    """FP8 rows of N(0, 1) values: E4M3 codes and an fp32 scale for each 128 dims."""
    x = torch.randn(shape, generator=g, device=DEV).reshape(*shape[:-1], shape[-1] // 128, 128)
    scale = x.abs().amax(-1) / E4M3_MAX
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape)
    return codes, scale


def _ints(c, low, high, g):
    return torch.randint(c[low], c[high] + 1, (c["rows"],), generator=g, device=DEV, dtype=torch.int32)


def _drafts(c, length, g):
    """Where each row's drafted tokens begin in the batch's list, which has room for the most there may be, and every
    token's parent: a chain with one branch in four, -1 for a child of the cached tokens."""
    count = torch.minimum(_ints(c, "drafts_low", "drafts", g), length)
    off = torch.zeros(c["rows"] + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(count, 0)
    n = c["rows"] * c["drafts"]
    index = torch.arange(n, device=DEV)
    index = index - off.long()[torch.searchsorted(off[1:].long(), index, right=True).clamp(max=c["rows"] - 1)]
    branch = (torch.rand(n, generator=g, device=DEV) * (index + 1)).long() - 1
    chain = torch.rand(n, generator=g, device=DEV) < 0.75
    return off, torch.where(chain, index - 1, branch).int()


def _table(c, length, g):
    ps = c["page"]
    ld = (c["high"] + ps - 1) // ps
    count = (length + ps - 1) // ps
    n_pages = c["rows"] * ld + 1 if c["op"] in ("accept", "evict") else int(count.sum()) + 1
    order = torch.randperm(n_pages, generator=g, device=DEV).int()
    j = torch.arange(ld, device=DEV)
    at = (torch.cumsum(count, 0) - count)[:, None] + j
    used = j < count[:, None]
    return torch.where(used, order[at.clamp(max=n_pages - 1)], -1), used, n_pages


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    s["seq_len"] = length = _ints(c, "low", "high", g)
    s["table"], used, n_pages = _table(c, length, g)
    ps, rows = c["page"], c["rows"]
    if c["op"] in ("tree", "accept"):
        s["off"], s["parent"] = _drafts(c, length, g)
    if c["op"] in ("tree", "weights"):
        Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["dim"]
        n = rows * c["drafts"] if c["op"] == "tree" else rows
        s["q"] = _randn((n, Hq, D), g)
        shape = (n_pages, ps, Hkv, D)
        s["kv"] = _quantised(shape, g) + _quantised(shape, g) if c["fp8"] else (_randn(shape, g), _randn(shape, g))
        s["out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(n, Hq, dtype=torch.float32, device=DEV)
        if c["op"] == "weights":               # what earlier steps accumulated
            s["weights"] = torch.rand((rows, s["table"].shape[1] * ps), generator=g, device=DEV)
            s["weights"] *= torch.arange(s["weights"].shape[1], device=DEV) < length[:, None]
    else:
        shape = (2 * c["layers"], n_pages, ps, c["width"])
        s["pool"] = list(_quantised(shape, g)) if c["fp8"] else [_randn(shape, g)]
        if c["op"] == "accept":                # the deepest accepted token of each row, -1: none
            count = s["off"][1:] - s["off"][:-1]
            s["last"] = ((torch.rand(rows, generator=g, device=DEV) * (count + 1)).int() - 1).clamp(max=count - 1)
        else:
            # the last rows share row 0's first pages (a common prompt)
            if c["shared"] and rows > 2:
                k = torch.minimum(length[0], length[rows - 2:].min()) // ps
                k = torch.clamp(k, max=c["shared"])
                j = torch.arange(s["table"].shape[1], device=DEV)
                s["table"][rows - 2:] = torch.where(j < k, s["table"][:1], s["table"][rows - 2:])
            # weights: heavy-tailed, a tenth of them zero; positions: out of order up to the budget, as earlier
            # evictions left them, in order behind it
            room = s["table"].shape[1] * ps
            w = torch.exp(2 * torch.randn((rows, room), generator=g, device=DEV))
            w = torch.where(torch.rand((rows, room), generator=g, device=DEV) < 0.1, 0.0, w)
            j = torch.arange(room, device=DEV)
            old = 2 * torch.argsort(torch.rand((rows, min(c["budget"], room)), generator=g, device=DEV), dim=1)
            pos = torch.where(j < c["budget"], 0, c["budget"] + j)[None].repeat(rows, 1)
            pos[:, :old.shape[1]] = old
            held = j < length[:, None]
            s["weights"], s["positions"] = torch.where(held, w, 0.0), torch.where(held, pos, -1).int()
            s["weights_out"], s["positions_out"] = torch.empty_like(s["weights"]), torch.empty_like(s["positions"])
            s["budget"] = torch.full((rows,), c["budget"], dtype=torch.int32, device=DEV)
        ref = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
        ref.scatter_add_(0, s["table"].long().clamp(min=0).reshape(-1), used.reshape(-1).long())
        s["ref"] = ref.int()
        s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
        s["len_out"] = torch.empty_like(length)
    if own:
        from indexer_driven_sparse_gb300 import binding as qb
        if c["op"] in ("tree", "weights"):
            s["cfg"] = qb.make_paged_config(c["q_heads"], c["kv_heads"], c["dim"], ps, window=c["window"])
            if c["op"] == "tree":
                s["ws"] = qb.tree_workspace(s["cfg"], c["drafts"], device=DEV)
            else:
                s["ws"] = qb.weights_workspace(s["cfg"], rows, int(length.sum()), device=DEV)
        else:
            s["ws"] = qb.keep_workspace(rows, s["table"].shape[1] * ps if c["op"] == "evict" else 0, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ one pass
def _rows_fp32(s, which, slots):
    """K (0) or V (1) rows of `slots` as fp32."""
    if not s["case"]["fp8"]:
        return s["kv"][which].flatten(0, 1)[slots].float()
    codes, scales = s["kv"][2 * which:2 * which + 2]
    values = codes.flatten(0, 1)[slots].view(torch.float8_e4m3fn).float()
    return values * scales.flatten(0, 1)[slots].repeat_interleave(128, -1)


def _softmax(s, q, seen):
    """q [B, rows, heads, D], seen [B, rows, tokens] -> out [B, rows, heads, D], lse and weights [B, Hkv, rows, G, tokens]."""
    c = s["case"]
    B, T = q.shape[:2]
    Hkv, G, D, ps = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"], c["page"]
    j = torch.arange(seen.shape[-1], device=DEV)
    slots = s["table"].long().clamp(min=0)[:, j // ps] * ps + j % ps
    x = q.float().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    logit = torch.matmul(x, _rows_fp32(s, 0, slots).permute(0, 2, 3, 1)) / math.sqrt(D)
    logit = torch.where(seen[:, None, :, None], logit.reshape(B, Hkv, T, G, -1), -torch.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = torch.exp(logit - top)
    total = weight.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, T, Hkv * G)
    weight = weight / total.clamp(min=1e-30)
    out = torch.matmul(weight.reshape(B, Hkv, T * G, -1), _rows_fp32(s, 1, slots).permute(0, 2, 1, 3))
    return out.reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D), lse, weight


def _family(s, T):
    """Drafted tokens laid out [rows, T]: their places in the list, which exist, and who is whose ancestor (or itself)."""
    at = s["off"][:-1, None].long() + torch.arange(T, device=DEV)
    exists = at < s["off"][1:, None]
    parent = s["parent"].long()[at.clamp(max=s["parent"].numel() - 1)]
    step = (parent[..., None] == torch.arange(T, device=DEV)) & exists[..., None]
    eye = torch.eye(T, dtype=torch.float64, device=DEV)
    return at, exists, torch.linalg.matrix_power(eye + step.double(), max(T - 1, 1)) > 0   # sums of paths of each length


def _plain_tree(s):
    c = s["case"]
    B, T = c["rows"], c["drafts"]
    at, exists, family = _family(s, T)
    count = s["off"][1:] - s["off"][:-1]
    base = (s["seq_len"] - count)[:, None, None].long()
    j = torch.arange(c["high"], device=DEV)[None, None]
    kin = torch.gather(family, 2, (j - base).clamp(0, T - 1).expand(B, T, -1))
    seen = exists[..., None] & ((j < base) | ((j < s["seq_len"][:, None, None]) & kin))
    if c["window"]:                            # by position: a drafted token's is its depth behind the cached ones
        depth = family.sum(-1)                 # 1 for a child of the cached tokens
        where = torch.where(j < base, j, base - 1 + torch.gather(depth, 1, (j - base).clamp(0, T - 1)[:, 0])[:, None])
        seen = seen & (where > base - 1 + depth[..., None] - c["window"])
    out, lse, _ = _softmax(s, s["q"][at.clamp(max=s["q"].shape[0] - 1)], seen)
    s["out"][at[exists]] = out[exists].to(torch.bfloat16)      # rows behind the last drafted token stay as they are
    s["lse"][at[exists]] = lse[exists]


def _plain_weights(s):
    c = s["case"]
    j = torch.arange(s["weights"].shape[1], device=DEV)
    length = s["seq_len"][:, None]
    seen = j < length
    if c["window"]:
        seen = seen & (j >= length - c["window"])
    out, lse, weight = _softmax(s, s["q"][:, None], seen[:, None])
    s["out"].copy_(out[:, 0])
    s["lse"].copy_(lse[:, 0])
    s["weights"] += weight.sum((1, 2, 3))


def _move(s, row, dst, src):
    """Tokens dst[i] of rows row[i] become what tokens src[i] were, in every plane."""
    ps, table = s["case"]["page"], s["table"].long()
    to, at = table[row, dst // ps], table[row, src // ps]
    for plane in s["pool"]:
        plane[:, to, dst % ps] = plane[:, at, src % ps]


def _release(s, new_len):
    """The page table and references of rows that are cut to new_len."""
    ps, table = s["case"]["page"], s["table"].long()
    j = torch.arange(table.shape[1], device=DEV) * ps
    dropped = (j < s["seq_len"][:, None]) & (j >= new_len[:, None])
    s["ref_out"].copy_(s["ref"].long().scatter_add(0, table.clamp(min=0).reshape(-1), -dropped.reshape(-1).long()))
    s["table_out"].copy_(torch.where(j < new_len[:, None], table, -1))
    s["len_out"].copy_(new_len)


def _plain_accept(s):
    c = s["case"]
    T = c["drafts"]
    _, _, family = _family(s, T)
    count = (s["off"][1:] - s["off"][:-1]).long()
    base, last = s["seq_len"].long() - count, s["last"].long()
    rows = torch.arange(c["rows"], device=DEV)
    path = family[rows, last.clamp(min=0)] & (last >= 0)[:, None]
    row, node = torch.nonzero(path, as_tuple=True)
    rank = torch.cumsum(path.long(), 1)[row, node] - 1
    _move(s, row, base[row] + rank, base[row] + node)
    _release(s, base + path.sum(1))


def _plain_evict(s):
    c = s["case"]
    ps = c["page"]
    j = torch.arange(s["weights"].shape[1], device=DEV)
    length = s["seq_len"].long()
    held = j < length[:, None]
    pos = s["positions"].long()
    newest = torch.where(held, pos, -1).amax(1, keepdim=True)
    shared = s["ref"][s["table"].long().clamp(min=0)].repeat_interleave(ps, 1) > 1
    always = held & ((pos < c["first"]) | (pos > newest - c["recent"]) | shared)
    keep = torch.maximum(s["budget"].long(), always.sum(1)).minimum(length)
    key = torch.where(always, torch.inf, torch.where(held, s["weights"], -torch.inf))
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, j[None].expand_as(order))
    kept = held & (rank < keep[:, None])
    hole, filler = ~kept & (j < keep[:, None]), kept & (j >= keep[:, None])
    row, dst = torch.nonzero(hole, as_tuple=True)      # both row by row, places ascending, as many of each in a row
    _, src = torch.nonzero(filler, as_tuple=True)
    stays = kept & (j < keep[:, None])
    s["weights_out"].copy_(torch.where(stays, s["weights"], 0.0))
    s["positions_out"].copy_(torch.where(stays, s["positions"], -1))
    s["weights_out"][row, dst], s["positions_out"][row, dst] = s["weights"][row, src], s["positions"][row, src]
    _move(s, row, dst, src)
    _release(s, keep)


def run(state):
    s = state
    c = s["case"]
    if own:
        from indexer_driven_sparse_gb300 import binding as qb
    if c["op"] == "tree":
        if not own:
            _plain_tree(s)
        elif c["fp8"]:
            qb.qsa_tree_decode_fp8kv(s["cfg"], s["q"], s["off"], s["parent"], c["drafts"], s["kv"], s["table"], s["seq_len"],
                                     s["out"], s["lse"], s["ws"])
        else:
            qb.qsa_tree_decode(s["cfg"], s["q"], s["off"], s["parent"], c["drafts"], *s["kv"], s["table"], s["seq_len"],
                               s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "weights":
        if not own:
            _plain_weights(s)
        elif c["fp8"]:
            qb.qsa_paged_decode_weights_fp8kv(s["cfg"], s["q"], s["kv"], s["table"], s["seq_len"], s["out"], s["lse"],
                                              s["weights"], s["ws"])
        else:
            qb.qsa_paged_decode_weights(s["cfg"], s["q"], *s["kv"], s["table"], s["seq_len"], s["out"], s["lse"],
                                        s["weights"], s["ws"])
        return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}
    if c["op"] == "accept":
        if own:
            qb.qsa_accept_drafts(c["page"], s["off"], s["parent"], s["last"], s["table"], s["seq_len"], s["ref"],
                                 s["table_out"], s["len_out"], s["ref_out"], s["pool"], s["ws"])
        else:
            _plain_accept(s)
        more = {}
    else:
        if own:
            qb.qsa_evict_tokens(c["page"], s["budget"], c["first"], c["recent"], s["weights"], s["positions"], s["table"],
                                s["seq_len"], s["ref"], s["weights_out"], s["positions_out"], s["table_out"], s["len_out"],
                                s["ref_out"], s["pool"], s["ws"])
        else:
            _plain_evict(s)
        more = {"weights": s["weights_out"], "positions": s["positions_out"]}
    pool = [s["pool"][0].view(torch.float8_e4m3fn), s["pool"][1]] if c["fp8"] else s["pool"]
    return {"table": s["table_out"], "seq_len": s["len_out"], "ref": s["ref_out"], "pool": pool, **more}


# ------------------------------------------------------------------------------------------ work
def work(case):
    """Bytes and operations of one pass, each input read once and each output written once. Lengths and drafted
    tokens are drawn uniformly: their means stand for them."""
    c = case
    mean = (c["low"] + c["high"]) / 2
    drafts = (c.get("drafts_low", 1) + c.get("drafts", 1)) / 2
    if c["op"] in ("tree", "weights"):
        D, Hq, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
        seen = min(mean, c["window"] + drafts) if c["window"] else mean
        row = D + D // 128 * 4 if c["fp8"] else 2 * D
        tokens = c["rows"] * seen
        add = 8 * tokens if c["op"] == "weights" else 4 * c["rows"] * drafts
        return {"bytes": tokens * 2 * Hkv * row + c["rows"] * drafts * (4 * Hq * D + 4 * Hq) + tokens / c["page"] * 4 + add,
                "flops": 4 * tokens * drafts * Hq * D}
    token = 2 * c["layers"] * (c["width"] + c["width"] // 128 * 4 if c["fp8"] else 2 * c["width"])   # in every plane
    pages = c["rows"] * (mean / c["page"] + 0.5)
    tables = c["rows"] * 8 * (c["high"] / c["page"] + 1) + 8 * pages
    if c["op"] == "accept":
        # a chain with branches of n tokens has an accepted path of a third of them; half of it moves
        return {"bytes": tables + c["rows"] * (12 + 4 * drafts) + c["rows"] * drafts / 6 * token * 2, "flops": 0}
    over = max(0.0, mean - c["budget"])
    moved = over * c["budget"] / max(mean, 1)
    return {"bytes": tables + c["rows"] * 16 * mean + c["rows"] * moved * 2 * token, "flops": 0}


# ------------------------------------------------------------------------------------------ 64 bits
def _row64(s, r, which, lo, n):
    """K or V rows [lo, n) of row r in 64 bits, [n - lo, Hkv, D]."""
    ps = s["case"]["page"]
    pages = s["table"][r, lo // ps:(n + ps - 1) // ps].long()
    cut = slice(lo % ps, lo % ps + n - lo)
    if not s["case"]["fp8"]:
        return s["kv"][which][pages].flatten(0, 1)[cut].double()
    codes, scales = s["kv"][2 * which], s["kv"][2 * which + 1]
    y = codes[pages].flatten(0, 1)[cut].view(torch.float8_e4m3fn).double()
    z = scales[pages].flatten(0, 1)[cut].double()
    return (y.reshape(*z.shape, 128) * z[..., None]).reshape(y.shape)


def _lines(parent):
    """For each drafted token the list of its ancestors and itself, oldest first."""
    found = []
    for i, p in enumerate(parent):
        found.append((found[p] if p >= 0 else []) + [i])
    return found


def _attention64(s):
    c = s["case"]
    Hkv, G, D = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
    tree = c["op"] == "tree"
    n_q = s["q"].shape[0]
    out = torch.zeros(n_q, c["q_heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(n_q, c["q_heads"], dtype=torch.float64, device=DEV)
    weights = None if tree else s["weights"].double()
    off = s["off"].tolist() if tree else list(range(c["rows"] + 1))
    for r, n in enumerate(s["seq_len"].tolist()):
        T = off[r + 1] - off[r]
        if n == 0:
            lse[off[r]:off[r + 1]] = -torch.inf
        if T == 0 or n == 0:
            continue
        base = n - T
        lines = _lines(s["parent"][off[r]:off[r + 1]].tolist()) if tree else [[0]]
        lo = max(0, base + 1 - c["window"]) if c["window"] else 0
        bias = torch.zeros(T, n - lo, dtype=torch.float64)
        bias[:, max(base - lo, 0):] = -torch.inf
        for i, line in enumerate(lines):
            own_position = base + len(line) - 1
            bias[i, [base + a - lo for k, a in enumerate(line) if not c["window"] or base + k > own_position - c["window"]]] = 0
            if c["window"]:
                bias[i, :max(0, min(base, own_position - c["window"] + 1) - lo)] = -torch.inf
        bias = bias.to(DEV).repeat_interleave(G, 0)
        K, V = _row64(s, r, 0, lo, n), _row64(s, r, 1, lo, n)
        for h in range(Hkv):
            x = s["q"][off[r]:off[r + 1], h * G:(h + 1) * G].double().reshape(T * G, D)
            t = x @ K[:, h].T * D ** -0.5 + bias
            l = torch.logsumexp(t, 1)
            t = torch.exp(t - l[:, None])
            lse[off[r]:off[r + 1], h * G:(h + 1) * G] = l.reshape(T, G)
            out[off[r]:off[r + 1], h * G:(h + 1) * G] = (t @ V[:, h]).reshape(T, G, D)
            if not tree:
                weights[r, lo:n] += t.sum(0)
    return {"out": out, "lse": lse} if tree else {"out": out, "lse": lse, "weights": weights}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("tree", "weights"):
        return _attention64(s)
    # whole numbers by hand on the host, rows' contents as they were copied
    ps = c["page"]
    table, length, ref = s["table"].tolist(), s["seq_len"].tolist(), s["ref"].tolist()
    new_table, new_len, new_ref, to, at = [], [], list(ref), [], []
    more = {}
    if c["op"] == "evict":
        weights, positions = s["weights"].tolist(), s["positions"].tolist()
        room = s["weights"].shape[1]
        more = {"weights": [], "positions": []}
    else:
        off, parent, last = s["off"].tolist(), s["parent"].tolist(), s["last"].tolist()
    for r, n in enumerate(length):
        slot = lambda j: (table[r][j // ps], j % ps)  # noqa: E731
        if c["op"] == "accept":
            T = off[r + 1] - off[r]
            line = _lines(parent[off[r]:off[r + 1]])[last[r]] if last[r] >= 0 else []
            keep = n - T + len(line)
            moves = [(n - T + k, n - T + a) for k, a in enumerate(line) if k != a]
        else:
            newest = max(positions[r][:n], default=-1)
            safe = {j for j in range(n) if positions[r][j] < c["first"] or positions[r][j] > newest - c["recent"]
                    or ref[table[r][j // ps]] > 1}
            keep = min(n, max(c["budget"], len(safe)))
            rest = sorted((j for j in range(n) if j not in safe), key=lambda j: (-weights[r][j], j))
            stays = safe | set(rest[:keep - len(safe)])
            moves = list(zip([j for j in range(keep) if j not in stays], [j for j in range(keep, n) if j in stays]))
            w, p = weights[r][:keep], positions[r][:keep]
            for d, a in moves:
                w[d], p[d] = weights[r][a], positions[r][a]
            more["weights"].append(w + [0.0] * (room - keep))
            more["positions"].append(p + [-1] * (room - keep))
        to += [slot(d) for d, _ in moves]
        at += [slot(a) for _, a in moves]
        pages = (keep + ps - 1) // ps
        for p in table[r][pages:(n + ps - 1) // ps]:
            new_ref[p] -= 1
        new_table.append(table[r][:pages] + [-1] * (len(table[r]) - pages))
        new_len.append(keep)
    index = lambda v: torch.tensor(v, dtype=torch.long, device=DEV).reshape(-1, 2).T  # noqa: E731
    (tp, to_), (ap, at_) = index(to), index(at)
    pool = [plane.clone() for plane in s["pool"]]
    for new, old in zip(pool, s["pool"]):
        new[:, tp, to_] = old[:, ap, at_]
    if c["fp8"]:
        pool[0] = pool[0].view(torch.float8_e4m3fn)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if more:
        more = {"weights": torch.tensor(more["weights"], dtype=torch.float64, device=DEV), "positions": ints(more["positions"])}
    return {"table": ints(new_table), "seq_len": ints(new_len), "ref": ints(new_ref), "pool": pool, **more}
