"""Plain 64-bit oracle of the paged-cache operators: rotary positions, appending, attention of one token
over a page table, forking and compacting pages. numpy only; no code of the library."""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def rope_frequencies(rot, base, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per token of each pair, amplitude)."""
    half = rot // 2
    f = np.array([base ** (-2.0 * i / rot) for i in range(half)])
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        b = base * factor ** (rot / (rot - 2.0))
        return np.array([b ** (-2.0 * i / rot) for i in range(half)]), 1.0
    assert scaling == "by_parts"

    def pair_turning(times):   # index of the pair that turns `times` times over the trained length
        return half * math.log(original_len / (2 * math.pi * times)) / math.log(base)

    lo, hi = max(math.floor(pair_turning(beta_fast)), 0), min(math.ceil(pair_turning(beta_slow)), rot - 1)
    out = []
    for i in range(half):
        g = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append((1 - g) * f[i] + g * f[i] / factor)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


def rope(x, pos, freq, amplitude, begin, interleaved):
    """x [N, H, D], pos [N] -> float64 [N, H, D]."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    for i in range(half):
        a, b = (begin + 2 * i, begin + 2 * i + 1) if interleaved else (begin + i, begin + i + half)
        angle = np.asarray(pos, dtype=np.float64) * freq[i]
        c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
    return y


def slots_of(table_row, n_tokens, page_size):
    t = np.arange(n_tokens)
    return np.asarray(table_row)[t // page_size].astype(np.int64) * page_size + t % page_size


def decode(q, K, V, lo, scale):
    """One query's heads q [Hq, D] over K, V [n, Hkv, D] from token lo on: (out, lse, weighted |V|, max |logit| terms)."""
    Hq, D = q.shape
    Hkv = K.shape[1]
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    mass, terms = np.zeros((Hq, D)), np.zeros(Hq)
    if lo >= len(K):
        return out, lse, mass, terms
    for h in range(Hq):
        k, v = K[lo:, h // (Hq // Hkv)], V[lo:, h // (Hq // Hkv)]
        t = scale * (k @ q[h])
        m = t.max()
        w = np.exp(t - m)
        lse[h] = m + math.log(w.sum())
        w /= w.sum()
        out[h], mass[h] = w @ v, w @ np.abs(v)
        terms[h] = scale * (np.abs(k) @ np.abs(q[h])).max()
    return out, lse, mass, terms


def fork(table, seq_len, ref, parent, add, page_size):
    """(table, seq_len, ref, copies [(src, dst, used tokens)], failed rows)."""
    free = [p for p in range(len(ref)) if ref[p] == 0]
    ld = table.shape[1]
    taken, seen, copies, failed = 0, set(), [], []
    rows, lens = [], []
    for i, (p, more) in enumerate(zip(parent, add)):
        n = int(seq_len[p]) if 0 <= p < len(table) else 0
        if p >= len(table) or p < -1 or more < 0 or n < 0 or -(-(n + more) // page_size) > ld:
            failed.append(i)
            rows.append([])
            lens.append(0)
            continue
        pages = [int(e) for e in table[p][:-(-n // page_size)]] if p >= 0 else []
        own = n % page_size and not (p not in seen and ref[pages[-1]] == 1)
        if p >= 0:
            seen.add(p)
        need = -(-(n + more) // page_size) - len(pages) + bool(own)
        new = free[taken:taken + need] if need == 0 or taken + need <= len(free) else None
        taken += need
        if new is None:
            failed.append(i)
            rows.append([])
            lens.append(0)
            continue
        if own:
            copies.append((pages[-1], new[0], n % page_size))
            pages[-1] = new.pop(0)
        rows.append(pages + new)
        lens.append(n + more)
    out = np.full((len(parent), ld), -1, np.int32)
    count = np.array(ref, dtype=np.int64)
    for row, n in zip(table, seq_len):
        for e in row[:-(-int(n) // page_size)]:
            count[e] -= 1
    for i, pages in enumerate(rows):
        out[i, :len(pages)] = pages
        for e in pages:
            count[e] += 1
    return out, np.array(lens, np.int32), count.astype(np.int32), copies, failed


def compact(table, seq_len, ref, page_size):
    """(table, ref, moves {old: new})."""
    n_live = int((ref > 0).sum())
    holes = [p for p in range(n_live) if ref[p] <= 0]
    movers = [p for p in range(n_live, len(ref)) if ref[p] > 0]
    moves = dict(zip(movers, holes))
    out = np.full_like(table, -1)
    for i, n in enumerate(seq_len):
        for j in range(-(-int(n) // page_size)):
            out[i, j] = moves.get(int(table[i, j]), int(table[i, j]))
    new = np.where(np.arange(len(ref)) < n_live, ref, 0)
    for old, at in moves.items():
        new[at] = ref[old]
    return out, new.astype(np.int32), moves
