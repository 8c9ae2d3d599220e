"""Plain 64-bit oracle of the paged cache's operators for drafted tokens and eviction. numpy only; no code of the library."""

from __future__ import annotations

import numpy as np

from . import paged_oracle as P


def lines(parent):
    """Of each drafted token its ancestors and itself, oldest first."""
    found = []
    for i, p in enumerate(parent):
        found.append((found[p] if p >= 0 else []) + [i])
    return found


def attended(n, parent, window=0):
    """The places each drafted token of a row of n tokens attends."""
    base = n - len(parent)
    out = []
    for line in lines(parent):
        own = base + len(line) - 1                     # its position
        places = [(j, j) for j in range(base)] + [(base + a, base + k) for k, a in enumerate(line)]
        out.append([place for place, pos in places if not window or pos > own - window])
    return out


def tree(q, K, V, parent, scale, window=0, leave_out=()):
    """q [T, Hq, D] over K, V [n, Hkv, D]: a list of (out, lse, mass, terms) of each drafted token; `leave_out`: places
    that nothing attends."""
    gone = set(leave_out)
    result = []
    for i, places in enumerate(attended(len(K), parent, window)):
        at = [j for j in places if j not in gone]
        result.append(P.decode(q[i], K[at], V[at], 0, scale) + (len(at),))
    return result


def token_weights(q, K, lo, scale):
    """What each token of K [n, Hkv, D] receives from one query's heads q [Hq, D], tokens before lo nothing."""
    Hq, Hkv = len(q), K.shape[1]
    total = np.zeros(len(K))
    for h in range(Hq):
        t = scale * (K[lo:, h // (Hq // Hkv)] @ q[h])
        w = np.exp(t - t.max())
        total[lo:] += w / w.sum()
    return total


def accept(n, parent, last):
    """(new length, moves [(to, from)])."""
    line = lines(parent)[last] if last >= 0 else []
    base = n - len(parent)
    return base + len(line), [(base + k, base + a) for k, a in enumerate(line) if k != a]


def evict(weights, positions, shared, budget, first, recent):
    """One row's new length and moves [(to, from)]: weights, positions [n], shared [n] (bool)."""
    n = len(weights)
    if budget < 0 or n <= budget:
        return n, []
    newest = max(int(p) for p in positions)
    safe = {j for j in range(n) if positions[j] < first or positions[j] > newest - recent or shared[j]}
    keep = max(budget, len(safe))
    heavy = [(-np.inf if np.isnan(w) else float(w)) for w in weights]
    nan = [bool(np.isnan(w)) for w in weights]
    rest = sorted((j for j in range(n) if j not in safe), key=lambda j: (nan[j], -heavy[j], j))
    stays = safe | set(rest[:keep - len(safe)])
    return keep, list(zip([j for j in range(keep) if j not in stays], [j for j in range(keep, n) if j in stays]))


def release(table, ref, old_len, new_len, page_size):
    """(table, ref) after the rows are cut to new_len."""
    table, ref = np.array(table), np.array(ref)
    for r in range(len(table)):
        kept, held = -(-int(new_len[r]) // page_size), -(-int(old_len[r]) // page_size)
        for e in table[r, kept:held]:
            ref[e] -= 1
        table[r, kept:] = -1
    return table, ref
