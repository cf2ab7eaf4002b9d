"""A batch that answers from one compressed prompt: page tables, appends, shared-prompt attention
and token sampling (fp64 / integers, test infrastructure only).

The pages have no counterpart of these steps except the logit bias alpha_c log R of [SelKV] Core
component 2, which the prompt's keys carry.  Written out from the definitions in include/kvc.h.
"""
from __future__ import annotations

import numpy as np

__all__ = ["page_tables", "page_append", "prefix_attention", "sample"]


def _pages(n: int, page: int) -> int:
    return -(-n // page)


def page_tables(lens, lens_new, table, ring, head: int, count: int, page: int, slots_cap=None):
    """(ok, table, ring, (head, count), lens, slots, slot_start) after the rows went from lens to
    lens_new tokens; on refusal (ok False) everything is as it was, slots -1 and slot_start 0."""
    table, ring = np.array(table), np.array(ring)
    n, cap = len(ring), table.shape[1] * page
    rows = len(lens)
    start = np.zeros(rows + 1, np.int64)
    take = sum(max(0, _pages(z, page) - _pages(a, page)) for a, z in zip(lens, lens_new))
    free = sum(max(0, _pages(a, page) - _pages(z, page)) for a, z in zip(lens, lens_new))
    new = sum(max(0, z - a) for a, z in zip(lens, lens_new))
    width = new if slots_cap is None else slots_cap
    slots = np.full(max(width, 0), -1, np.int64)
    if (any(not 0 <= x <= cap for x in list(lens) + list(lens_new)) or not 0 <= head < n or not 0 <= count <= n
            or take > count or count + free > n or (slots_cap is not None and new > slots_cap)):
        return False, table, ring, (head, count), list(lens), slots, start
    first_free = head + count
    at = head
    for r in range(rows):
        for j in range(_pages(lens[r], page), _pages(lens_new[r], page)):
            table[r, j] = ring[at % n]
            at += 1
        start[r + 1] = start[r] + max(0, lens_new[r] - lens[r])
        for i, t in enumerate(range(lens[r], lens_new[r])):
            slots[start[r] + i] = table[r, t // page] * page + t % page
    for r in range(rows):
        for j in range(_pages(lens_new[r], page), _pages(lens[r], page)):
            ring[first_free % n] = table[r, j]
            first_free += 1
    return True, table, ring, (at % n, count - take + free), list(lens_new), slots, start


def page_append(k, v, K, V, slots):
    """Pools [pages][H][page][d] after token t entered slot slots[t] (negative: skipped)."""
    K, V = np.array(K), np.array(V)
    page = K.shape[2]
    for t, s in enumerate(slots):
        if s >= 0:
            K[s // page, :, s % page] = k[t]
            V[s // page, :, s % page] = v[t]
    return K, V


def prefix_attention(q, kp, vp, ko, vo, R=None, alpha_c: float = 1.0, scale=None):
    """o [G][d], lse [G], weights [G][n] of query rows q [G][d] over prompt keys kp, vp [P][d] (logit
    bias alpha_c log R) and own keys ko, vo [n][d]; a row without keys gives 0 and -inf."""
    q = np.asarray(q, np.float64)
    d = q.shape[1]
    s = 1.0 / np.sqrt(d) if scale is None else scale
    kk = np.concatenate([np.asarray(kp, np.float64).reshape(-1, d), np.asarray(ko, np.float64).reshape(-1, d)])
    vv = np.concatenate([np.asarray(vp, np.float64).reshape(-1, d), np.asarray(vo, np.float64).reshape(-1, d)])
    if len(kk) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    z = q @ kk.T * s
    if R is not None:
        P = len(np.asarray(kp).reshape(-1, d))
        z[:, :P] += alpha_c * np.log(np.asarray(R, np.float64))[None, :P]
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    w = e / e.sum(axis=1, keepdims=True)
    return w @ vv, (m + np.log(e.sum(axis=1, keepdims=True)))[:, 0], w


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, kept) of one row of logits."""
    z = np.asarray(z, np.float64).copy()
    z[np.isnan(z)] = -np.inf
    order = np.lexsort((np.arange(len(z)), -z))
    order = order[z[order] > -np.inf]
    if len(order) == 0:
        return -1, -np.inf, 0
    if not temperature > 0:
        return int(order[0]), 0.0, 1
    zm = z[order[0]]
    if zm == np.inf:                           # infinite logits are the only ones kept, all alike
        order = order[z[order] == np.inf]
        z = np.where(z == np.inf, 0.0, -np.inf)
        zm = 0.0
    dist = z - zm
    with np.errstate(invalid="ignore"):
        x = np.where(np.isneginf(dist), -np.inf, dist / temperature)
    w = np.exp(x)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        c = np.cumsum(w[order].astype(np.longdouble))
        before = np.concatenate([[0], c[:-1]])
        n = int((before < np.longdouble(top_p) * c[-1]).sum())
        order = order[:max(1, n)]
    if min_p > 0:
        order = order[w[order] >= min(min_p, 1.0)]
    kept = np.sort(order)
    c = np.cumsum(w[kept].astype(np.longdouble))
    uu = 0.0 if np.isnan(u) else min(max(float(u), 0.0), 1 - 2.0 ** -24)
    i = int(np.searchsorted(c, np.longdouble(uu) * c[-1], side="right"))
    return int(kept[i]), float(np.log(w[kept[i]] / c[-1])), len(kept)
