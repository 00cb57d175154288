"""CPU oracle of the paged-cache entry points: rotary positions with the append, attention over the
pages, accumulated attention weights, eviction.

TEST INFRASTRUCTURE ONLY (see the package header).  Plain numpy in float64, one sequence and head
after the other, written from the definitions in ``include/specdec.h``.  Pools are [num_pages,
page_size, kv_heads, dim] arrays, records [num_pages, kv_heads, page_size], both already widened to
float64 (positions: integers).
"""
from __future__ import annotations

import math

import numpy as np


def place(table, b, slot, page_size):
    """(page id, place in the page) of a slot."""
    return int(table[b, slot // page_size]), slot % page_size


def round_rows(num_draft, kv_len, b, K, capacity):
    """(valid, rows the sequence has or poisons)."""
    k = K if num_draft is None else int(num_draft[b])
    if k < 0 or k > K:
        return False, K + 1
    L = int(kv_len[b])
    return L >= 0 and L + k + 1 <= capacity, k + 1


def pages_good(table, b, slots, page_size, num_pages):
    used = table[b, : -(-slots // page_size)]
    return bool(((used >= 0) & (used < num_pages)).all())


def rope_row(x, position, inv_freq, interleaved, scale):
    """One head's row turned by its position (complex multiplication, one pair at a time)."""
    y = np.array(x, dtype=np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = float(position) * float(inv_freq[i])
        z = complex(x[a], x[b]) * complex(math.cos(t), math.sin(t)) * scale
        y[a], y[b] = z.real, z.imag
    return y


def rope_append(q, k, v, pool_k, pool_v, table, kv_len, inv_freq, *, interleaved=False, scale=1.0,
                num_draft=None, first_pos=None, weight=None, position=None):
    """Returns (q_out, pool_k, pool_v, weight, position), the inputs not modified."""
    B, T, H, _ = q.shape
    num_pages, page_size, Hkv, _ = pool_k.shape
    capacity = table.shape[1] * page_size
    out = np.zeros(q.shape)
    pk, pv = pool_k.copy(), pool_v.copy()
    w = None if weight is None else weight.copy()
    ps = None if position is None else position.copy()
    for b in range(B):
        valid, rows = round_rows(num_draft, kv_len, b, T - 1, capacity)
        start = int(kv_len[b] if first_pos is None else first_pos[b])
        valid = valid and start >= 0 and start + rows - 1 <= 2 ** 31 - 1
        for i in range(rows):
            page = -1
            if valid:
                page, off = place(table, b, int(kv_len[b]) + i, page_size)
            if not 0 <= page < num_pages:
                out[b, i] = np.nan
                continue
            for h in range(H):
                out[b, i, h] = rope_row(q[b, i, h], start + i, inv_freq, interleaved, scale)
            for h in range(Hkv):
                pk[page, off, h] = rope_row(k[b, i, h], start + i, inv_freq, interleaved, scale)
                pv[page, off, h] = v[b, i, h]
            if w is not None:
                w[page, :, off] = 0.0
            if ps is not None:
                ps[page, :, off] = start + i
    return out, pk, pv, w, ps


def gathered(pool, table, b, count, h):
    """Slots 0..count-1 of head h, [count, dim]."""
    j = np.arange(count)
    return pool[table[b, j // pool.shape[1]], j % pool.shape[1], h]


def paged_attention(q, pool_k, pool_v, table, kv_len, *, num_draft=None, scale=1.0):
    """Returns (out, lse, spread, score_size): spread [B, T, H, D] = sum_j p_j |v_j| and score_size
    [B, T, H] = scale max_j sum_d |q_d k_jd|, from which a test derives its tolerances."""
    B, T, H, D = q.shape
    num_pages, page_size, Hkv, _ = pool_k.shape
    capacity = table.shape[1] * page_size
    out, spread = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    lse, size = np.full((B, T, H), -np.inf), np.zeros((B, T, H))
    for b in range(B):
        valid, rows = round_rows(num_draft, kv_len, b, T - 1, capacity)
        valid = valid and pages_good(table, b, int(kv_len[b]) + rows, page_size, num_pages)
        if not valid:
            out[b, :rows], lse[b, :rows] = np.nan, np.nan
            continue
        total = int(kv_len[b]) + rows
        for g in range(Hkv):
            k, v = gathered(pool_k, table, b, total, g), gathered(pool_v, table, b, total, g)
            for i in range(rows):
                n = int(kv_len[b]) + i + 1
                for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                    x = scale * (k[:n] @ q[b, i, h])
                    top = x.max()
                    e = np.exp(x - top)
                    p = e / e.sum()
                    out[b, i, h] = p @ v[:n]
                    lse[b, i, h] = top + np.log(e.sum())
                    spread[b, i, h] = p @ np.abs(v[:n])
                    size[b, i, h] = scale * (np.abs(k[:n]) @ np.abs(q[b, i, h])).max()
    return out, lse, spread, size


def kv_weights(q, lse, pool_k, table, kv_len, weight, *, num_draft=None, accept_len=None, scale=1.0):
    """Returns (weight, added, score_size): the new records, what was added to each, and the largest
    scale sum_d |q_d k_jd| of the call."""
    B, T, H, _ = q.shape
    num_pages, page_size, Hkv, _ = pool_k.shape
    capacity = table.shape[1] * page_size
    w, added, size = weight.copy(), np.zeros(weight.shape), 0.0
    for b in range(B):
        valid, rows = round_rows(num_draft, kv_len, b, T - 1, capacity)
        A = rows - 1 if accept_len is None else int(accept_len[b])
        if not valid or not 0 <= A < rows:
            continue
        for j in range(int(kv_len[b]) + A + 1):
            page, off = place(table, b, j, page_size)
            if not 0 <= page < num_pages:
                continue
            for g in range(Hkv):
                k = pool_k[page, off, g]
                total = 0.0
                for i in range(max(0, j - int(kv_len[b])), A + 1):
                    for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                        total += math.exp(scale * float(k @ q[b, i, h]) - float(lse[b, i, h]))
                        size = max(size, scale * float(np.abs(k) @ np.abs(q[b, i, h])))
                w[page, g, off] += total
                added[page, g, off] += total
    return w, added, size


def kv_evict(pool_k, pool_v, table, kv_len, weight, position, budget, *, keep_first=0, keep_last=0):
    """Returns (pool_k, pool_v, weight, position, new_len), the inputs not modified."""
    k, v, w, p = pool_k.copy(), pool_v.copy(), weight.copy(), position.copy()
    num_pages, page_size, Hkv, _ = pool_k.shape
    capacity = table.shape[1] * page_size
    new_len = np.zeros(len(kv_len), dtype=np.int64)
    for b, L in enumerate(int(x) for x in kv_len):
        if L < 0 or L > capacity:
            new_len[b] = -1
            continue
        new_len[b] = min(L, budget)
        if L <= budget:
            continue
        if not pages_good(table, b, L, page_size, num_pages):
            new_len[b] = -1
            continue
        at = [place(table, b, j, page_size) for j in range(L)]
        for h in range(Hkv):
            pos = [int(position[pg, h, o]) for pg, o in at]
            wt = [float(weight[pg, h, o]) for pg, o in at]
            newest = max(pos)

            def rank(j):
                if pos[j] < keep_first or pos[j] > newest - keep_last:
                    return (0, 0.0, j)
                return (2, 0.0, j) if math.isnan(wt[j]) else (1, -wt[j], j)

            kept = set(sorted(range(L), key=rank)[:budget])
            movers = [j for j in range(budget, L) if j in kept]
            holes = [j for j in range(budget) if j not in kept]
            assert len(movers) == len(holes)
            for src, dst in zip(movers, holes):
                (sp, so), (dp, do) = at[src], at[dst]
                k[dp, do, h], v[dp, do, h] = pool_k[sp, so, h], pool_v[sp, so, h]
                w[dp, h, do], p[dp, h, do] = weight[sp, h, so], position[sp, h, so]
    return k, v, w, p, new_len
