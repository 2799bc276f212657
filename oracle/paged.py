"""Float64 reference of the paged-cache operators: page plan, key/value write, attention.

Plain loops over sequences, heads and tokens, from the definitions in
include/paged_attn.h. Shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np


def page_plan(context_lens, held_lens, cu_seqlens, block_table, free_pages, free_count, n_tokens, page_size):
    """One step's plan; returns a dict of every output (the inputs are not changed)."""
    table = np.array(block_table)
    n, width = table.shape
    stack = list(np.asarray(free_pages)[: int(free_count)])
    free = np.array(free_pages)
    ceil = lambda a: -(-int(a) // page_size)  # noqa: E731
    new = [int(cu_seqlens[i + 1]) - int(cu_seqlens[i]) for i in range(n)]
    have = [ceil(h) for h in held_lens]
    need = [ceil(int(context_lens[i]) + new[i]) for i in range(n)]
    for i in range(n):
        for c in range(need[i], have[i]):
            free[len(stack)] = table[i, c]
            stack.append(table[i, c])
    slots, pos = np.full(n_tokens, -1, np.int32), np.full(n_tokens, -1, np.int32)
    kv, held = np.array(context_lens, np.int32), np.array(held_lens, np.int32)
    unserved, asked, avail = 0, 0, len(stack)
    for i in range(n):
        take = max(need[i] - have[i], 0) if need[i] <= width else 0
        asked += take
        if need[i] > width or (take and asked > avail):
            unserved += 1
            continue
        for c in range(have[i], have[i] + take):
            table[i, c] = stack.pop()
        kv[i] += new[i]
        held[i] = kv[i]
        for t in range(new[i]):
            p = int(context_lens[i]) + t
            pos[int(cu_seqlens[i]) + t] = p
            slots[int(cu_seqlens[i]) + t] = table[i, p // page_size] * page_size + p % page_size
    return dict(slot_map=slots, positions=pos, kv_lens=kv, held_lens_out=held, free_count_out=len(stack), unserved=unserved,
                block_table=table, free_pages=free)


def kv_write(k, cache, slot_map):
    """Rows of k [T, H, D] into a copy of the cache [P, H, S, D]; returns the copy."""
    cache = np.array(cache)
    size = cache.shape[2]
    for t, s in enumerate(slot_map):
        if 0 <= s < cache.shape[0] * size:
            cache[s // size, :, s % size] = k[t]
    return cache


def gather(cache, row, length):
    """The first `length` rows of a sequence, [H, length, D], through its row of the block table."""
    size = cache.shape[2]
    out = np.empty((cache.shape[1], length, cache.shape[3]), cache.dtype)
    for j in range(length):
        out[:, j] = cache[row[j // size], :, j % size]
    return out


def attention(q, k, v, kv_len, window, scale):
    """One sequence: q [m, Hq, D] at positions kv_len - m .., k, v [Hkv, kv_len, D], all float64.

    Returns (o [m, Hq, D], lse [m, Hq], weight [m, Hq, D], size [m, Hq], seen [m]): weight is the softmax-weighted sum of
    |v|, size the largest scale * sum |q||k| of a row, seen the number of keys of a row (for error bounds).
    """
    m, hq, d = q.shape
    g = hq // k.shape[0]
    o, weight = np.zeros((m, hq, d)), np.zeros((m, hq, d))
    lse, size = np.full((m, hq), -np.inf), np.zeros((m, hq))
    seen = np.zeros(m, np.int64)
    for i in range(m):
        p = kv_len - m + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        seen[i] = p + 1 - lo
        for h in range(hq):
            kk, vv = k[h // g, lo:p + 1], v[h // g, lo:p + 1]
            s = scale * (kk @ q[i, h])
            top = s.max()
            size[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            if top == -np.inf:
                continue
            w = np.exp(s - top)
            lse[i, h] = top + np.log(w.sum())
            o[i, h] = (w / w.sum()) @ vv
            weight[i, h] = (w / w.sum()) @ np.abs(vv)
    return o, lse, weight, size, seen
