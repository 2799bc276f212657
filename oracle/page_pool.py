"""Reference of the page pool: fork, free, compact and copy, as loops over rows and pages.

From the definitions in include/page_pool.h. Shares no code with the GPU path. Inputs are not
changed; every function returns a dict of its outputs.
"""
from __future__ import annotations

import numpy as np


def _pages(tokens, page_size):
    return -(-int(tokens) // page_size)


def fork(fork_from, lens, held_lens, block_table, shares, free_pages, free_count, page_size):
    table, shares = np.array(block_table), np.array(shares)
    n = len(table)
    stack = list(free_pages[: int(free_count)])
    lens_out, held_out = np.array(lens), np.array(held_lens)
    pairs, unserved = np.full((n, 2), -1, np.int32), 0
    for i in range(n):
        s = int(fork_from[i])
        if s < 0:
            continue
        if s >= n or s == i or fork_from[s] >= 0 or lens[i] != 0 or held_lens[i] != 0:
            unserved += 1
            continue
        full, part = divmod(int(lens[s]), page_size)
        if part and not stack:
            unserved += 1
            continue
        for c in range(full):
            table[i, c] = block_table[s][c]
            shares[table[i, c]] += 1
        if part:
            table[i, full] = stack.pop()
            pairs[i] = block_table[s][full], table[i, full]
        lens_out[i] = held_out[i] = lens[s]
    return dict(pairs=pairs, lens_out=lens_out, held_lens_out=held_out, free_count_out=len(stack), unserved=unserved,
                block_table=table, shares=shares)


def free(keep_lens, held_lens, block_table, shares, free_pages, free_count, page_size):
    shares, stack = np.array(shares), np.array(free_pages)
    count, held_out = int(free_count), np.array(held_lens)
    gone = []
    for i, row in enumerate(block_table):
        held_out[i] = min(max(int(keep_lens[i]), 0), int(held_lens[i]))
        for c in range(_pages(held_out[i], page_size), _pages(held_lens[i], page_size)):
            if shares[row[c]] == 0:
                gone.append(int(row[c]))
            else:
                shares[row[c]] -= 1
    for p in sorted(gone, reverse=True):
        stack[count] = p
        count += 1
    return dict(held_lens_out=held_out, free_count_out=count, shares=shares, free_pages=stack)


def compact(held_lens, block_table, shares, free_pages, free_count, page_size, keep_pages):
    n_pages = len(free_pages)
    used = sorted({int(row[c]) for row, h in zip(block_table, held_lens) for c in range(_pages(h, page_size))})
    places = sorted(int(p) for p in free_pages[: int(free_count)] if p < keep_pages)
    late = [p for p in used if p >= keep_pages]
    moves = list(zip(late, places))
    to = dict(moves)
    table, shares_out = np.array(block_table), np.array(shares)
    for row, h in zip(table, held_lens):
        for c in range(_pages(h, page_size)):
            row[c] = to.get(int(row[c]), row[c])
    for a, b in moves:
        shares_out[b], shares_out[a] = shares[a], 0
    left = places[len(moves):][::-1]
    free_out = np.full(n_pages, -1, np.int32)
    free_out[: len(left)] = left
    pairs = np.full((min(keep_pages, n_pages - keep_pages), 2), -1, np.int32)
    if moves:
        pairs[: len(moves)] = moves
    return dict(block_table_out=table, shares_out=shares_out, free_pages_out=free_out, free_count_out=len(left), pairs=pairs,
                n_pairs=len(moves), unmoved=len(late) - len(moves))


def copy(pairs, cache, count=None):
    """A copy of the cache [n_pages, ...] after the pairs."""
    out = np.array(cache)
    for a, b in pairs[: len(pairs) if count is None else max(int(count), 0)]:
        if 0 <= a < len(cache) and 0 <= b < len(cache):
            out[b] = cache[a]
    return out
