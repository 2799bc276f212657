"""Shared by the page-pool tests: random pools and what has to hold of one."""
from __future__ import annotations

import numpy as np


def random_pool(rng, *, n, page, most, spare, share=0.4, empty=0.3, width=None):
    """A pool of n rows of up to `most` tokens; some rows share the full pages at the start of another's."""
    held = np.where(rng.random(n) < empty, 0, rng.integers(0, most + 1, n))
    have = -(-held // page)
    width = max(1, int(have.max()) if width is None else width)
    table = rng.integers(0, 1 << 20, (n, width)).astype(np.int32)   # what is not held is not looked at
    shared, source = np.zeros(n, int), [None] * n
    base = None
    for i in range(n):
        if base is not None and held[i] and rng.random() < share:
            source[i], shared[i] = base, int(rng.integers(0, min(held[base], held[i]) // page + 1))
        elif held[i]:
            base = i
    n_pages = max(1, int(have.sum() - shared.sum()) + spare)
    order = list(rng.permutation(n_pages))
    shares = np.zeros(n_pages, np.int32)
    for i in range(n):
        for c in range(have[i]):
            if c < shared[i]:
                table[i, c] = table[source[i], c]
                shares[table[i, c]] += 1
            else:
                table[i, c] = order.pop()
    free = np.full(n_pages, -7, np.int32)
    free[: len(order)] = order
    return dict(table=table, held=held.astype(np.int32), shares=shares, free=free, count=len(order))


def check_pool(s, page):
    n_pages = len(s["free"])
    holders = np.zeros(n_pages, int)
    for row, h in zip(s["table"], s["held"]):
        pages = row[: -(-int(h) // page)]
        assert len(set(pages.tolist())) == len(pages)
        holders[pages] += 1
    free = s["free"][: s["count"]]
    assert len(set(free.tolist())) == len(free) and (holders[free] == 0).all()
    assert (holders[np.setdiff1d(np.arange(n_pages), free)] > 0).all()
    assert (s["shares"] == np.maximum(holders - 1, 0)).all()
