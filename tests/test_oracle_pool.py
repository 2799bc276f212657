"""The page pool's reference: steps worked out by hand, and what has to hold of any pool."""
import numpy as np
import pytest

from _pool import check_pool, random_pool
from oracle import page_pool as pool


def test_fork_by_hand():
    # pages of 8 tokens; row 0 holds 20 tokens in pages 4, 2, 7; rows 1 and 3 are empty, row 2 holds 16 in pages 0 and 1
    table = np.array([[4, 2, 7, 0], [9, 9, 9, 9], [0, 1, 0, 0], [9, 9, 9, 9]])
    lens = np.array([20, 0, 16, 0])
    r = pool.fork([-1, 0, -1, 2], lens, lens, table, np.zeros(8, int), [6, 5, 3, 9, 9, 9, 9, 9], 3, 8)
    assert r["block_table"].tolist() == [[4, 2, 7, 0], [4, 2, 3, 9], [0, 1, 0, 0], [0, 1, 9, 9]]
    assert r["shares"].tolist() == [1, 1, 1, 0, 1, 0, 0, 0]
    assert r["pairs"].tolist() == [[-1, -1], [7, 3], [-1, -1], [-1, -1]]
    assert r["lens_out"].tolist() == [20, 20, 16, 16] and r["free_count_out"] == 2 and r["unserved"] == 0


def test_fork_refusals_by_hand():
    table = np.zeros((5, 2), int)
    lens = np.array([3, 0, 0, 5, 0])
    # row 1 from itself, 2 from a forked row, 3 is not empty, 4 finds no page
    r = pool.fork([-1, 1, 4, 0, 0], lens, lens, table, np.zeros(4, int), [3, 3, 3, 3], 0, 8)
    assert r["unserved"] == 4 and (r["block_table"] == table).all() and (r["lens_out"] == lens).all() and r["free_count_out"] == 0


def test_free_by_hand():
    # row 0 ends, row 1 goes from 17 tokens to 9; page 5 is held by both, page 2 by row 0 alone
    table = np.array([[5, 2, 3], [5, 1, 6]])
    shares = np.array([0, 0, 0, 0, 0, 1, 0, 0])
    r = pool.free([0, 9], [24, 17], table, shares, [7, 0, 0, 0, 0, 0, 0, 0], 1, 8)
    assert r["free_pages"][:4].tolist() == [7, 6, 3, 2] and r["free_count_out"] == 4
    assert r["shares"].tolist() == [0] * 8 and r["held_lens_out"].tolist() == [0, 9]


def test_compact_by_hand():
    # 8 pages, keep 4: rows hold 6, 1 and 6, 5 (6 shared); 0, 3 and 7 are free
    table = np.array([[6, 1, 2], [6, 5, 0]])
    r = pool.compact([16, 10], table, [0, 0, 0, 0, 0, 0, 1, 0], [7, 3, 0, 9, 9, 9, 9, 9], 3, 8, 4)
    assert r["block_table_out"].tolist() == [[3, 1, 2], [3, 0, 0]]
    assert r["pairs"][:2].tolist() == [[5, 0], [6, 3]] and r["n_pairs"] == 2 and r["unmoved"] == 0
    assert r["shares_out"].tolist() == [0, 0, 0, 1, 0, 0, 0, 0] and r["free_count_out"] == 0


@pytest.mark.parametrize("seed", range(20))
def test_a_pool_stays_whole(seed):
    """After any run of forks, ends and compactions every page is held or free, once, and shares counts the holders."""
    rng = np.random.default_rng(seed)
    page = int(rng.choice([8, 16]))
    s = random_pool(rng, n=int(rng.integers(2, 12)), page=page, most=int(rng.integers(1, 90)), spare=int(rng.integers(0, 12)))
    check_pool(s, page)
    n = len(s["table"])
    for _ in range(6):
        empty = np.flatnonzero(s["held"] == 0)
        full = np.flatnonzero(s["held"] > 0)
        src = np.full(n, -1)
        if len(full):
            src[empty] = np.where(rng.random(len(empty)) < 0.7, rng.choice(full, len(empty)), -1)
        r = pool.fork(src, s["held"], s["held"], s["table"], s["shares"], s["free"], s["count"], page)
        s.update(table=r["block_table"], shares=r["shares"], count=r["free_count_out"], held=r["held_lens_out"])
        check_pool(s, page)
        keep = np.where(rng.random(n) < 0.4, 0, s["held"])
        r = pool.free(keep, s["held"], s["table"], s["shares"], s["free"], s["count"], page)
        s.update(shares=r["shares"], free=r["free_pages"], count=r["free_count_out"], held=r["held_lens_out"])
        check_pool(s, page)
        # as many pages as are in use: all fit in front
        in_use = len(s["free"]) - s["count"]
        r = pool.compact(s["held"], s["table"], s["shares"], s["free"], s["count"], page, in_use)
        assert r["unmoved"] == 0 and r["free_count_out"] == 0
        table = r["block_table_out"]
        assert all((table[i, : -(-int(h) // page)] < max(in_use, 1)).all() for i, h in enumerate(s["held"]))
        back = np.concatenate([np.arange(len(s["free"]) - 1, in_use - 1, -1), np.full(in_use, -1)]).astype(np.int32)
        s.update(table=table, shares=r["shares_out"], free=back, count=len(s["free"]) - in_use)
        check_pool(s, page)
