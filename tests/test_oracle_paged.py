"""Pins of the paged-cache oracle: hand-worked plans, closed forms of the attention, invariances."""
import numpy as np
import pytest

from oracle import paged


def test_plan_worked_by_hand():
    """Pages of 8. Sequence 0 grows from 7 to 9 tokens (a second page), sequence 1 keeps 3 of 17 (gives two pages back),
    sequence 2 is new with 8 tokens. Stack [40, 41, 42]: pages 11 and 12 are pushed, 12 goes to sequence 0, 11 to 2."""
    table = np.array([[5, -1, -1], [10, 11, 12], [-1, -1, -1]], np.int32)
    r = paged.page_plan([7, 3, 0], [7, 17, 0], [0, 2, 2, 10], table, np.array([40, 41, 42, 0, 0, 0], np.int32), 3, 12, 8)
    assert r["block_table"].tolist() == [[5, 12, -1], [10, 11, 12], [11, -1, -1]]
    assert r["slot_map"].tolist() == [47, 96, 88, 89, 90, 91, 92, 93, 94, 95, -1, -1]
    assert r["positions"].tolist() == [7, 8, 0, 1, 2, 3, 4, 5, 6, 7, -1, -1]
    assert r["kv_lens"].tolist() == [9, 3, 8]
    assert r["free_count_out"] == 3 and r["unserved"] == 0
    assert r["free_pages"].tolist() == [40, 41, 42, 11, 12, 0]


def test_plan_runs_out():
    """Two pages are free, the sequences ask for 1, 2, 0 and 1: the second is not served, nor the fourth, which asked after it."""
    table = np.full((4, 4), -1, np.int32)
    table[2, 0] = 9
    r = paged.page_plan([0, 0, 3, 0], [0, 0, 3, 0], [0, 8, 17, 18, 19], table, np.array([20, 21], np.int32), 2, 19, 8)
    assert r["unserved"] == 2 and r["free_count_out"] == 1
    assert r["kv_lens"].tolist() == [8, 0, 4, 0] and r["held_lens_out"].tolist() == [8, 0, 4, 0]
    assert (r["slot_map"][8:17] == -1).all() and r["slot_map"][17] == 75 and r["slot_map"][18] == -1


def test_plan_never_gives_a_page_twice():
    rng = np.random.default_rng(0)
    n, width, page, n_pages = 9, 6, 8, 60
    table, free, count = np.zeros((n, width), np.int32), rng.permutation(n_pages).astype(np.int32), n_pages
    held = np.zeros(n, np.int64)
    for _ in range(200):
        ctx = np.array([rng.integers(0, h + 1) if rng.random() < 0.4 else h for h in held])
        new = rng.integers(0, 12, n)
        cu = np.concatenate([[0], np.cumsum(new)])
        r = paged.page_plan(ctx, held, cu, table, free, count, int(cu[-1]), page)
        table, free, count, held = r["block_table"], r["free_pages"], r["free_count_out"], r["held_lens_out"].astype(np.int64)
        used = [int(table[i, c]) for i in range(n) for c in range(-(-int(held[i]) // page))]
        assert sorted(used + free[:count].tolist()) == list(range(n_pages))


@pytest.mark.parametrize("window", [0, 3])
def test_attention_closed_forms(window):
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((2, 9, 4)), rng.standard_normal((2, 9, 4)), rng.standard_normal((5, 6, 4))
    o, lse, *_ = paged.attention(0 * q, k, v, 9, window, 1.0)     # equal scores: the mean of what is seen
    for i in range(5):
        lo = max(0, 4 + i - window + 1) if window else 0
        for h in range(6):
            assert np.allclose(o[i, h], v[h // 3, lo:5 + i].mean(0), rtol=0, atol=1e-15)
            assert abs(lse[i, h] - np.log(5 + i - lo)) < 1e-15
    o1, l1, *_ = paged.attention(q, k, v, 9, window, 0.5)         # a shift of all keys along q moves lse, not o
    o2, l2, *_ = paged.attention(q[:, :1], k[:1] + 0.0, v[:1] + 2.0, 9, window, 0.5)
    assert np.allclose(o2, o1[:, :1] + 2.0) and np.allclose(l2, l1[:, :1])
    far = k.copy()
    far[:, 0] = 100 * q[0, 0]                                     # one key far ahead takes all the weight
    o3, *_ = paged.attention(q[:1, :1], far[:1, :5], v[:1, :5], 5, 0, 1.0)
    assert np.allclose(o3[0, 0], v[0, 0])


def test_attention_rows_before_the_start():
    q, k = np.ones((3, 1, 4)), np.ones((1, 2, 4))
    o, lse, _, _, seen = paged.attention(q, k, k, 2, 0, 1.0)
    assert (o[0] == 0).all() and lse[0, 0] == -np.inf and seen.tolist() == [0, 1, 2]


def test_write_and_gather_are_inverse():
    rng = np.random.default_rng(2)
    cache = rng.standard_normal((7, 2, 8, 3))
    row, k = np.array([4, 0, 6]), rng.standard_normal((20, 2, 3))
    slots = [row[j // 8] * 8 + j % 8 for j in range(20)]
    out = paged.kv_write(k, cache, slots + [])
    assert (paged.gather(out, row, 20) == k.transpose(1, 0, 2)).all()
    left = [i for i in range(7) if i not in (0, 4, 6)]
    assert (out[left] == cache[left]).all() and (out[6, :, 4:] == cache[6, :, 4:]).all()
    assert (paged.kv_write(k[:2], cache, [-1, 56]) == cache).all()
