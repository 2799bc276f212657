"""Fork, free, compact and copy of a page pool against the reference: equal, entry by entry."""
import numpy as np
import pytest
import torch

from _pool import check_pool, random_pool
from oracle import page_pool as pool

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def on_gpu(s):
    return dict(table=i32(s["table"]), held=i32(s["held"]), shares=i32(s["shares"]), free=i32(s["free"]), count=i32([s["count"]]))


def same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1))


SIZES = [  # rows, tokens a page, most tokens, spare pages
    (1, 8, 1, 0), (1, 8, 50, 3), (2, 16, 40, 1), (5, 8, 30, 2), (64, 16, 300, 9), (70, 8, 900, 40), (300, 8, 200, 0), (1030, 16, 100, 50),
    (3, 8, 40000, 7), (2100, 8, 20, 300)]


@pytest.mark.parametrize("n,page,most,spare", SIZES)
def test_fork(gpu_lib, n, page, most, spare):
    rng = np.random.default_rng(n + most)
    s = random_pool(rng, n=n, page=page, most=most, spare=spare, empty=0.5)
    # anything at all: rows that are not empty, sources that are forked, themselves or not there
    src = np.where(rng.random(n) < 0.8, rng.integers(0, n, n), rng.integers(-3, n + 3, n))
    src[s["held"] > 0] = np.where(rng.random((s["held"] > 0).sum()) < 0.95, -1, src[s["held"] > 0])
    lens = np.maximum(s["held"] - rng.integers(0, 5, n) * (rng.random(n) < 0.3), 0)   # some hold drafts beyond
    want = pool.fork(src, lens, s["held"], s["table"], s["shares"], s["free"], s["count"], page)
    d = on_gpu(s)
    pairs, lens_out, held_out, count, unserved = gpu_lib.rglru_page_fork(
        i32(src), i32(lens), d["table"], d["shares"], d["free"], d["count"], page_size=page, held_lens=d["held"])
    for got, name in ((pairs, "pairs"), (lens_out, "lens_out"), (held_out, "held_lens_out"), (count, "free_count_out"),
                      (unserved, "unserved"), (d["table"], "block_table"), (d["shares"], "shares")):
        same(got, want[name])
    same(d["free"], s["free"])


@pytest.mark.parametrize("n,page,most,spare", SIZES)
def test_free(gpu_lib, n, page, most, spare):
    rng = np.random.default_rng(n + most + 1)
    s = random_pool(rng, n=n, page=page, most=most, spare=spare)
    keep = np.where(rng.random(n) < 0.4, rng.integers(-2, most + 3, n), np.where(rng.random(n) < 0.5, 0, s["held"]))
    want = pool.free(keep, s["held"], s["table"], s["shares"], s["free"], s["count"], page)
    d = on_gpu(s)
    held, count = gpu_lib.rglru_page_free(i32(keep), d["held"], d["table"], d["shares"], d["free"], d["count"], page_size=page)
    for got, name in ((held, "held_lens_out"), (count, "free_count_out"), (d["shares"], "shares"), (d["free"], "free_pages")):
        same(got, want[name])
    same(d["table"], s["table"])
    check_pool(dict(s, held=want["held_lens_out"], shares=want["shares"], free=want["free_pages"], count=want["free_count_out"]), page)


@pytest.mark.parametrize("n,page,most,spare", SIZES)
@pytest.mark.parametrize("part", [0.0, 0.3, 0.5, 0.9, 1.0])
def test_compact(gpu_lib, n, page, most, spare, part):
    rng = np.random.default_rng(n + most + 2)
    s = random_pool(rng, n=n, page=page, most=most, spare=spare)
    n_pages = len(s["free"])
    if s["count"] > 3:
        s["count"] -= 2   # two pages are the caller's own: neither held nor free
    keep = int(part * n_pages)
    want = pool.compact(s["held"], s["table"], s["shares"], s["free"], s["count"], page, keep)
    d = on_gpu(s)
    got = gpu_lib.rglru_page_compact(d["held"], d["table"], d["shares"], d["free"], d["count"], page_size=page, keep_pages=keep)
    for x, name in zip(got, ("block_table_out", "shares_out", "free_pages_out", "free_count_out", "pairs", "n_pairs", "unmoved")):
        same(x, want[name])
    for x, name in ((d["table"], "table"), (d["shares"], "shares"), (d["free"], "free")):
        same(x, s[name])


@pytest.mark.parametrize("shape,dtype", [((2, 8, 64), torch.bfloat16), ((8, 16, 4), torch.uint8), ((3, 64, 128), torch.float32), ((1, 8, 2), torch.uint8)])
def test_copy(gpu_lib, shape, dtype):
    rng = np.random.default_rng(len(shape))
    n_pages = 50
    caches = [torch.from_numpy(rng.integers(0, 100, (n_pages, *shape))).to(dtype).cuda(),
              torch.from_numpy(rng.integers(0, 100, (n_pages, 16))).to(torch.uint8).cuda()]
    order = rng.permutation(n_pages)
    pairs = np.stack([order[:20], order[20:40]], 1).astype(np.int32)
    pairs[3], pairs[5], pairs[7] = (-1, -1), (n_pages, 4), (order[45], -1)
    for count in (None, 0, 13, 99):
        want = [pool.copy(pairs, c.float().cpu().numpy(), count) for c in caches]
        work = [c.clone() for c in caches]
        gpu_lib.rglru_page_copy(i32(pairs), work, n_pairs=None if count is None else i32([count]))
        for x, y in zip(work, want):
            same(x.float(), y)


def test_copy_of_many_caches_and_none(gpu_lib):
    """More caches than one launch takes, of pages larger than a workgroup's piece; and no pairs at all."""
    caches = [torch.randn(6, 5000 + 4 * i, device="cuda") for i in range(130)]
    want = [c.clone() for c in caches]
    gpu_lib.rglru_page_copy(torch.empty(0, 2, dtype=torch.int32, device="cuda"), caches)
    assert all(torch.equal(x, y) for x, y in zip(caches, want))
    gpu_lib.rglru_page_copy(i32([[5, 0], [1, 2]]), caches)
    for w in want:
        w[0], w[2] = w[5].clone(), w[1].clone()
    assert all(torch.equal(x, y) for x, y in zip(caches, want))


def test_nothing_is_copied_where_a_cache_is_refused(gpu_lib):
    """The last of more caches than one launch takes is not aligned: the call raises and leaves all of them."""
    caches = [torch.randn(6, 64, device="cuda") for _ in range(70)]
    want = [c.clone() for c in caches]
    odd = torch.zeros(6 * 64 + 1, device="cuda")[1:].view(6, 64)
    with pytest.raises(RuntimeError, match="align"):
        gpu_lib.rglru_page_copy(i32([[5, 0]]), caches + [odd])
    assert all(torch.equal(x, y) for x, y in zip(caches, want)) and not bool(odd.any())


def test_rows_that_go_back_share_to_the_end_of_a_page(gpu_lib):
    """Two rows share a prompt; both go back to a page's end and go on: fresh pages for the new tokens, the others stay shared."""
    page, width, n_pages = 16, 8, 20
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = i32([3, 4, 5, 6, 7])
    shares, free = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), i32(list(range(19, 7, -1)) + [0] * 8)
    _, lens, held, count, unserved = gpu_lib.rglru_page_fork(i32([-1, 0]), i32([80, 0]), table, shares, free, i32([12]), page_size=page)
    assert lens.tolist() == [80, 80] and int(unserved) == 0 and shares[3:8].tolist() == [1] * 5
    held, count = gpu_lib.rglru_page_free(i32([48, 32]), held, table, shares, free, count, page_size=page)
    assert held.tolist() == [48, 32] and shares[3:8].tolist() == [1, 1, 0, 0, 0] and int(count) == 14
    slots, _, kv, held, count, unserved = gpu_lib.rglru_page_plan(held, i32([0, 3, 6]), table, free, count, n_tokens=6, page_size=page,
                                                                  held_lens=held)
    assert int(unserved) == 0 and kv.tolist() == [51, 35]
    at = (slots // page).tolist()
    assert len(set(at)) == 2 and not set(at) & {3, 4, 5} and table[:, :3].tolist() == [[3, 4, 5], [3, 4, at[3]]]


def test_copy_past_32_bit_offsets(gpu_lib):
    cache = torch.zeros(70, 1 << 26, dtype=torch.uint8, device="cuda")
    cache[69].fill_(3)
    cache[68, -1] = 9
    gpu_lib.rglru_page_copy(i32([[69, 1], [68, 66]]), [cache])
    assert bool((cache[1] == 3).all()) and int(cache[66, -1]) == 9 and not bool(cache[0].any()) and not bool(cache[2].any())


def test_lengths_and_entries_that_make_no_sense(gpu_lib):
    """What is in the arrays is anything at all: every access stays in bounds and the calls end."""
    rng = np.random.default_rng(0)
    n, width, n_pages, page = 40, 9, 100, 8
    wild = lambda *s: i32(rng.integers(-2 ** 31, 2 ** 31, s))  # noqa: E731
    guard = [torch.full((4096,), 11, dtype=torch.int32, device="cuda") for _ in range(2)]
    for _ in range(3):
        pairs = gpu_lib.rglru_page_fork(i32(rng.integers(-5, n + 5, n)), wild(n), wild(n, width), wild(n_pages), wild(n_pages), wild(1),
                                        page_size=page, held_lens=i32(rng.integers(0, 2, n)))[0]
        gpu_lib.rglru_page_free(wild(n), wild(n), wild(n, width), wild(n_pages), wild(n_pages), wild(1), page_size=page)
        out = gpu_lib.rglru_page_compact(wild(n), wild(n, width), wild(n_pages), wild(n_pages), wild(1), page_size=page, keep_pages=50)
        cache = torch.zeros(n_pages, 16, dtype=torch.uint8, device="cuda")
        gpu_lib.rglru_page_copy(pairs, [cache])
        gpu_lib.rglru_page_copy(out[4], [cache], n_pairs=wild(1))
    torch.cuda.synchronize()
    assert all(bool((g == 11).all()) for g in guard)


def test_replays_with_other_lengths(gpu_lib):
    """A captured step of all four operations, replayed over other pools."""
    n, page, width, n_pages = 24, 8, 30, 400
    rng = np.random.default_rng(11)

    def fresh():
        s = random_pool(rng, n=n, page=page, most=200, spare=0, empty=0.5, width=width)
        used = len(s["free"])
        extra = np.arange(used, n_pages)
        s["shares"] = np.concatenate([s["shares"], 0 * extra]).astype(np.int32)
        s["free"] = np.concatenate([s["free"][: s["count"]], rng.permutation(extra), np.zeros(n_pages)]).astype(np.int32)[:n_pages]
        s["count"] += len(extra)
        src = np.where((s["held"] == 0) & (s["held"].max() > 0), int(s["held"].argmax()), -1)
        keep = np.where(rng.random(n) < 0.5, 0, s["held"])
        return s, src, keep

    s, src, keep = fresh()
    d = on_gpu(s)
    d_src, d_keep = i32(src), i32(keep)
    cache = torch.randint(0, 100, (n_pages, 64), dtype=torch.uint8, device="cuda")
    space = [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step():
        pairs, lens, held, count, unserved = gpu_lib.rglru_page_fork(d_src, d["held"], d["table"], d["shares"], d["free"], d["count"], page_size=page)
        gpu_lib.rglru_page_copy(pairs, [cache])
        kept, count2 = gpu_lib.rglru_page_free(d_keep, held, d["table"], d["shares"], d["free"], count, page_size=page, workspace=space[0])
        out = gpu_lib.rglru_page_compact(kept, d["table"], d["shares"], d["free"], count2, page_size=page, keep_pages=n_pages // 2, workspace=space[1])
        gpu_lib.rglru_page_copy(out[4], [cache], n_pairs=out[5])
        return (pairs, held, kept, count2, *out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        s, src, keep = fresh()
        for name, x in on_gpu(s).items():
            d[name].copy_(x)
        d_src.copy_(i32(src)), d_keep.copy_(i32(keep))
        before = cache.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        f = pool.fork(src, s["held"], s["held"], s["table"], s["shares"], s["free"], s["count"], page)
        g = pool.free(keep, f["held_lens_out"], f["block_table"], f["shares"], s["free"], f["free_count_out"], page)
        c = pool.compact(g["held_lens_out"], f["block_table"], g["shares"], g["free_pages"], g["free_count_out"], page, n_pages // 2)
        for x, w in zip(got, (f["pairs"], f["held_lens_out"], g["held_lens_out"], g["free_count_out"], *c.values())):
            same(x, w)
        same(cache, pool.copy(c["pairs"], pool.copy(f["pairs"], before), c["n_pairs"]))
