"""Pools on both sides of what one launch takes: many pages, long rows, many chunks; and anything at all in the arrays, with every output
between guards."""
import numpy as np
import pytest
import torch

from _pool import random_pool
from oracle import page_pool as pool

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1))


# rows, tokens a page, most tokens, spare pages, pages of the pool before those (None: as many as the rows hold) or columns of the table
SIZES = {
    "long rows": (24, 8, 16000, 50, None),                    # slices past the first, several launches
    "very long rows": (5, 8, 80000, 3, None),
    "2^13 pages": (40, 8, 400, 0, 1 << 13),                   # the last pool of one launch of free
    "2^13 + 1 pages": (40, 8, 400, 1, 1 << 13),
    "2^15 pages": (40, 8, 400, 0, 1 << 15),                   # the last pool of one launch of compact
    "2^15 + 1 pages": (40, 8, 400, 1, 1 << 15),
    "2^14 entries": (16, 8, 4000, 20, "1024 columns"),        # as many as one launch of free takes
    "more than 2^14 entries": (16, 8, 4000, 20, "1025 columns"),
    "2^15 entries": (32, 8, 6000, 20, "1024 columns"),        # as many as one launch of compact takes
    "more than 2^15 entries": (32, 8, 6000, 20, "1025 columns"),
    "33 000 free pages": (9, 8, 100, 33000, None),
    "2^17 pages": (40, 8, 400, 0, 1 << 17),
    "2^17 + 1 pages": (40, 8, 400, 1, 1 << 17),
    "530 000 pages": (30, 8, 4000, 530000, None),             # more than 256 chunks
    "64 rows": (64, 8, 600, 5, None),                         # the most rows of one launch of free
    "65 rows": (65, 8, 600, 5, None),
    "2048 rows": (2048, 8, 50, 5, None),                      # of compact
    "2049 rows": (2049, 8, 50, 5, None),
}


def pool_of(name, rng):
    n, page, most, spare, size = SIZES[name]
    if isinstance(size, int):
        s = random_pool(rng, n=n, page=page, most=most, spare=0)
        more = size + spare - len(s["free"])
        extra = len(s["free"]) + rng.permutation(more)
        s["shares"] = np.concatenate([s["shares"], np.zeros(more, np.int32)])
        s["free"] = np.concatenate([s["free"][: s["count"]], extra, np.full(len(s["free"]) - s["count"], -7)]).astype(np.int32)
        s["count"] += more
        return s, page, most
    return random_pool(rng, n=n, page=page, most=most, spare=spare, width=size and int(size.split()[0])), page, most


@pytest.mark.parametrize("name", SIZES)
def test_free(gpu_lib, name):
    rng = np.random.default_rng(len(name))
    s, page, most = pool_of(name, rng)
    n = len(s["held"])
    keep = np.where(rng.random(n) < 0.4, rng.integers(-2, most + 3, n), np.where(rng.random(n) < 0.5, 0, s["held"]))
    want = pool.free(keep, s["held"], s["table"], s["shares"], s["free"], s["count"], page)
    shares, free = i32(s["shares"]), i32(s["free"])
    held, count = gpu_lib.rglru_page_free(i32(keep), i32(s["held"]), i32(s["table"]), shares, free, i32([s["count"]]), page_size=page)
    for got, x in ((held, "held_lens_out"), (count, "free_count_out"), (shares, "shares"), (free, "free_pages")):
        same(got, want[x])


@pytest.mark.parametrize("part", [0.2, 0.5, 0.95])
@pytest.mark.parametrize("name", SIZES)
def test_compact(gpu_lib, name, part):
    rng = np.random.default_rng(len(name) + 1)
    s, page, _ = pool_of(name, rng)
    keep = int(part * len(s["free"]))
    want = pool.compact(s["held"], s["table"], s["shares"], s["free"], s["count"], page, keep)
    got = gpu_lib.rglru_page_compact(i32(s["held"]), i32(s["table"]), i32(s["shares"]), i32(s["free"]), i32([s["count"]]), page_size=page,
                                     keep_pages=keep)
    for x, y in zip(got, ("block_table_out", "shares_out", "free_pages_out", "free_count_out", "pairs", "n_pairs", "unmoved")):
        same(x, want[y])


@pytest.mark.parametrize("name", ["long rows", "very long rows", "2^17 + 1 pages", "2049 rows"])
def test_fork(gpu_lib, name):
    rng = np.random.default_rng(len(name) + 2)
    s, page, _ = pool_of(name, rng)
    n = len(s["held"])
    src = np.where((s["held"] == 0) & (rng.random(n) < 0.8), rng.integers(0, n, n), -1)
    want = pool.fork(src, s["held"], s["held"], s["table"], s["shares"], s["free"], s["count"], page)
    table, shares = i32(s["table"]), i32(s["shares"])
    got = gpu_lib.rglru_page_fork(i32(src), i32(s["held"]), table, shares, i32(s["free"]), i32([s["count"]]), page_size=page)
    for x, y in zip((*got, table, shares), ("pairs", "lens_out", "held_lens_out", "free_count_out", "unserved", "block_table", "shares")):
        same(x, want[y])


class Guarded:
    """Arrays cut out of one buffer, 64 words of guards around each."""
    WORD = 0x5A5A5A5A

    def __init__(self, words):
        self.buf = torch.full((words,), self.WORD, dtype=torch.int32, device="cuda")
        self.taken, self.at = torch.zeros(words, dtype=torch.bool, device="cuda"), 64

    def __call__(self, *shape, like=None):
        size = int(np.prod(shape))
        part = self.buf[self.at: self.at + size]
        self.taken[self.at: self.at + size] = True
        self.at = (self.at + size + 64 + 3) // 4 * 4   # a workspace may be next
        assert self.at <= self.buf.numel()
        if like is not None:
            part.copy_(like.reshape(-1))
        return part.view(shape)

    def check(self):
        assert bool((self.buf[~self.taken] == self.WORD).all())


@pytest.mark.parametrize("n,width,n_pages", [(40, 9, 100), (3, 5, 40000), (2100, 20, 3000), (33, 1100, 9000), (7, 3, 140000)])
def test_anything_at_all_in_the_arrays(gpu_lib, n, width, n_pages):
    """Lengths, entries, counts and pairs of any value, small ones that pass some of the checks among them: nothing beside the outputs
    is written."""
    rng = np.random.default_rng(n + width)
    page = 8

    def wild(*s):
        some = rng.integers(0, 4, s)
        near, far = rng.integers(-3, 3 + max(n_pages, n, width * page), s), rng.integers(-2 ** 31, 2 ** 31, s)
        return i32(np.where(some == 0, far, np.where(some == 1, 0, near)))

    for _ in range(3):
        g = Guarded(8 * n * width + 40 * n_pages + 40 * n + 20000)
        table, shares = g(n, width, like=wild(n, width)), g(n_pages, like=wild(n_pages))
        pairs = gpu_lib.rglru_page_fork(wild(n), wild(n), table, shares, wild(n_pages), wild(1), page_size=page, held_lens=wild(n),
                                        pairs=g(n, 2), lens_out=g(n), held_lens_out=g(n), free_count_out=g(1), unserved=g(1))[0]
        words = [gpu_lib.ops._pool_bytes(f"rglru_page_{x}_workspace_bytes", n_pages, n, width, page) // 4 for x in ("free", "compact")]
        gpu_lib.rglru_page_free(wild(n), wild(n), table, g(n_pages, like=wild(n_pages)), g(n_pages, like=wild(n_pages)), wild(1), page_size=page,
                                held_lens_out=g(n), free_count_out=g(1), workspace=g(words[0]).view(torch.uint8))
        keep = int(rng.integers(0, n_pages + 1))
        room = min(keep, n_pages - keep)
        out = gpu_lib.rglru_page_compact(wild(n), wild(n, width), wild(n_pages), wild(n_pages), wild(1), page_size=page, keep_pages=keep,
                                         block_table_out=g(n, width), shares_out=g(n_pages), free_pages_out=g(n_pages), free_count_out=g(1),
                                         pairs=g(room, 2), n_pairs=g(1), unmoved=g(1), workspace=g(words[1]).view(torch.uint8))
        caches = [g(n_pages, 4, like=torch.zeros(n_pages, 4, dtype=torch.int32, device="cuda")) for _ in range(2)]
        gpu_lib.rglru_page_copy(pairs.clone(), caches)
        gpu_lib.rglru_page_copy(wild(50, 2), caches, n_pairs=wild(1))
        gpu_lib.rglru_page_copy(out[4].clone(), caches, n_pairs=wild(1))
        torch.cuda.synchronize()
        g.check()
