"""rglru_page_copy with more caches than one launch takes: whatever is wrong with one of them is found before the first is copied."""
import pytest
import torch

import gated_linear_recurrence_amd as glr
from gated_linear_recurrence_amd import _lib, ops

MOST = _lib.RGLRU_PAGE_COPY_ARRAYS


@pytest.fixture
def launches(monkeypatch):
    """Calls that would launch, as (arrays, pairs) in order; the library's own checks run on the others."""
    seen = []

    def call_on(device, fn, where, n_pages, pairs, max_pairs, n_pairs, n, at, sizes):
        if max_pairs:
            seen.append((n, max_pairs))
            return
        _lib.check(fn(n_pages, pairs, 0, n_pairs, n, at, sizes, None), where)

    monkeypatch.setattr(ops, "_call_on", call_on)
    return seen


def caches_and_buffer(n, extra=64):
    """n caches of 4 pages of 64 bytes and a buffer of its own behind them, pieces of one allocation with room between them."""
    size = 4 * 64
    buf = torch.zeros((n + extra) * 2 * size + 16, dtype=torch.uint8)
    buf = buf[-buf.data_ptr() % 16:]
    return [buf[2 * i * size: (2 * i + 1) * size].view(4, 64) for i in range(n)], buf[2 * n * size:]


def pairs_in(c):
    """A [2, 2] tensor of pairs that lies in the second page of a cache."""
    return c.view(-1)[64:80].view(torch.int32).view(2, 2)


@pytest.mark.parametrize("n", [2, MOST, MOST + 1, 2 * MOST + 5])
def test_disjoint_caches_are_copied(launches, n):
    caches, rest = caches_and_buffer(n)
    pairs = torch.zeros(3, 2, dtype=torch.int32)
    glr.rglru_page_copy(pairs, caches[::-1], n_pairs=rest[:4].view(torch.int32))
    assert launches == [(min(MOST, n - i), 3) for i in range(0, n, MOST)]


@pytest.mark.parametrize("n", [MOST + 1, 2 * MOST + 5])
@pytest.mark.parametrize("first", [0, 5, MOST - 1])
@pytest.mark.parametrize("shift", [0, 64, -192])
def test_caches_of_different_launches_that_overlap(launches, n, first, shift):
    caches, rest = caches_and_buffer(n + 1)
    whole = torch.as_strided(caches[0].view(-1), (rest.data_ptr() - caches[0].data_ptr(),), (1,))
    at = caches[first + 1].data_ptr() - caches[0].data_ptr() + shift
    caches[n] = whole[at: at + 256].view(4, 64)
    with pytest.raises(RuntimeError, match="INVALID"):
        glr.rglru_page_copy(torch.zeros(3, 2, dtype=torch.int32), caches)
    assert not launches


@pytest.mark.parametrize("which", [0, MOST - 1, MOST, MOST + 6])
def test_pairs_or_their_number_in_a_cache(launches, which):
    caches, _ = caches_and_buffer(MOST + 7)
    inside = pairs_in(caches[which])
    with pytest.raises(RuntimeError, match="INVALID"):
        glr.rglru_page_copy(inside, caches)
    with pytest.raises(RuntimeError, match="INVALID"):
        glr.rglru_page_copy(torch.zeros(3, 2, dtype=torch.int32), caches, n_pairs=inside.view(-1)[3:])
    assert not launches


def test_no_pairs_overlap_nothing(launches):
    """No pairs are read, so where they would lie does not matter; nothing is launched."""
    caches, _ = caches_and_buffer(MOST + 7)
    glr.rglru_page_copy(pairs_in(caches[MOST])[:0], caches)
    assert not launches


@pytest.mark.gpu
def test_nothing_is_copied_where_the_pairs_lie_in_a_later_cache(gpu_lib):
    caches = [torch.randint(0, 100, (6, 64), dtype=torch.uint8, device="cuda") for _ in range(MOST + 7)]
    pairs = pairs_in(caches[-1])
    pairs.copy_(torch.tensor([[5, 0], [4, 2]], dtype=torch.int32))
    want = [c.clone() for c in caches]
    with pytest.raises(RuntimeError, match="INVALID"):
        gpu_lib.rglru_page_copy(pairs, caches)
    with pytest.raises(RuntimeError, match="INVALID"):
        gpu_lib.rglru_page_copy(pairs.clone(), caches[:-1] + [caches[3]])
    assert all(torch.equal(x, y) for x, y in zip(caches, want))
    gpu_lib.rglru_page_copy(pairs.clone(), caches)
    for w in want:
        w[0], w[2] = w[5].clone(), w[4].clone()
    assert all(torch.equal(x, y) for x, y in zip(caches, want))
