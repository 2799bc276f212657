"""4-bit caches whose blocks differ in size as far as the format goes, within one tile of keys and across tiles."""
import numpy as np
import pytest
import torch

from _paged_q4 import Q4Batch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CASES = [dict(ctx=[150, 40], new=[1, 1]), dict(ctx=[200, 3], new=[4, 7]), dict(ctx=[100, 10], new=[80, 33])]


def batch(case, dim, dtype, seed):
    return Q4Batch(case["ctx"], case["new"], hq=4, hkv=2, dim=dim, page=16, dtype=dtype, seed=seed)


def rescale(b, change):
    """Puts change(values' scales [tokens, Hkv, D / 32], sequence) in place of the scales of every sequence's values."""
    for i in range(len(b.new)):
        for j in range(b.kv[i]):
            at = (int(b.table[i, j // b.page]), slice(None), j % b.page)
            b.cache[3][at] = change(i, j, b.cache[3][at])
    b.d_cache[3] = torch.from_numpy(b.cache[3]).to(b.device)


def run(gpu_lib, b, **kw):
    o, lse = b.call(gpu_lib, **kw)
    torch.cuda.synchronize()
    b.check(o, lse, **kw)
    return o, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("case", range(3))
def test_scales_of_the_whole_range(gpu_lib, dtype, dim, case):
    """Every block its own power, from the smallest to 2^100 (larger values could pass the sums' range)."""
    b = batch(CASES[case], dim, dtype, dim + case)
    rng = np.random.default_rng(dim)
    rescale(b, lambda i, j, s: rng.integers(1, 228, s.shape))
    run(gpu_lib, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("case", range(3))
def test_columns_of_their_own_size(gpu_lib, dtype, dim, case):
    """One block of columns near 2^90, the next near 2^-90, with zeros' scale among them: the small columns keep all of their bits."""
    b = batch(CASES[case], dim, dtype, dim + case)
    rescale(b, lambda i, j, s: np.where(np.arange(s.shape[-1]) % 2 == 0, s + 90, np.where(j % 7 == 3, 1, s - 90)).astype(np.uint8))
    run(gpu_lib, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("case", range(3))
def test_what_is_not_seen_is_huge(gpu_lib, dtype, dim, window, case):
    """Larger scales, the largest there is, or NaN, in keys that a row does not see (behind the window, later tokens of a chunk): no bit
    of it changes."""
    c = CASES[case]
    b = plain = batch(c, dim, dtype, dim + case)
    want = run(gpu_lib, plain, window=window)
    first = [b.kv[i] - c["new"][i] for i in range(2)]   # the position of a sequence's first row
    hidden = lambda i, j: j > first[i] or (window > 0 and j <= first[i] - window)  # noqa: E731
    for big in (lambda s: s + 25, lambda s: s + 40, lambda s: s + 95, lambda s: 0 * s + 252, lambda s: 0 * s + 255, lambda s: 0 * s + 1):
        b = batch(c, dim, dtype, dim + case)
        rescale(b, lambda i, j, s: big(s) if hidden(i, j) else s)  # noqa: B023
        o, lse = b.call(gpu_lib, window=window)
        for i in range(2):
            row = int(b.cu[i])
            assert torch.equal(o[row], want[0][row]) and torch.equal(lse[row], want[1][row])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(3))
def test_nan_beside_scales_far_apart(gpu_lib, dtype, case):
    b = batch(CASES[case], 128, dtype, 3)
    rng = np.random.default_rng(8)
    odd = {(0, 20), (1, 5), (0, 99)}
    rescale(b, lambda i, j, s: np.where((np.arange(4) == j % 4) & ((i, j) in odd), 255, rng.integers(1, 228, s.shape)).astype(np.uint8))
    o, _ = run(gpu_lib, b)
    assert torch.isnan(o[0]).any() and not torch.isnan(o[0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(3))
def test_keys_of_all_sizes(gpu_lib, dtype, case):
    """Keys' blocks between 2^-60 and 2^60 with queries that make scores of ordinary size of the largest."""
    b = batch(CASES[case], 128, dtype, 4)
    rng = np.random.default_rng(9)
    for i in range(2):
        for j in range(b.kv[i]):
            at = (int(b.table[i, j // b.page]), slice(None), j % b.page)
            b.cache[1][at] = 127 + rng.integers(-60, 61, b.cache[1][at].shape)
    b.d_cache[1] = torch.from_numpy(b.cache[1]).to(b.device)
    run(gpu_lib, b, scale=2.0 ** -61)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(3))
def test_all_values_tiny(gpu_lib, dtype, case):
    """Values near 2^-100: nothing is lost of them."""
    b = batch(CASES[case], 128, dtype, 5)
    rescale(b, lambda i, j, s: s - 100)
    run(gpu_lib, b)
