"""Few rows over a 4-bit cache: what a row does not see changes no bit of it, however its scales lie to those that the row sees."""
import numpy as np
import pytest
import torch

from _paged_q4 import Q4Batch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# (context, new tokens, window): decode steps, drafts of up to 16 rows and of up to 32, with what lies before a window and with what comes after a row
CASES = [([150, 40], [1, 1], 25), ([200, 3], [4, 7], 0), ([90, 70], [5, 8], 30), ([100, 10], [16, 9], 0)]


def with_scales(case, dim, dtype, change):
    """The case's batch with change(scales of the values, sequence, token) in place of the scales of every token's values."""
    ctx, new, _ = case
    b = Q4Batch(ctx, new, hq=4, hkv=2, dim=dim, page=16, dtype=dtype, seed=dim + sum(new))
    for i in range(len(new)):
        for j in range(b.kv[i]):
            at = (int(b.table[i, j // b.page]), slice(None), j % b.page)
            b.cache[3][at] = change(b.cache[3][at], i, j)
    b.d_cache[3] = torch.from_numpy(b.cache[3]).to(b.device)
    return b


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shift", [0, -14, 16, -22, 23, -40])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_scales_at_every_distance(gpu_lib, dtype, dim, shift, case):
    """Hidden scales 24 to 35 powers above the seen ones, or below them: the seen ones (a few powers) lie across any border that
    hidden ones could draw. `shift` moves all of them."""
    ctx, new, window = CASES[case]
    base = with_scales(CASES[case], dim, dtype, lambda s, i, j: s.astype(int) + shift)
    want = base.call(gpu_lib, window=window)
    base.check(*want, window=window)
    for row in (0, 2) if min(new) > 2 else (0,):
        place = [ctx[i] + row for i in range(len(new))]
        for more in (*range(24, 36), -20, -29):
            hidden = lambda i, j: j > place[i] or (window > 0 and j <= place[i] - window)  # noqa: E731, B023
            b = with_scales(CASES[case], dim, dtype, lambda s, i, j: s.astype(int) + shift + (more if hidden(i, j) else 0))  # noqa: B023
            o, lse = b.call(gpu_lib, window=window)
            for i in range(len(new)):
                at = int(b.cu[i]) + row
                assert torch.equal(o[at], want[0][at]) and torch.equal(lse[at], want[1][at]), (row, more, i)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_across_the_whole_range(gpu_lib, dtype, dim):
    """Seen scales anywhere from 2^-126 to 2^100 beside hidden ones anywhere, NaN among them."""
    case = CASES[1]
    ctx, new, _ = case
    rng = np.random.default_rng(dim)
    seen = {(i, j): rng.integers(1, 228, (2, dim // 32)) for i in range(2) for j in range(ctx[i] + new[i])}
    base = with_scales(case, dim, dtype, lambda s, i, j: seen[i, j])
    want = base.call(gpu_lib)
    base.check(*want)
    for seed in range(8):
        other = np.random.default_rng(seed)
        b = with_scales(case, dim, dtype, lambda s, i, j: seen[i, j] if j <= ctx[i] else other.choice(  # noqa: B023
            [1, 28, 29, 100, 129, 140, 141, 200, 252, 255], (2, dim // 32)))
        o, lse = b.call(gpu_lib)
        for i in range(2):
            at = int(b.cu[i])
            assert torch.equal(o[at], want[0][at]) and torch.equal(lse[at], want[1][at]), (seed, i)
