"""Paged attention on values near a type's largest and scores far apart, held to the definition by the strict check."""
import pytest
import torch

from _paged_strict import StrictBatch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def far_keys(new, n, hkv, dim, dtype):
    """Sequences whose keys score 0 but for a few in their second half at some 100 and the last new token's own at some 200.

    So many units that every wave goes from tiles of the first kind to tiles of the second. Column 1 of the values is 1e35 at
    every key of score 0, where its weight is e^-100 at most.
    """
    b = StrictBatch([300 + 7 * i % 90 for i in range(n)], [new] * n, hq=hkv, hkv=hkv, dim=dim, page=16, dtype=dtype, pad=1, seed=dim + new)
    b.q.copy_(b.q.abs() + 0.1)
    b.d_q.copy_(b.q)
    b.d_k.zero_()
    b.d_v[..., 1] = 1e35
    step = 100 / (0.9 * dim ** 0.5)   # the sum of a row of q is some 0.9 D
    for i in range(n):
        b.k[i].zero_()
        b.v[i][..., 1] = 1e35
        for j in range(200, 300, 33):
            b.put(i, j, k=step, v=1.0, dims=slice(None))
            b.put(i, j, v=float(j % 7), dims=slice(2, 9))
        b.put(i, b.kv[i] - 1, k=2 * step)
        b.put(i, b.kv[i] - 1, v=0.5, dims=1)
    return b


CASES = [(1, 130, 4), (3, 90, 4), (70, 36, 8)]
KINDS = [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 128), (F32, 256)]


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("new,n,hkv", CASES)
def test_large_values_of_no_weight_leave_nothing(gpu_lib, dtype, dim, new, n, hkv):
    b = far_keys(new, n, hkv, dim, dtype)
    b.check(*b.call(gpu_lib))
    b.check(*b.call(gpu_lib, window=280), window=280)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("new,n,hkv", CASES)
def test_an_infinite_value_where_the_maximum_grows(gpu_lib, dtype, dim, new, n, hkv):
    """The key that takes all the weight, in a tile that some rows see in part, has infinite values."""
    b = far_keys(new, n, hkv, dim, dtype)
    for i in range(n):
        b.put(i, b.kv[i] - 1, v=(INF, -INF)[i % 2], dims=5)
        b.put(i, b.kv[i] - 1, v=NAN, dims=dim - 1)
        b.put(i, b.kv[i] - 2, v=-INF, dims=7)           # of no weight but for the rows that do not see the last
    b.check(*b.call(gpu_lib))
