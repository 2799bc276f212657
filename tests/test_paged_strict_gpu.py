"""Paged attention where answers are infinite, NaN or empty, held to the definition by the strict check."""
import pytest
import torch

from _paged_strict import StrictBatch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,hq", [(1, 2), (6, 10), (50, 2)])
def test_infinities_keep_their_sign_and_place(gpu_lib, dtype, dim, new, hq):
    """Infinite values and NaN in columns all over a row, in a tile that some rows see in part and in one that all do."""
    b = StrictBatch([700], [new], hq=hq, hkv=2, dim=dim, page=16, dtype=dtype, seed=dim + new)
    for x in range(dim // 32):
        b.put(0, 700 + new // 2, v=(INF, -INF)[x % 2], dims=32 * x + 5 * x % 32)
    b.put(0, 320, v=INF, dims=dim - 1)
    b.put(0, 321, v=-INF, dims=dim - 2)
    b.put(0, 700 + new - 1, v=NAN, dims=dim // 2)
    b.put(0, 699, v=NAN, heads=1, dims=0)
    b.put(0, 330, v=INF, dims=1)              # both signs: NaN
    b.put(0, 700, v=-INF, dims=1)
    b.check(*b.call(gpu_lib))
    b.check(*b.call(gpu_lib, window=9), window=9)


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 256)])
@pytest.mark.parametrize("new", [1, 5, 80])
def test_rows_before_the_start(gpu_lib, dtype, dim, new):
    """More new tokens than the cache holds: o = 0 and lse = -inf in every sequence's first rows. Lengths of zero."""
    b = StrictBatch([0] * 4, [new] * 4, hq=4, hkv=2, dim=dim, page=16, dtype=dtype, kv_lens=[0, max(new - 1, 0), new, new + 3], pad=2,
                    seed=new)
    b.check(*b.call(gpu_lib))
    b.check(*b.call(gpu_lib, window=2), window=2)


def test_many_empty_rows_in_a_batch(gpu_lib):
    b = StrictBatch([0] * 40, [3, 1, 0, 120] * 10, hq=4, hkv=1, dim=64, page=16, kv_lens=[i % 7 * (i % 4) for i in range(40)], pad=4, seed=6)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("new", [1, 50])
def test_infinite_columns_of_split_rows(gpu_lib, new):
    """Infinite values in pieces of a row that the join merges."""
    b = StrictBatch([9000, 3000], [new, new], hq=4, hkv=1, dim=128, page=64, seed=new)
    for j, d in ((3, 0), (4000, 1), (8990, 2)):
        b.put(0, j, v=INF, dims=d)
        b.put(0, j + 1, v=-INF, dims=d + 8)
        b.put(0, j, v=NAN, dims=d + 16)
    b.put(1, 2999, v=-INF, dims=5)
    b.check(*b.call(gpu_lib))


KINDS = [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 128), (F32, 256)]


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("ctx,new,n,heads", [(20, 1, 1, 1), (20, 60, 1, 1), (9000, 1, 1, 1), (9000, 60, 1, 1), (20, 1, 70, 4), (20, 60, 36, 8)])
def test_no_weights_over_values_that_are_not_finite(gpu_lib, dtype, dim, ctx, new, n, heads):
    """All scores -inf: o = 0 and lse = -inf whatever the values are, in cut units and (of many) in whole ones."""
    b = StrictBatch([ctx] * n + [5], [new] * (n + 1), hq=heads, hkv=heads, dim=dim, page=64, dtype=dtype, seed=dim + new)
    b.q.copy_(b.q.abs() + 0.1)
    b.d_q.copy_(b.q)
    for i in range(n):
        b.d_k[b.d_table[i].long()] = -INF
        b.k[i].fill_(-INF)
        for j, d in ((3, 0), (ctx // 2, 1), (ctx - 1, 2)):
            b.put(i, j, v=INF, dims=d)
            b.put(i, j + 1, v=-INF, dims=d + 8)
            b.put(i, j, v=NAN, dims=d + 16)
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    assert (o[: n * new] == 0).all() and (lse[: n * new] == -INF).all()
    b.check(*b.call(gpu_lib, window=7), window=7)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("ctx,n", [(250, 70), (9000, 2)])
def test_values_that_are_not_finite_at_scores_of_minus_infinity(gpu_lib, dtype, dim, new, ctx, n):
    """The first half of the keys scores -inf and has infinite values: their weight of 0 gives infinity or NaN, never a number,
    whichever wave or piece of the row they fell to."""
    b = StrictBatch([ctx] * n, [new] * n, hq=2, hkv=2, dim=dim, page=64, dtype=dtype, seed=dim + new)
    b.q.copy_(b.q.abs() + 0.1)
    b.d_q.copy_(b.q)
    pages = ctx // 2 // 64
    for i in range(n):
        b.d_k[b.d_table[i, :pages].long()] = -INF
        b.k[i][: pages * 64].fill_(-INF)
        for j, d in ((3, 0), (40, 1), (pages * 64 - 1, 2)):
            b.put(i, j, v=INF, dims=d)
            b.put(i, j, v=-INF, dims=d + 8)
            b.put(i, j, v=NAN, dims=d + 16)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("new", [1, 7, 70])
def test_rows_aligned_to_16_bytes_and_no_more(gpu_lib, dtype, dim, new):
    """Queries that start 16 bytes into wider rows of an odd number of 16-byte pieces, the outputs and the log-sum-exps of a like kind."""
    b = StrictBatch([90, 300], [new, new], hq=6, hkv=2, dim=dim, page=16, dtype=dtype, pad=2, seed=new)
    one = 16 // b.d_q.element_size()
    rows = b.q.shape[0]
    wide = torch.full((rows, 6 * dim + 3 * one), NAN, dtype=dtype, device="cuda")
    q = wide[:, one:one + 6 * dim].unflatten(1, (6, dim))
    q.copy_(b.q)
    o = torch.full((rows * 6 * dim + one,), 7.0, dtype=dtype, device="cuda")[one:].view(rows, 6, dim)
    lse = torch.full((rows * 6 + 1,), 7.0, device="cuda")[1:].view(rows, 6)
    assert q.data_ptr() % 32 == o.data_ptr() % 32 == 16 and q.stride(0) * q.element_size() % 32 == 16
    gpu_lib.rglru_paged_attn_fwd(q, b.d_k, b.d_v, b.d_table, b.d_cu, b.d_kv, o=o, lse=lse)
    b.check(o, lse)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 8), (16, 4)])
@pytest.mark.parametrize("n", [2, 6, 16, 19])
def test_single_tokens_beside_chunks(gpu_lib, dtype, dim, hq, hkv, n):
    """Batches on both sides of the rules by which the two kernels share a call, with the bound on new tokens and without it; in a
    workspace of the largest call."""
    new = [90 if i % 7 == 1 else 2 if i % 5 == 4 else 1 for i in range(n)]
    b = StrictBatch([150 + 11 * i for i in range(n)], new, hq=hq, hkv=hkv, dim=dim, page=16, dtype=dtype, pad=5, seed=n)
    ws = torch.full((160 << 20,), 255, dtype=torch.uint8, device="cuda")
    for kw in (dict(max_new=90), dict(max_new=0), dict(max_new=b.q.shape[0])):
        b.check(*b.call(gpu_lib, workspace=ws, **kw))
    b.check(*b.call(gpu_lib, window=33, workspace=ws), window=33)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("ctx,new", [(70, 1), (70, 60), (9000, 4), (9000, 60)])
def test_scores_of_infinity_and_nan(gpu_lib, dtype, dim, bad, ctx, new):
    """A score of +inf or NaN makes o and lse of its row NaN; rows that do not see that key are as without it."""
    b = StrictBatch([ctx, 33], [new, new], hq=2, hkv=1, dim=dim, page=64, dtype=dtype, seed=dim + new)
    b.q.copy_(b.q.abs() + 0.1)
    b.d_q.copy_(b.q)
    b.put(0, ctx + new // 2, k=bad)
    b.put(0, 5, v=INF, dims=1)
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    assert torch.isnan(o[new // 2:new]).all() and torch.isnan(lse[new // 2:new]).all()
    b.put(1, 7, k=bad)            # out of every row's window
    b.check(*b.call(gpu_lib, window=20), window=20)
