"""Attention over the 4-bit cache against the float64 reference, row by row."""
import numpy as np
import pytest
import torch

from _paged_q4 import Q4Batch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def run(gpu_lib, batch, **kw):
    window, scale = kw.pop("window", 0), kw.pop("scale", None)
    o, lse = batch.call(gpu_lib, window, scale, **kw)
    torch.cuda.synchronize()
    batch.check(o, lse, window, scale)
    return o, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 8), (4, 4, 16), (8, 2, 32), (10, 1, 64), (16, 1, 16), (24, 3, 128)])
def test_single_tokens(gpu_lib, dtype, dim, hq, hkv, page):
    """Decode steps around the borders of tiles and pages."""
    ctx = [0, 1, 7, 14, 15, 16, 30, 31, 32, 62, 63, 64, 65, 127, 128, 200, 255, 256, 300]
    run(gpu_lib, Q4Batch(ctx, [1] * len(ctx), hq=hq, hkv=hkv, dim=dim, page=page, dtype=dtype, pad=2, seed=dim + hq, spread=2.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [[2, 5, 1, 3, 0, 4], [8, 16, 1, 7, 9, 2], [33, 1, 64, 0, 40, 17]])
def test_a_few_tokens(gpu_lib, dtype, dim, new):
    run(gpu_lib, Q4Batch([0, 33, 100, 5, 64, 129], new, hq=8, hkv=4, dim=dim, page=16, dtype=dtype, pad=3, seed=sum(new), spread=2.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 4, 2), (128, 4, 1), (256, 3, 1)])
@pytest.mark.parametrize("window", [0, 1, 31, 64, 100])
def test_chunks_and_windows(gpu_lib, dtype, dim, hq, hkv, window):
    run(gpu_lib, Q4Batch([0, 150, 3], [130, 77, 1], hq=hq, hkv=hkv, dim=dim, page=32, dtype=dtype, seed=window + dim), window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 50, 700])
def test_long_axis(gpu_lib, dtype, window):
    """Few rows over an axis that is split over many workgroups."""
    run(gpu_lib, Q4Batch([5000, 1, 2777], [1, 1, 2], hq=4, hkv=1, dim=128, page=64, dtype=dtype, seed=3, spread=3.0), window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_sequences(gpu_lib, dtype):
    rng = np.random.default_rng(4)
    new = [1] * 60
    new[17], new[40] = 50, 9
    run(gpu_lib, Q4Batch(rng.integers(0, 200, 60).tolist(), new, hq=6, hkv=2, dim=64, page=8, dtype=dtype, seed=4, pad=7))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", [[0, 3, 40, 1], [2, 0, 5, 64]])
def test_rows_that_see_nothing(gpu_lib, dtype, kv):
    """Fewer keys than new tokens: the first rows stand before the start and give 0 and -inf."""
    b = Q4Batch([0] * 4, [4, 5, 70, 2], hq=4, hkv=2, dim=128, page=16, dtype=dtype, kv_lens=kv, seed=9)
    o, lse = run(gpu_lib, b)
    assert torch.isneginf(lse[: 4 - kv[0]]).all() and (o[: 4 - kv[0]] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_nan_stays_where_it_is_seen(gpu_lib, dtype, dim, new):
    """A key or value that is NaN reaches the rows that see it, a value in its block's columns alone; nothing else moves by a bit."""
    kw = dict(hq=4, hkv=2, dim=dim, page=16, dtype=dtype, seed=dim)
    clean = Q4Batch([150, 40], [new, new], **kw)
    want, want_lse = run(gpu_lib, clean, window=100)
    b = Q4Batch([150, 40], [new, new], **kw)
    b.put(0, 30, k_scale=255, v_scale=255)                  # outside every window
    if new > 2:
        b.put(0, 150 + new - 1, v_scale=255, heads=1, blocks=1)   # seen by the last row alone
        b.put(1, 40 + new - 2, k_scale=255, heads=0, blocks=0)    # by the last two rows
    o, lse = run(gpu_lib, b, window=100)
    same = torch.ones_like(o, dtype=torch.bool)
    same_lse = torch.ones_like(lse, dtype=torch.bool)
    if new > 2:
        assert torch.isnan(o[new - 1, 2:, 32:64]).all() and torch.isnan(o[2 * new - 2:, :2]).all() and torch.isnan(lse[2 * new - 2:, :2]).all()
        same[new - 1, 2:, 32:64] = False
        same[2 * new - 2:, :2] = False
        same_lse[2 * new - 2:, :2] = False
    assert torch.equal(o[same], want[same]) and torch.equal(lse[same_lse], want_lse[same_lse])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 70])
def test_queries_that_are_not_finite(gpu_lib, dtype, new):
    """An infinity or NaN in a query makes that row NaN (a code of 0 times an infinity is), and no other."""
    b = Q4Batch([90], [new + 1], hq=2, hkv=1, dim=128, page=16, dtype=dtype, seed=1)
    for at, x in ((0, float("inf")), (1, float("nan"))):
        b.d_q[0, at, 3], b.q[0, at, 3] = x, x
    o, lse = b.call(gpu_lib)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(o[1:]).all() and torch.isfinite(lse[1:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [-60, 40])
def test_blocks_of_extreme_powers(gpu_lib, dtype, power):
    """Keys and values scaled by 2^power, the scale of the scores by 2^-power: weights and outputs as they are."""
    b = Q4Batch([100, 30], [1, 40], hq=4, hkv=2, dim=64, page=16, dtype=dtype, seed=6)
    for which in (1, 3):
        live = b.cache[which] != 255
        b.cache[which] = np.where(live, b.cache[which].astype(int) + power, 255).astype(np.uint8)
        b.d_cache[which] = torch.from_numpy(b.cache[which]).cuda()
    run(gpu_lib, b, scale=0.125 * 2.0 ** -power)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [3, 60])
@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_scales(gpu_lib, dtype, new, scale):
    run(gpu_lib, Q4Batch([70], [new], hq=2, hkv=1, dim=64, page=8, dtype=dtype, seed=2), scale=scale)


def test_rows_of_a_wider_tensor_and_no_lse(gpu_lib):
    b = Q4Batch([40, 9], [3, 20], hq=4, hkv=2, dim=128, page=16, q_extra=64, seed=7)
    o, lse = run(gpu_lib, b)
    o2, none = gpu_lib.rglru_paged_attn_q4_fwd(b.d_q, *b.d_cache, b.d_table, b.d_cu, b.d_kv, want_lse=False)
    assert none is None and torch.equal(o2[: b.tokens], o[: b.tokens])


def test_max_new_not_known(gpu_lib):
    b = Q4Batch([40, 9, 300], [3, 1, 2], hq=4, hkv=2, dim=128, page=16, seed=17, pad=4)
    run(gpu_lib, b, max_new=0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_same_bits_each_time(gpu_lib, dtype):
    b = Q4Batch([3000, 10, 900], [1, 60, 5], hq=8, hkv=2, dim=128, page=32, dtype=dtype, seed=12)
    first = b.call(gpu_lib)
    for _ in range(5):
        again = b.call(gpu_lib)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_workspace_of_any_contents(gpu_lib):
    b = Q4Batch([700, 10], [1, 90], hq=8, hkv=2, dim=128, page=32, seed=13)
    want = b.call(gpu_lib)
    for fill in (0, 255, 127):
        ws = torch.full((192 << 20,), fill, dtype=torch.uint8, device="cuda")
        got = b.call(gpu_lib, workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("new", [[1, 1, 1], [60, 1, 7]])
def test_captured_and_replayed_with_other_lengths(gpu_lib, new):
    b = Q4Batch([200, 31, 90], new, hq=4, hkv=2, dim=128, page=16, seed=21, pad=5)
    ws = torch.empty(192 << 20, dtype=torch.uint8, device="cuda")
    o = torch.full((b.q.shape[0], 4, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((b.q.shape[0], 4), 7.0, device="cuda")
    args = (b.d_q, *b.d_cache, b.d_table, b.d_cu, b.d_kv)
    kw = dict(max_new=max(new), workspace=ws, o=o, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.rglru_paged_attn_q4_fwd(*args, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.rglru_paged_attn_q4_fwd(*args, **kw)
    for kv in ([200 + new[0], 31 + new[1], 90 + new[2]], [100, 12, 91], [61, 2, 7]):
        b.kv = kv
        b.d_kv.copy_(torch.tensor(kv, dtype=torch.int32))
        o.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        b.check(o, lse)
        want = b.call(gpu_lib)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_past_32_bit_offsets(gpu_lib):
    """Pages whose codes lie behind 2^32 bytes."""
    b = Q4Batch([70, 20], [1, 40], hq=2, hkv=1, dim=128, page=1024, seed=5, spare=0)
    n_pages = (1 << 32) // (1024 * 64) + 8
    base = n_pages - b.cache[0].shape[0]
    for c in range(4):
        big = torch.zeros(n_pages, *b.cache[c].shape[1:], dtype=torch.uint8, device="cuda")
        big[base:] = b.d_cache[c]
        b.d_cache[c] = big
    b.d_table += base
    o, lse = b.call(gpu_lib)
    b.check(o, lse)


def test_on_another_stream(gpu_lib):
    b = Q4Batch([200, 31], [1, 40], hq=4, hkv=2, dim=64, page=16, seed=23)
    want = b.call(gpu_lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.call(gpu_lib)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
