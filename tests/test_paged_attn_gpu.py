"""Paged attention against the float64 oracle, element by element, with bounds derived from the arithmetic (tests/_paged.py)."""
import numpy as np
import pytest
import torch

from _paged import Batch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (10, 1), (12, 4), (16, 1), (6, 2)])
def test_single_tokens(gpu_lib, dtype, dim, hq, hkv):
    b = Batch([0, 1, 31, 32, 33, 100, 257, 512], [1] * 8, hq=hq, hkv=hkv, dim=dim, page=16, dtype=dtype, pad=3, seed=dim + hq)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 7, 64, 100])
def test_chunks(gpu_lib, dtype, dim, window):
    b = Batch([0, 3, 64, 130, 0, 5], [1, 70, 0, 33, 129, 64], hq=4, hkv=2, dim=dim, page=32, dtype=dtype, pad=9, seed=window)
    b.check(*b.call(gpu_lib, window=window), window=window)


@pytest.mark.parametrize("page", [8, 16, 64, 256, 1024])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_page_sizes(gpu_lib, page, new):
    b = Batch([page - 1, page, 2 * page + 5, 40], [new] * 4, hq=8, hkv=2, dim=128, page=page, seed=page + new)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("hq,hkv,new", [(5, 1, 2), (5, 1, 77), (10, 2, 30), (24, 8, 20), (128, 1, 3), (33, 1, 1), (40, 1, 40), (300, 1, 2)])
def test_groups(gpu_lib, hq, hkv, new):
    """Head groups that do not divide a tile, and groups longer than one."""
    b = Batch([200, 0, 17], [new, new, 1], hq=hq, hkv=hkv, dim=64, page=16, seed=hq)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("window", [0, 300, 1500])
def test_long_axis(gpu_lib, window):
    """Few rows over a long axis: the work is split along it and joined."""
    b = Batch([5003, 9000, 2], [1, 2, 1], hq=8, hkv=2, dim=128, page=64, seed=3)
    b.check(*b.call(gpu_lib, window=window), window=window)
    b = Batch([5003], [40], hq=8, hkv=1, dim=128, page=64, seed=4)
    b.check(*b.call(gpu_lib, window=window), window=window)


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 128), (BF, 256), (F32, 128)])
def test_long_chunk(gpu_lib, dtype, dim):
    """A chunk that fills many tiles; a few sequences of one token beside it."""
    b = Batch([0, 700, 1, 90], [600, 1, 1, 3], hq=4, hkv=1, dim=dim, page=16, dtype=dtype, pad=2, seed=dim)
    b.check(*b.call(gpu_lib))
    b.check(*b.call(gpu_lib, window=129), window=129)


@pytest.mark.parametrize("new", [1, 5, 80])
def test_rows_that_see_nothing(gpu_lib, new):
    """More new tokens than the cache holds: the first rows stand before the start. Lengths of zero."""
    b = Batch([0] * 4, [new] * 4, hq=4, hkv=2, dim=64, page=16, kv_lens=[0, max(new - 1, 0), new, new + 3], seed=new)
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    assert (o[:new] == 0).all() and (lse[:new] == -INF).all()


def test_no_tokens(gpu_lib):
    b = Batch([3, 5], [0, 0], hq=4, hkv=2, dim=64, page=16, pad=4)
    b.check(*b.call(gpu_lib))
    b = Batch([3, 5], [0, 0], hq=4, hkv=2, dim=64, page=16, pad=0)
    o, lse = b.call(gpu_lib)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("bad", [NAN, INF, -INF, torch.finfo(BF).min])
@pytest.mark.parametrize("new", [1, 6, 100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_not_seen_has_no_influence(gpu_lib, bad, new, dtype):
    """Infinities, NaN and the lowest values in keys and values that a row does not see, everywhere but in what it sees."""
    ctx, window = 150, 40
    kw = dict(hq=4, hkv=2, dim=128, page=16, dtype=dtype, seed=new)
    plain = Batch([ctx, ctx], [new, new], garbage=0.0, **kw)
    o, lse = plain.call(gpu_lib, window=window)
    plain.check(o, lse, window=window)
    dirty = Batch([ctx, ctx], [new, new], garbage=bad, **kw)
    for j in range(0, ctx - window + 1):       # before the window of every row
        dirty.put(0, j, k=bad, v=bad)
    last = ctx + new - 1
    dirty.put(1, last, k=bad, v=bad)           # seen by the last row alone
    if new > window:
        dirty.put(1, ctx, k=bad, v=bad)        # seen by the first `window` rows
    got, glse = dirty.call(gpu_lib, window=window)
    assert torch.equal(got[:new], o[:new]) and torch.equal(glse[:new], lse[:new])
    clean = slice(new + (window if new > window else 0), 2 * new - 1)
    assert torch.equal(got[clean], o[clean]) and torch.equal(glse[clean], lse[clean])
    if bad != bad:
        assert torch.isnan(got[2 * new - 1]).all()


@pytest.mark.parametrize("new", [1, 50])
def test_infinite_values_that_are_seen(gpu_lib, new):
    """An infinite value gives an infinite column to the rows that see it and leaves the other columns and rows alone."""
    b = Batch([40], [new], hq=2, hkv=1, dim=64, page=16, seed=1)
    b.put(0, 40 + new // 2, v=INF, dims=3)
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    assert torch.isinf(o[new // 2:, :, 3]).all() and torch.isfinite(o[: new // 2]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,hq", [(1, 2), (6, 10), (50, 2)])
def test_infinite_values_across_the_columns(gpu_lib, dtype, dim, new, hq):
    """Infinite values and NaN in columns all over a row, in a tile that some rows see in part and in one that all do."""
    b = Batch([700], [new], hq=hq, hkv=2, dim=dim, page=16, dtype=dtype, seed=dim + new)
    for x in range(dim // 32):
        b.put(0, 700 + new // 2, v=(INF, -INF)[x % 2], dims=32 * x + 5 * x % 32)
    b.put(0, 320, v=INF, dims=dim - 1)
    b.put(0, 700 + new - 1, v=NAN, dims=dim // 2)
    b.put(0, 699, v=NAN, heads=1, dims=0)
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    b.check(*b.call(gpu_lib, window=9), window=9)


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (BF, 256), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("new", [1, 7])
def test_many_tiles_a_wave(gpu_lib, dtype, dim, new):
    """Few rows over an axis so long that every wave of every workgroup goes through many tiles."""
    b = Batch([16000, 40, 20011], [new, 0, new], hq=8, hkv=4, dim=dim, page=64, dtype=dtype, seed=dim + new)
    b.check(*b.call(gpu_lib))
    b.check(*b.call(gpu_lib, window=9001), window=9001)


@pytest.mark.parametrize("new", [1, 40])
def test_large_scores(gpu_lib, new):
    """Scores far apart: one key takes all the weight; the running maximum moves by hundreds."""
    b = Batch([300], [new], hq=4, hkv=2, dim=64, page=16, dtype=F32, seed=2)
    b.check(*b.call(gpu_lib, scale=20.0), scale=20.0)
    b.check(*b.call(gpu_lib, scale=-3.0), scale=-3.0)
    b.check(*b.call(gpu_lib, scale=0.0), scale=0.0)
    b = Batch([300], [new], hq=4, hkv=2, dim=128, page=16, seed=2)
    b.check(*b.call(gpu_lib, scale=20.0), scale=20.0)


@pytest.mark.parametrize("new", [1, 4, 60])
def test_all_scores_minus_infinity(gpu_lib, new):
    """A row whose every score is -inf counts as one that sees nothing."""
    b = Batch([20], [new], hq=2, hkv=1, dim=64, page=16, dtype=F32, seed=5)
    b.q.copy_(b.q.abs() + 0.1)
    b.d_q.copy_(b.q)
    for j in range(20 + new):
        b.put(0, j, k=-INF)
    o, lse = b.call(gpu_lib)
    assert (o == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("max_new", [0, 1, 2, 33, 1000])
def test_max_new_is_a_bound_only(gpu_lib, max_new):
    b = Batch([100, 0, 333], [1, 1, 1], hq=8, hkv=2, dim=128, page=16, pad=2, seed=9)
    b.check(*b.call(gpu_lib, max_new=max_new))


@pytest.mark.parametrize("new", [1, 70])
def test_sliced_queries_and_no_lse(gpu_lib, new):
    b = Batch([90, 4], [new, new], hq=4, hkv=2, dim=64, page=16, q_extra=256, seed=11)
    assert not b.d_q.is_contiguous()
    o, lse = b.call(gpu_lib)
    b.check(o, lse)
    got, none = gpu_lib.rglru_paged_attn_fwd(b.d_q, b.d_k, b.d_v, b.d_table, b.d_cu, b.d_kv, want_lse=False)
    assert none is None and torch.equal(got[: b.tokens], o[: b.tokens])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_each_time(gpu_lib, dtype):
    b = Batch([4000, 31, 800], [1, 1, 1], hq=8, hkv=2, dim=128, page=32, dtype=dtype, seed=13)
    c = Batch([1000, 31, 0], [20, 1, 300], hq=8, hkv=2, dim=128, page=32, dtype=dtype, seed=13)
    ref = b.call(gpu_lib), c.call(gpu_lib)
    for _ in range(3):
        again = b.call(gpu_lib), c.call(gpu_lib)
        for x, y in zip(ref, again):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("new", [1, 40])
def test_cache_past_32_bit_offsets(gpu_lib, new):
    """Pages at the end of a cache of more than 2^31 elements (more than 2^32 bytes)."""
    page, hkv, dim = 256, 8, 256
    n_pages = (1 << 31) // (page * hkv * dim) + 40
    kc = torch.zeros((n_pages, hkv, page, dim), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    b = Batch([500, 900], [new, new], hq=8, hkv=hkv, dim=dim, page=page, seed=17)
    m = b.d_k.shape[0]
    kc[-m:], vc[-m:] = b.d_k, b.d_v
    b.d_k, b.d_v = kc, vc
    b.d_table = b.d_table + (n_pages - m)
    b.check(*b.call(gpu_lib))


def test_block_table_outside_the_cache_stays_in_bounds(gpu_lib):
    """Page numbers outside the cache and lengths past the table are clamped: unspecified results, no fault."""
    for new in (1, 40):
        b = Batch([100, 100], [new, new], hq=4, hkv=2, dim=64, page=16, garbage=0.0)
        b.d_table.fill_(1 << 30)
        b.d_table[1].fill_(-5)
        b.d_kv.copy_(torch.tensor([1 << 30, -3], dtype=torch.int32))
        o, _ = b.call(gpu_lib)
        torch.cuda.synchronize()
        assert (o[new:] == 0).all()


def test_two_streams_and_graph_replay(gpu_lib):
    """Two calls on two streams with workspaces of their own, and both captured in a graph whose lengths change."""
    a = Batch([700, 60], [1, 1], hq=8, hkv=2, dim=128, page=16, seed=21, garbage=0.0)   # a replay reads past its 61 tokens
    c = Batch([100, 3], [50, 20], hq=8, hkv=2, dim=128, page=16, seed=22)
    refs = [x.call(gpu_lib) for x in (a, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s, x in zip(streams, (a, c)):
        with torch.cuda.stream(s):
            outs.append([x.call(gpu_lib) for _ in range(5)])
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        for o, lse in got:
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = [x.call(gpu_lib, max_new=50) for x in (a, c)]
    for kv in ([701, 61], [5, 1], [320, 700], [701, 61]):
        a.d_kv.copy_(torch.tensor(kv, dtype=torch.int32))
        eager = a.call(gpu_lib, max_new=50)
        eager_c = c.call(gpu_lib)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(caught[0][0], eager[0]) and torch.equal(caught[0][1], eager[1])
        assert torch.equal(caught[1][0], eager_c[0]) and torch.equal(caught[1][1], eager_c[1])


def test_one_workspace_for_calls_in_a_row(gpu_lib):
    """A workspace sized for the larger of two calls serves both, one after the other, in either order."""
    a = Batch([3000], [1], hq=8, hkv=2, dim=128, page=16, seed=31)
    c = Batch([100, 3], [50, 20], hq=8, hkv=2, dim=128, page=16, seed=32)
    ra, rc = a.call(gpu_lib), c.call(gpu_lib)
    ws = torch.full((256 << 20,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        ga, gc = a.call(gpu_lib, workspace=ws), c.call(gpu_lib, workspace=ws)
        assert torch.equal(ga[0], ra[0]) and torch.equal(gc[0], rc[0])
        assert torch.equal(ga[1], ra[1]) and torch.equal(gc[1], rc[1])


def test_many_sequences(gpu_lib):
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 60, 1500).tolist()
    b = Batch(ctx, [1] * 1500, hq=2, hkv=1, dim=64, page=16, seed=41)
    b.check(*b.call(gpu_lib))
    new = rng.integers(0, 4, 1500).tolist()
    b = Batch(ctx, new, hq=32, hkv=1, dim=64, page=16, seed=42)
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("n", [2, 20])
def test_many_row_tiles(gpu_lib, n):
    """More row tiles than a workgroup lists for itself, and (20 sequences) than the list's workgroup has threads."""
    new = [8200 // n - 7 * (i % 3) for i in range(n)]
    b = Batch([i % 5 for i in range(n)], new, hq=8, hkv=1, dim=64, page=64, seed=n)
    b.check(*b.call(gpu_lib, window=20), window=20)


@pytest.mark.parametrize("n,dim,dtype", [(5, 128, BF), (20, 128, BF), (20, 256, BF), (20, 64, F32), (300, 64, BF)])
def test_replayed_with_other_lengths(gpu_lib, n, dim, dtype):
    """One captured call for batches of other shapes: chunks and single tokens change places, sequences come and go,
    rows turn into padding. Each replay has the bits of an eager call."""
    rng = np.random.default_rng(n)
    cap, keys = 700, 160
    b = Batch([keys] * n, [0] * n, hq=4, hkv=2, dim=dim, page=16, dtype=dtype, pad=cap, seed=n, garbage=0.0)
    graph = torch.cuda.CUDAGraph()
    b.call(gpu_lib, max_new=0)
    torch.cuda.synchronize()
    o = torch.zeros((cap, 4, dim), dtype=dtype, device="cuda")
    lse = torch.zeros((cap, 4), device="cuda")
    args = (b.d_q, b.d_k, b.d_v, b.d_table, b.d_cu, b.d_kv)
    with torch.cuda.graph(graph):
        gpu_lib.rglru_paged_attn_fwd(*args, o=o, lse=lse)
    for step in range(5):
        new = rng.integers(0, 2, n)
        if step % 2 == 0:
            new[rng.integers(0, n)] = int(rng.integers(2, 150))
        kv = np.maximum(rng.integers(0, keys + 1, n), new)
        b.new, b.kv, b.cu = new.tolist(), kv.tolist(), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b.tokens = int(b.cu[-1])
        b.d_cu.copy_(torch.from_numpy(b.cu))
        b.d_kv.copy_(torch.tensor(b.kv, dtype=torch.int32))
        eager = b.call(gpu_lib, max_new=0)
        b.check(*eager)
        o.fill_(7.0), lse.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])


def test_refusals(gpu_lib):
    b = Batch([10], [2], hq=4, hkv=2, dim=64, page=16)
    call = gpu_lib.rglru_paged_attn_fwd
    args = [b.d_q, b.d_k, b.d_v, b.d_table, b.d_cu, b.d_kv]
    for i, wrong in ((0, b.d_q[:, :3]), (0, b.d_q.float()), (0, b.d_q.transpose(0, 1)), (1, b.d_k[:, :, :, ::2]), (2, b.d_v.float()),
                     (3, b.d_table.long()), (3, b.d_table[:0]), (4, b.d_cu.long()), (4, b.d_cu[:1]), (5, b.d_kv.cpu()),
                     (5, torch.cat([b.d_kv, b.d_kv]))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call(*args[:i], wrong, *args[i + 1:])
    for kw in (dict(window=-1), dict(max_new=-1), dict(scale=NAN), dict(workspace=torch.empty(8, device="cuda")),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(o=torch.empty(1, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            call(*args, **kw)
    odd = Batch([10], [2], hq=4, hkv=2, dim=96, page=16)
    with pytest.raises(gpu_lib.RglruError, match="UNSUPPORTED"):
        odd.call(gpu_lib)
