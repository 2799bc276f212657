"""Page plan and key/value write against the oracle (whole numbers and copies: equal), and a serving run of the set."""
import numpy as np
import pytest
import torch

from _paged import Batch
from oracle import paged as oracle_paged

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def run_plan(glr, ctx, held, new, table, free, count, page, pad=0, max_new=0):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = int(cu[-1]) + pad
    ref = oracle_paged.page_plan(ctx, held, cu, table, free, count, rows, page)
    d_table, d_free = i32(table), i32(free)
    out = glr.rglru_page_plan(i32(ctx), i32(cu), d_table, d_free, i32([count]), n_tokens=rows, page_size=page,
                              held_lens=i32(held), max_new=max_new)
    names = ("slot_map", "positions", "kv_lens", "held_lens_out", "free_count_out", "unserved")
    got = dict(zip(names, (t.cpu().numpy() for t in out)), block_table=d_table.cpu().numpy(), free_pages=d_free.cpu().numpy())
    for k, v in ref.items():
        assert np.array_equal(got[k], np.atleast_1d(v)), (k, got[k], v)
    return ref


@pytest.mark.parametrize("n", [1, 3, 4, 5, 64, 255, 257, 2500])
@pytest.mark.parametrize("page", [8, 64])
def test_plan_steps(gpu_lib, n, page):
    """Steps in a row: chunks, single tokens, requests that end, drafts given back, a pool that runs short."""
    rng = np.random.default_rng(n + page)
    width = 6
    for pool in (n * width, max(2, n * 2)):
        table, free, count = np.full((n, width), -1, np.int32), rng.permutation(pool).astype(np.int32), pool
        held = np.zeros(n, np.int64)
        for step in range(4):
            ctx = np.array([0 if rng.random() < 0.1 else rng.integers(0, h + 1) if rng.random() < 0.3 else h for h in held])
            new = rng.integers(0, 2 * page, n) * (rng.random(n) < 0.7)
            r = run_plan(gpu_lib, ctx, held, new, table, free, count, page, pad=int(rng.integers(0, 5)),
                         max_new=int(rng.choice([0, 2 * page])))
            table, free, count, held = r["block_table"], r["free_pages"], r["free_count_out"], r["held_lens_out"].astype(np.int64)


def test_plan_long_sequences(gpu_lib):
    """Slices of long chunks, and pages given back that others of the same step take."""
    rng = np.random.default_rng(7)
    table = rng.permutation(3 * 900).reshape(3, 900).astype(np.int32)
    free = np.zeros(2700, np.int32)
    r = run_plan(gpu_lib, [0, 3, 5000], [7000, 3, 5001], [0, 6000, 1200], table, free, 0, 8)
    assert r["unserved"] == 1        # 876 pages came back: 750 go to the second, the third asks for more than are left
    run_plan(gpu_lib, [0, 3, 5000], [7000, 3, 5001], [0, 6000, 100], table, free, 0, 8, pad=1000, max_new=6000)


def test_plan_nothing_to_do(gpu_lib):
    free = np.arange(4, dtype=np.int32)
    run_plan(gpu_lib, [0, 0], [0, 0], [0, 0], np.zeros((2, 1), np.int32), free, 4, 16)
    run_plan(gpu_lib, [0, 0], [0, 0], [0, 0], np.zeros((2, 1), np.int32), free, 0, 16, pad=70)
    run_plan(gpu_lib, [0], [0], [17], np.zeros((1, 1), np.int32), free, 4, 16)    # the row of the table is too short


def test_plan_lengths_out_of_range_stay_in_bounds(gpu_lib):
    big = (1 << 31) - 1
    for ctx, cu, held, count in (([big, -5, 3], [0, 5, 2, 9], [big, big, -1], 1 << 30), ([0, 0, 0], [-4, big, 1, big], [big] * 3, -7)):
        out = gpu_lib.rglru_page_plan(i32(ctx), i32(cu), i32(np.zeros((3, 4))), i32(np.arange(12)), i32([count]), n_tokens=8,
                                      page_size=16, held_lens=i32(held))
        torch.cuda.synchronize()
        assert out[0].shape == (8,)


def test_plan_refusals(gpu_lib):
    a = dict(context_lens=i32([0]), cu_seqlens=i32([0, 1]), block_table=i32([[0]]), free_pages=i32([0]), free_count=i32([1]))
    for bad in (dict(page_size=12), dict(page_size=4), dict(page_size=2048), dict(n_tokens=-1), dict(max_new=-1),
                dict(context_lens=i32([0, 0])), dict(cu_seqlens=i32([0])), dict(block_table=i32([0])), dict(free_count=i32([1, 1])),
                dict(held_lens=i32([0]).long()), dict(slot_map=i32([0, 0])), dict(free_pages=i32([[0]])),
                dict(free_count_out=a["free_count"])):
        with pytest.raises((ValueError, RuntimeError)):
            gpu_lib.rglru_page_plan(**{**a, "n_tokens": 1, "page_size": 16, **bad})


@pytest.mark.parametrize("heads,dim,page,t", [(1, 64, 8, 1), (3, 128, 16, 33), (8, 128, 64, 500), (16, 256, 16, 70), (5, 8, 32, 90), (1, 4, 8, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_write(gpu_lib, dtype, heads, dim, page, t):
    if dtype == torch.bfloat16:
        dim = max(dim, 8)      # whole 16-byte pieces
    gen = torch.Generator().manual_seed(t)
    n_pages = -(-t // page) + 3
    kc, vc = (torch.randn(n_pages, heads, page, dim, generator=gen).to(dtype) for _ in range(2))
    wide = torch.randn(t, 3, heads, dim, generator=gen).to(dtype)
    slots = torch.randperm(n_pages * page, generator=gen)[:t].int()
    if t > 5:
        slots[2], slots[t - 1], slots[3] = -1, n_pages * page, -100
    for rows in (wide, wide[:, :2].contiguous()):      # slices of wider rows; other strides
        dk, dv, dw = kc.cuda(), vc.cuda(), rows.cuda()
        gpu_lib.rglru_paged_kv_write(dw[:, 0], dw[:, 1], dk, dv, slots.cuda())
        for cache, got, x in ((kc, dk, rows[:, 0]), (vc, dv, rows[:, 1])):
            ref = oracle_paged.kv_write(x.float().numpy(), cache.float().numpy(), slots.numpy())
            assert np.array_equal(got.float().cpu().numpy(), ref)


def test_write_past_32_bit_offsets(gpu_lib):
    kc = torch.zeros((520, 16, 1024, 256), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn(3, 16, 256, device="cuda").bfloat16()
    gpu_lib.rglru_paged_kv_write(k, k + 1, kc, vc, i32([520 * 1024 - 1, 0, 515 * 1024 + 7]))
    assert torch.equal(kc[519, :, 1023], k[0]) and torch.equal(vc[515, :, 7], k[2] + 1) and torch.equal(kc[0, :, 0], k[1])
    assert int((kc != 0).any(-1).sum()) == 3 * 16


def test_write_refusals(gpu_lib):
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = i32([0, 1, 2])
    flat = torch.zeros(3 * 132, dtype=torch.bfloat16, device="cuda")
    for args in ((k.float(), k, kc, kc, slots), (k, k[:2], kc, kc, slots), (k, k, kc, kc[:1], slots), (k, k, kc, kc, slots[:2]),
                 (k, k, kc.transpose(1, 2), kc.transpose(1, 2), slots), (k, k, kc, kc, slots.long()), (k, k, kc[0], kc[0], slots),
                 (flat.as_strided((3, 2, 64), (132, 64, 1)), flat.as_strided((3, 2, 64), (132, 64, 1)), kc, kc, slots),
                 (flat.as_strided((3, 2, 64), (64, 64, 1)), flat.as_strided((3, 2, 64), (64, 64, 1)), kc, kc, slots),
                 (k, k, torch.zeros((2, 2, 12, 64), dtype=torch.bfloat16, device="cuda"),
                  torch.zeros((2, 2, 12, 64), dtype=torch.bfloat16, device="cuda"), slots)):
        with pytest.raises((ValueError, RuntimeError)):
            gpu_lib.rglru_paged_kv_write(*args)


@pytest.mark.parametrize("graph", [False, True])
def test_serving_run_of_a_hybrid_model(gpu_lib, graph):
    """Steps of a recurrent layer and an attention layer over one packed batch: prompt chunks, then single tokens, then
    rejected drafts, lengths on the device throughout; each sequence is held to the oracle over its whole history. With
    `graph`, one captured step is replayed for every batch up to its capacity."""
    glr, dev, io = gpu_lib, "cuda", torch.bfloat16
    hq, hkv, dim, page, n, rows, width, w = 10, 1, 64, 16, 3, 64, 8, 640
    n_pages = n * width
    gen = torch.Generator().manual_seed(3)
    lam = torch.rand(w, generator=gen).to(dev)
    proj = (torch.randn(w, (hq + 2 * hkv) * dim, generator=gen) / w ** 0.5).to(dev)
    kc, vc = (torch.full((n_pages, hkv, page, dim), float("nan"), dtype=io, device=dev) for _ in range(2))
    table = torch.zeros((n, width), dtype=torch.int32, device=dev)
    free, count = torch.randperm(n_pages, generator=gen).int().to(dev), i32([n_pages])
    held, ctx, cu = i32([0] * n), i32([0] * n), i32([0] * (n + 1))
    x, gates = torch.zeros((rows, w), dtype=io, device=dev), torch.zeros((2, rows, w), dtype=io, device=dev)
    state = torch.zeros((n, w), device=dev)
    ws = glr.Workspace(dev)

    def step():
        # the packed offsets of the recurrent call cover every row: padding goes to a last sequence of its own
        slots, pos, kv, held_out, left, short = glr.rglru_page_plan(ctx, cu, table, free, count, n_tokens=rows, page_size=page, held_lens=held)
        ends = torch.cat([cu, cu.new_full((1,), rows)])
        h0 = torch.cat([state, state.new_zeros((1, w))])
        h, last, _ = glr.rglru_fwd_varlen(x, gates[0], gates[1], lam, ends, h0=h0, workspace=ws)
        qkv = (h.float() @ proj).to(io).view(rows, hq + 2 * hkv, dim)
        k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        glr.rglru_paged_kv_write(k, v, kc, vc, slots)
        o, lse = glr.rglru_paged_attn_fwd(qkv[:, :hq], kc, vc, table, cu, kv, window=20)
        return dict(qkv=qkv, o=o, lse=lse, kv=kv, left=left, short=short, last=last, held=held_out)

    step()                          # sizes the workspace before any capture
    torch.cuda.synchronize()
    kc.fill_(float("nan")), vc.fill_(float("nan"))
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            caught = step()
    history = [[] for _ in range(n)]   # (k, v) of every token kept, on the host
    plan = [([0, 0, 0], [17, 30, 1]), ([17, 30, 1], [1, 1, 20]), ([18, 31, 21], [5, 1, 0]), ([20, 32, 21], [1, 1, 1]),
            ([0, 33, 22], [9, 1, 33]), ([9, 0, 55], [1, 0, 1])]
    for c, new in plan:
        ctx.copy_(i32(c)), cu.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        x.copy_(torch.randn(x.shape, generator=gen)), gates.copy_(torch.randn(gates.shape, generator=gen))
        torch.cuda.synchronize()
        if graph:
            g.replay()
            r = caught
        else:
            r = step()
        torch.cuda.synchronize()
        assert int(r["short"]) == 0 and r["kv"].tolist() == [a + b for a, b in zip(c, new)]
        used = sum(-(-(a + b) // page) for a, b in zip(c, new))
        assert int(r["left"]) == n_pages - used
        qkv, at = r["qkv"].double().cpu().numpy(), 0
        for i in range(n):
            history[i] = history[i][: c[i]] + [(qkv[at + t, hq:hq + hkv], qkv[at + t, hq + hkv:]) for t in range(new[i])]
            if new[i]:
                k, v = (np.stack([e[j] for e in history[i]], 1) for j in (0, 1))
                ref, ref_lse, weight, size, seen = oracle_paged.attention(qkv[at:at + new[i], :hq], k, v, c[i] + new[i], 20, dim ** -0.5)
                e = (dim + 8) * 2.0 ** -24 * size
                rel = (2 * e + ((seen + 8) * 2.0 ** -23)[:, None])[..., None]
                got = r["o"][at:at + new[i]].double().cpu().numpy()
                assert (np.abs(got - ref) <= rel * weight + 1.01 * 2.0 ** -8 * (weight + np.abs(ref))).all()
            at += new[i]
        held.copy_(r["held"]), count.copy_(r["left"]), state.copy_(r["last"][:n])


def test_attention_reads_what_was_written(gpu_lib):
    """Plan, write and attention give what a batch laid out on the host gives, bit for bit."""
    b = Batch([0, 0], [75, 20], hq=4, hkv=2, dim=128, page=16, seed=8)
    ref = b.call(gpu_lib)
    n_pages = b.d_k.shape[0]
    table = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    slots, pos, kv, _, _, short = gpu_lib.rglru_page_plan(i32([0, 0]), b.d_cu, table, i32(np.arange(n_pages)), i32([n_pages]),
                                                       n_tokens=95, page_size=16)
    assert int(short) == 0 and pos.tolist() == list(range(75)) + list(range(20))
    kc, vc = torch.zeros_like(b.d_k), torch.zeros_like(b.d_v)
    gpu_lib.rglru_paged_kv_write(torch.cat(b.k).cuda(), torch.cat(b.v).cuda(), kc, vc, slots)
    o, lse = gpu_lib.rglru_paged_attn_fwd(b.d_q, kc, vc, table, b.d_cu, kv)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
