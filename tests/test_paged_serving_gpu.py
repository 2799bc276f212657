"""A step whose pool runs short: what the served sequences get, and what the others' rows are worth."""
import numpy as np
import pytest
import torch

from _paged_strict import StrictBatch

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [[5, 40, 3, 1], [1, 20, 1, 1], [70, 90, 2, 33]])
def test_sequences_that_are_not_served(gpu_lib, dtype, new):
    """The pool holds the pages of the first sequence alone and the third needs none: the others' tokens get no slot, their cache
    and lengths stay, and the rows of the served ones are right. Rows without a slot are known by slot_map -1."""
    page, dim, hkv, width = 16, 64, 2, 12
    ctx = [0, 30, 17, 16]
    b = StrictBatch(ctx, new, hq=4, hkv=hkv, dim=dim, page=page, dtype=dtype, pad=3, seed=sum(new), garbage=0.0)
    n_pages = 4 * width
    kc, vc = (torch.full((n_pages, hkv, page, dim), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    have = [-(-c // page) for c in ctx]
    table, at = np.zeros((4, width), np.int32), 0
    for i in range(4):
        table[i, : have[i]] = np.arange(at, at + have[i])
        at += have[i]
    first = -(-new[0] // page)
    free = np.zeros(n_pages, np.int32)
    free[:first] = np.arange(at, at + first)
    d_table, rows = i32(table), b.q.shape[0]
    slots, pos, kv, held, count, short = gpu_lib.rglru_page_plan(i32(ctx), b.d_cu, d_table, i32(free), i32([first]), n_tokens=rows, page_size=page)
    served = [True] + [-(-(ctx[i] + new[i]) // page) == have[i] for i in (1, 2, 3)]
    assert not served[1] and served[2] and int(short) == 4 - sum(served) and int(count) == 0
    assert kv.tolist() == held.tolist() == [c + m * s for c, m, s in zip(ctx, new, served)]
    # the contexts, as earlier steps wrote them
    for i in range(4):
        for j in range(ctx[i]):
            kc[table[i, j // page], :, j % page], vc[table[i, j // page], :, j % page] = b.k[i][j].cuda(), b.v[i][j].cuda()
    before = kc.clone(), vc.clone()
    k, v = (torch.cat([t[i][ctx[i]:] for i in range(4)] + [torch.full((3, hkv, dim), 5.0, dtype=dtype)]).cuda() for t in (b.k, b.v))
    gpu_lib.rglru_paged_kv_write(k, v, kc, vc, slots)
    for i in range(4):
        where = slice(int(b.cu[i]), int(b.cu[i + 1]))
        assert bool((slots[where] >= 0).all() if served[i] else (slots[where] == -1).all())
        if not served[i]:
            for p in table[i, : have[i]].tolist():
                assert torch.equal(kc[p], before[0][p]) and torch.equal(vc[p], before[1][p])
    o = torch.full((rows, 4, dim), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((rows, 4), 7.0, device="cuda")
    gpu_lib.rglru_paged_attn_fwd(b.d_q, kc, vc, d_table, b.d_cu, kv, o=o, lse=lse)
    lost = slots[: b.tokens] < 0
    assert torch.isfinite(o).all() and bool(lost.any())
    for i in range(4):
        if not served[i]:
            b.new[i] = 0   # no rows of its own to hold to anything
    b.check(o, lse)
