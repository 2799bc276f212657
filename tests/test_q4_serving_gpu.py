"""A serving run: one page pool under two attention layers, one with a 4-bit cache and one in bf16 or float32. Requests come, go on
from each other's context, decode, drop drafts, end, and the pool moves together, all through the public entry points."""
import numpy as np
import pytest
import torch

from _paged_q4 import fast_quantise, hold
from _pool import check_pool
from oracle import paged_q4

pytestmark = pytest.mark.gpu
HQ, HKV, DIM, PAGE, N, WIDTH, PAGES = 4, 2, 64, 16, 10, 24, 130


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, glr, dtype, seed):
        self.glr, self.dtype, self.rng = glr, dtype, np.random.default_rng(seed)
        self.q4 = [torch.full((PAGES, HKV, PAGE, DIM // (32 if c % 2 else 2)), 255, dtype=torch.uint8, device="cuda") for c in range(4)]
        self.plain = [torch.full((PAGES, HKV, PAGE, DIM), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
        self.table, self.shares = i32(np.zeros((N, WIDTH))), i32(np.zeros(PAGES))
        self.free, self.count = i32(self.rng.permutation(PAGES)), i32([PAGES])
        self.lens = self.held = i32(np.zeros(N))
        self.keys, self.values = ([np.zeros((0, HKV, DIM)) for _ in range(N)] for _ in range(2))
        self.pages = PAGES

    def pool(self):
        s = dict(table=self.table.cpu().numpy(), held=self.held.cpu().numpy(), shares=self.shares.cpu().numpy(),
                 free=self.free.cpu().numpy(), count=int(self.count))
        s["free"], s["shares"] = s["free"][: self.pages], s["shares"][: self.pages]
        check_pool(s, PAGE)
        return s

    def step(self, new):
        glr, rng = self.glr, self.rng
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        rows = int(sum(new)) + 3
        slots, _, kv, self.held, self.count, unserved = glr.rglru_page_plan(
            self.lens, cu, self.table, self.free, self.count, n_tokens=rows, page_size=PAGE, held_lens=self.held)
        assert int(unserved) == 0
        q, k, v = (torch.from_numpy(rng.standard_normal((rows, h, DIM))).to(self.dtype) for h in (HQ, HKV, HKV))
        glr.rglru_paged_kv_write_q4(k.cuda(), v.cuda(), *self.q4, slots)
        glr.rglru_paged_kv_write(k.cuda(), v.cuda(), *self.plain, slots)
        o4, lse4 = glr.rglru_paged_attn_q4_fwd(q.cuda(), *self.q4, self.table, cu, kv)
        o, lse = glr.rglru_paged_attn_fwd(q.cuda(), *self.plain, self.table, cu, kv)
        at = 0
        for n, m in enumerate(new):
            part = slice(at, at + m)
            at += m
            self.keys[n] = np.concatenate([self.keys[n], k[part].double().numpy()])
            self.values[n] = np.concatenate([self.values[n], v[part].double().numpy()])
            if m:
                length = len(self.keys[n])
                kk, vv = self.keys[n].transpose(1, 0, 2), self.values[n].transpose(1, 0, 2)
                args = (length, 0, DIM ** -0.5, self.dtype)
                hold(o[part].cpu().double().numpy(), lse[part].cpu().double().numpy(), q[part].double().numpy(), kk, vv, *args, name=("plain", n))
                hold(o4[part].cpu().double().numpy(), lse4[part].cpu().double().numpy(), q[part].double().numpy(),
                     paged_q4.values(*fast_quantise(kk)), paged_q4.values(*fast_quantise(vv)), *args, name=("q4", n))
        self.lens = kv
        self.pool()

    def fork(self, src):
        pairs, self.lens, self.held, self.count, unserved = self.glr.rglru_page_fork(
            i32(src), self.lens, self.table, self.shares, self.free, self.count, page_size=PAGE, held_lens=self.held)
        self.glr.rglru_page_copy(pairs, [*self.q4, *self.plain])
        assert int(unserved) == 0
        for n, s in enumerate(src):
            if s >= 0:
                self.keys[n], self.values[n] = self.keys[s].copy(), self.values[s].copy()
        self.pool()

    def end(self, keep):
        self.held, self.count = self.glr.rglru_page_free(i32(keep), self.held, self.table, self.shares, self.free, self.count, page_size=PAGE)
        self.lens = self.held
        for n, m in enumerate(self.held.tolist()):
            self.keys[n], self.values[n] = self.keys[n][:m], self.values[n][:m]
        self.pool()

    def drop(self, n, m):
        """The last m tokens of row n were drafts that are not kept; the next plan gives their pages back."""
        self.lens = self.lens.clone()
        self.lens[n] -= m
        self.keys[n], self.values[n] = self.keys[n][:-m], self.values[n][:-m]

    def compact(self, keep):
        self.table, self.shares, self.free, self.count, pairs, n_pairs, unmoved = self.glr.rglru_page_compact(
            self.held, self.table, self.shares, self.free, self.count, page_size=PAGE, keep_pages=keep)
        self.glr.rglru_page_copy(pairs, [*self.q4, *self.plain], n_pairs=n_pairs)
        assert int(unmoved) == 0 and int(self.table.max()) < PAGES
        for c in self.q4:   # what lies behind is given away
            c[keep:] = 255
        for c in self.plain:
            c[keep:] = float("nan")
        self.pages = keep
        self.pool()

    def grow(self):
        """The pages behind come back, by the caller's own doing."""
        count = int(self.count)
        self.free[count: count + PAGES - self.pages] = i32(np.arange(self.pages, PAGES))
        self.count, self.pages = i32([count + PAGES - self.pages]), PAGES
        self.pool()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_serving_run(gpu_lib, dtype):
    s = Server(gpu_lib, dtype, 7)
    s.step([40, 5, 100, 0, 0, 0, 0, 0, 0, 16])
    s.fork([-1, -1, -1, 0, 2, 2, 9, 0, -1, -1])
    for _ in range(3):
        s.step([1, 1, 1, 1, 1, 1, 1, 1, 0, 1])
    s.step([4, 1, 1, 1, 1, 3, 1, 1, 20, 1])   # drafts of rows 0 and 5
    s.drop(0, 3)
    s.drop(5, 2)
    s.step([1] * 10)
    s.end([0 if n in (2, 7) else 10 ** 6 for n in range(N)])   # row 2 ends, what 4 and 5 share with it stays
    s.step([1, 1, 0, 1, 1, 1, 1, 0, 1, 1])
    s.fork([-1, -1, 4, -1, -1, -1, -1, -1, -1, -1])
    held = s.pool()
    s.compact(PAGES - held["count"] + 12)
    s.step([1, 1, 1, 1, 1, 1, 1, 0, 1, 1])
    s.grow()
    s.step([2, 30, 1, 1, 1, 1, 1, 64, 1, 1])
    s.end([0] * N)
    state = s.pool()
    assert state["count"] == PAGES and not state["shares"].any()


def test_answers_that_share_a_prompt_are_the_same_as_alone(gpu_lib):
    """Rows that went on from one context give, bit by bit, what a row that wrote it all itself gives."""
    glr, rng = gpu_lib, np.random.default_rng(3)
    s = Server(glr, torch.bfloat16, 3)
    s.step([50, 50, 0, 0, 0, 0, 0, 0, 0, 0])
    # row 1 gets the tokens of row 0, row 2 goes on from row 0
    slots = [s.table[n, torch.arange(50, device="cuda") // PAGE] * PAGE + torch.arange(50, device="cuda") % PAGE for n in (0, 1)]
    for x in (s.q4, s.plain):
        for c in x:
            flat = c.view(torch.uint8)
            flat[slots[1] // PAGE, :, slots[1] % PAGE] = flat[slots[0] // PAGE, :, slots[0] % PAGE]
    s.fork([-1, -1, 0] + [-1] * 7)
    q = torch.from_numpy(rng.standard_normal((1, HQ, DIM))).to(torch.bfloat16).cuda().expand(3, HQ, DIM).contiguous()
    lens = i32([50, 50, 50])
    o, lse = glr.rglru_paged_attn_q4_fwd(q, *s.q4, s.table[:3].contiguous(), i32([0, 1, 2, 3]), lens)
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2]) and torch.equal(lse[0], lse[2])
