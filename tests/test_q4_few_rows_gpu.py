"""The kernel for few rows over a 4-bit cache by itself and beside the one for many: repeated, on other streams, over workspaces of any
contents, behind 2^32 bytes, with more sequences than a workgroup has threads, and a serving step replayed from graphs."""
import numpy as np
import pytest
import torch

from _paged_q4 import Q4Batch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SPACE = 224 << 20
# single tokens; drafts, two sets of 16 rows a wave; more than 16 sequences, so that both kernels run
MIXED = [1] * 10 + [60, 1, 3, 0, 1, 70, 1, 2, 1, 1]
BATCHES = {"decode": ([3000, 10, 900], [1, 1, 1]), "drafts": ([2000, 5, 700, 64], [8, 3, 1, 5]),
           "mixed": ([2500, 40, 1, 0, 63, 64, 65, 7, 300, 900, 20, 0, 128, 5, 511, 30, 1000, 2, 77, 6], MIXED)}


def batch(name, dtype, **kw):
    ctx, new = BATCHES[name]
    return Q4Batch(ctx, new, **{**dict(hq=8, hkv=2, dim=128, page=32, dtype=dtype, seed=len(new)), **kw})


def equal(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("name", BATCHES)
def test_the_same_bits_each_time(gpu_lib, name, dim, dtype):
    b = batch(name, dtype, dim=dim)
    first = b.call(gpu_lib)
    b.check(*first)
    for _ in range(5):
        assert equal(b.call(gpu_lib), first)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", BATCHES)
def test_a_workspace_of_any_contents(gpu_lib, name, dtype):
    b = batch(name, dtype)
    want = b.call(gpu_lib)
    b.check(*want)
    space = torch.empty(SPACE, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127, 1):
        space.fill_(fill)
        assert equal(b.call(gpu_lib, workspace=space), want)
    # what another call left there
    other = Q4Batch([400] * 30, [1] * 30, hq=8, hkv=2, dim=128, page=32, dtype=dtype, seed=5)
    other.call(gpu_lib, workspace=space)
    assert equal(b.call(gpu_lib, workspace=space), want)


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("new", [[1, 1], [5, 16]])
def test_past_32_bit_offsets(gpu_lib, dim, new):
    """Pages whose codes lie behind 2^32 bytes, one and two sets of rows."""
    b = Q4Batch([1500, 20], new, hq=2, hkv=1, dim=dim, page=1024, seed=5, spare=0)
    n_pages = (1 << 32) // (1024 * dim // 2) + 8
    base = n_pages - b.cache[0].shape[0]
    for c in range(4):
        big = torch.zeros(n_pages, *b.cache[c].shape[1:], dtype=torch.uint8, device="cuda")
        big[base:] = b.d_cache[c]
        b.d_cache[c] = big
    b.d_table += base
    b.check(*b.call(gpu_lib))


@pytest.mark.parametrize("name", BATCHES)
def test_on_other_streams(gpu_lib, name):
    """Two calls on two streams at once, each with a workspace of its own."""
    b, c = batch(name, BF16), batch(name, F32)
    want = b.call(gpu_lib), c.call(gpu_lib)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(SPACE, dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for x, (s, y) in enumerate(zip(streams, (b, c))):
            with torch.cuda.stream(s):
                got[x].append(y.call(gpu_lib, workspace=spaces[x]))
    for s in streams:
        s.synchronize()
    for x in range(2):
        assert all(equal(g, want[x]) for g in got[x])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [256, 257, 700])
@pytest.mark.parametrize("most", [1, 5, 40])
def test_more_sequences_than_threads(gpu_lib, n, most, dtype):
    """Empty ones among them; with 40 new tokens some go to the kernel for many rows."""
    rng = np.random.default_rng(n + most)
    new = np.where(rng.random(n) < 0.1, 0, 1)
    some = rng.random(n) < 0.05
    new[some] = rng.integers(1, most + 1, some.sum())
    new[n // 2] = most
    ctx = rng.integers(0, 90, n)
    ctx[[0, n - 1]] = 700, 600
    b = Q4Batch(ctx.tolist(), new.tolist(), hq=4, hkv=2, dim=64, page=16, dtype=dtype, seed=n, pad=9)
    first = b.call(gpu_lib)
    b.check(*first)
    assert equal(b.call(gpu_lib), first)


@pytest.mark.parametrize("names", [("decode", "drafts"), ("drafts", "mixed")])
def test_graphs_that_share_a_workspace(gpu_lib, names):
    """Two captured calls of different shapes over one workspace, replayed in turn."""
    space = torch.empty(SPACE, dtype=torch.uint8, device="cuda")
    batches = [batch(n, BF16) for n in names]
    want, got, graphs = [b.call(gpu_lib) for b in batches], [], []
    for b in batches:
        out = (torch.empty(b.q.shape[0], b.hq, b.dim, dtype=BF16, device="cuda"), torch.empty(b.q.shape[0], b.hq, device="cuda"))
        call = lambda: gpu_lib.rglru_paged_attn_q4_fwd(b.d_q, *b.d_cache, b.d_table, b.d_cu, b.d_kv, max_new=max(b.new), o=out[0],  # noqa: E731, B023
                                                       lse=out[1], workspace=space)  # noqa: B023
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
        got.append(out)
    for _ in range(4):
        for x in (0, 1):
            got[x][0].fill_(7.0), got[x][1].fill_(7.0)
            graphs[x].replay()
            torch.cuda.synchronize()
            assert equal(got[x], want[x])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_serving_step_replayed(gpu_lib, dtype):
    """Plan, write and attention in one graph, fork and copy in another: replayed step after step, equal to the same calls made eagerly."""
    n, page, width, pages, hq, hkv, dim, rows = 6, 8, 20, 100, 4, 2, 64, 12
    rng = np.random.default_rng(1)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731

    class State:
        def __init__(self):
            self.table, self.shares, self.free, self.count = i32(np.zeros((n, width))), i32(np.zeros(pages)), i32(np.arange(pages)), i32([pages])
            self.lens, self.held, self.src, self.cu = i32(np.zeros(n)), i32(np.zeros(n)), i32(-np.ones(n)), i32(np.zeros(n + 1))
            self.cache = [torch.full((pages, hkv, page, dim // (32 if c % 2 else 2)), 255, dtype=torch.uint8, device="cuda") for c in range(4)]
            self.q, self.k, self.v = (torch.zeros(rows, h, dim, dtype=dtype, device="cuda") for h in (hq, hkv, hkv))
            self.o, self.lse = torch.zeros(rows, hq, dim, dtype=dtype, device="cuda"), torch.zeros(rows, hq, device="cuda")
            self.space = torch.empty(SPACE, dtype=torch.uint8, device="cuda")

        def step(self):
            slots, _, kv, held, count, unserved = gpu_lib.rglru_page_plan(
                self.lens, self.cu, self.table, self.free, self.count, n_tokens=rows, page_size=page, held_lens=self.held)
            gpu_lib.rglru_paged_kv_write_q4(self.k, self.v, *self.cache, slots)
            gpu_lib.rglru_paged_attn_q4_fwd(self.q, *self.cache, self.table, self.cu, kv, max_new=4, o=self.o, lse=self.lse, workspace=self.space)
            return kv, held, count, unserved

        def fork(self):
            pairs, lens, held, count, unserved = gpu_lib.rglru_page_fork(
                self.src, self.lens, self.table, self.shares, self.free, self.count, page_size=page, held_lens=self.held)
            gpu_lib.rglru_page_copy(pairs, self.cache)
            return lens, held, count, unserved

        def take(self, out):
            self.lens.copy_(out[0]), self.held.copy_(out[1]), self.count.copy_(out[2])
            assert int(out[3]) == 0

        def all(self):
            return [self.table, self.shares, self.free, self.count, self.lens, self.held, *self.cache, self.o, self.lse]

    def captured(call):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        return graph, out

    eager, replayed = State(), State()
    step, fork = captured(replayed.step), captured(replayed.fork)   # no tokens and no forks yet: nothing changes
    for t in range(14):
        src = [-1] * n
        if t in (2, 5):   # rows that hold nothing go on from others
            src = [-1, -1, -1, 0, 1, -1] if t == 2 else [-1] * 5 + [3]
        new = [3, 4, 2, 0, 0, 0] if t == 0 else rng.integers(0, 3, n) * (eager.lens.cpu().numpy() > 0)
        if t not in (0, 2, 5):
            new = np.minimum(new + (eager.lens.cpu().numpy() > 0), 4)
        while sum(new) > rows:
            new[int(np.argmax(new))] -= 1
        q, k, v = (torch.from_numpy(rng.standard_normal((rows, h, dim))).to(dtype).cuda() for h in (hq, hkv, hkv))
        for s in (eager, replayed):
            s.src.copy_(i32(src)), s.cu.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
            s.q.copy_(q), s.k.copy_(k), s.v.copy_(v)
        eager.take(eager.fork())
        eager.take(eager.step())
        fork[0].replay()
        replayed.take(fork[1])
        step[0].replay()
        replayed.take(step[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(eager.all(), replayed.all())), t
    assert int(eager.shares.sum()) > 0 and min(eager.lens.tolist()) > 0
