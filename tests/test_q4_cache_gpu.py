"""Write and read-back of the 4-bit cache against the float64 reference: equal bit by bit."""
import numpy as np
import pytest
import torch

from _paged_q4 import fast_quantise
from oracle import paged_q4

pytestmark = pytest.mark.gpu


def cache_of(n_pages, heads, page, dim, fill=77):
    return [torch.full((n_pages, heads, page, dim // (32 if c % 2 else 2)), fill + c, dtype=torch.uint8, device="cuda")
            for c in range(4)]


def rows_of(rng, t, heads, dim, dtype):
    """Rows whose blocks are of very different sizes, some all 0, some not finite, some with ties."""
    x = rng.standard_normal((t, heads, dim // 32, 32)) * np.exp(8 * rng.standard_normal((t, heads, dim // 32, 1)))
    x[rng.random((t, heads, dim // 32)) < 0.05] = 0.0
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -2.5, -5.0, -0.0], x.shape)
    x = np.where(rng.random((t, heads, dim // 32, 1)) < 0.2, ties * 2.0 ** rng.integers(-20, 20, (t, heads, dim // 32, 1)), x)
    odd = rng.random((t, heads, dim // 32)) < 0.03
    x[..., 5] = np.where(odd, rng.choice([np.inf, -np.inf, np.nan], odd.shape), x[..., 5])
    x[..., 9] = np.where(rng.random(odd.shape) < 0.03, 3.3e38, x[..., 9])
    return torch.from_numpy(x.reshape(t, heads, dim)).to(dtype)


def put(expected, slots, parts, page):
    """The cache after the write, on the host."""
    for t, s in enumerate(slots):
        if 0 <= s < expected[0].shape[0] * page:
            for c in range(4):
                expected[c][s // page, :, s % page] = parts[c][t]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,heads,page,dim", [(1, 1, 8, 32), (7, 3, 8, 96), (64, 8, 16, 128), (130, 2, 64, 64), (33, 1, 16, 256), (5, 5, 1024, 160)])
def test_write_and_read(gpu_lib, t, heads, page, dim, dtype):
    rng = np.random.default_rng(t * dim + heads)
    n_pages = -(-t // page) * 2 + 3
    k, v = rows_of(rng, t, heads, dim, dtype), rows_of(rng, t, heads, dim, dtype)
    slots = rng.permutation(n_pages * page)[:t].astype(np.int32)
    if t > 4:
        slots[[1, 3]] = -1, n_pages * page
    cache = cache_of(n_pages, heads, page, dim)
    want = [c.cpu().numpy() for c in cache]
    parts = [*fast_quantise(k.double().numpy()), *fast_quantise(v.double().numpy())]
    put(want, slots, parts, page)
    d_slots = torch.from_numpy(slots).cuda()
    gpu_lib.rglru_paged_kv_write_q4(k.cuda(), v.cuda(), *cache, d_slots)
    for c in range(4):
        np.testing.assert_array_equal(cache[c].cpu().numpy(), want[c])
    for out in (torch.bfloat16, torch.float32):
        rk, rv = gpu_lib.rglru_paged_kv_read_q4(*cache, d_slots, dtype=out)
        for got, codes, scales in ((rk, *parts[:2]), (rv, *parts[2:])):
            ref = paged_q4.values(codes, scales)
            ref[(slots < 0) | (slots >= n_pages * page)] = 0.0
            np.testing.assert_array_equal(got.cpu().double().numpy(), ref)


def test_the_rule_over_arrays_is_the_oracles():
    x = rows_of(np.random.default_rng(3), 9, 2, 128, torch.float32).double().numpy()
    for a, b in zip(fast_quantise(x), paged_q4.quantise(x)):
        np.testing.assert_array_equal(a, b)


def test_every_code_and_scale_reads_back(gpu_lib):
    """All 256 bytes of codes under all scales that the write gives, and under 0."""
    scales = np.concatenate([np.arange(253), [255]]).astype(np.uint8)
    codes = np.tile(np.arange(256, dtype=np.uint8), (254, 1))   # 512 elements: 16 blocks
    cache = [codes.reshape(254, 1, 1, 256).repeat(8, 2), np.repeat(scales[:, None], 16, 1).reshape(254, 1, 1, 16).repeat(8, 2)] * 2
    cache = [torch.from_numpy(np.ascontiguousarray(c)).cuda() for c in cache]
    slots = torch.arange(0, 254 * 8, 8, dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        for got in gpu_lib.rglru_paged_kv_read_q4(*cache, slots, dtype=dtype):
            np.testing.assert_array_equal(got[:, 0].cpu().double().numpy(), paged_q4.values(codes, np.repeat(scales[:, None], 16, 1)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_numbers(gpu_lib, dtype):
    """Blocks down to the smallest float32, whose powers stop at 2^-126."""
    x = np.zeros((40, 1, 32))
    x[:, 0, 0] = 2.0 ** -np.arange(110.0, 150.0)
    x[:, 0, 1] = -0.75 * x[:, 0, 0]
    k = torch.from_numpy(x).to(dtype)
    cache = cache_of(5, 1, 8, 32)
    gpu_lib.rglru_paged_kv_write_q4(k.cuda(), k.cuda(), *cache, torch.arange(40, dtype=torch.int32, device="cuda"))
    codes, scales = paged_q4.quantise(k.double().numpy())
    np.testing.assert_array_equal(cache[0].cpu().numpy().reshape(40, 1, 16), codes)
    np.testing.assert_array_equal(cache[3].cpu().numpy().reshape(40, 1, 1), scales)


def test_rows_of_a_wider_tensor(gpu_lib):
    rng = np.random.default_rng(8)
    fused = torch.from_numpy(rng.standard_normal((21, 3, 2, 64))).to(torch.bfloat16).cuda()
    slots = torch.from_numpy(rng.permutation(64)[:21].astype(np.int32)).cuda()
    a, b = cache_of(8, 2, 8, 64), cache_of(8, 2, 8, 64)
    gpu_lib.rglru_paged_kv_write_q4(fused[:, 1], fused[:, 2], *a, slots)
    gpu_lib.rglru_paged_kv_write_q4(fused[:, 1].contiguous(), fused[:, 2].contiguous(), *b, slots)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_rows(gpu_lib):
    cache = cache_of(2, 1, 8, 64)
    before = [c.clone() for c in cache]
    none = torch.empty(0, 1, 64, device="cuda")
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    gpu_lib.rglru_paged_kv_write_q4(none, none, *cache, slots)
    assert all(torch.equal(x, y) for x, y in zip(cache, before))
    assert gpu_lib.rglru_paged_kv_read_q4(*cache, slots)[0].shape == (0, 1, 64)


def test_past_32_bit_offsets(gpu_lib):
    """A cache whose codes pass 2^32 bytes: the last slots are written and read, the first ones stay."""
    page, dim = 1024, 256
    n_pages = (1 << 32) // (page * dim // 2) + 2
    codes = torch.zeros(n_pages, 1, page, dim // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_pages, 1, page, dim // 32, dtype=torch.uint8, device="cuda")
    v_codes, v_scales = torch.zeros_like(codes), torch.zeros_like(scales)
    k = rows_of(np.random.default_rng(1), 4, 1, dim, torch.float32)
    last = n_pages * page
    slots = torch.tensor([last - 1, last - page, 0, last - 2 * page - 5], dtype=torch.int32, device="cuda")
    gpu_lib.rglru_paged_kv_write_q4(k.cuda(), k.cuda(), codes, scales, v_codes, v_scales, slots)
    want = paged_q4.values(*fast_quantise(k.double().numpy()))
    for got in gpu_lib.rglru_paged_kv_read_q4(codes, scales, v_codes, v_scales, slots, dtype=torch.float32):
        np.testing.assert_array_equal(got.cpu().double().numpy(), want)
    assert int((scales.view(-1, dim // 32).amax(-1) > 0).sum()) == 4


def test_another_stream_and_replays(gpu_lib):
    rng = np.random.default_rng(2)
    k = rows_of(rng, 32, 2, 128, torch.bfloat16).cuda()
    v = rows_of(rng, 32, 2, 128, torch.bfloat16).cuda()
    slots = torch.from_numpy(rng.permutation(64)[:32].astype(np.int32)).cuda()
    want, got = cache_of(4, 2, 16, 128), cache_of(4, 2, 16, 128)
    rk, rv = (torch.empty(32, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        gpu_lib.rglru_paged_kv_write_q4(k, v, *got, slots)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        gpu_lib.rglru_paged_kv_write_q4(k, v, *got, slots)
        gpu_lib.rglru_paged_kv_read_q4(*got, slots, k=rk, v=rv)
    for step in range(3):
        k.copy_(rows_of(rng, 32, 2, 128, torch.bfloat16))
        slots.copy_(torch.from_numpy(rng.permutation(64)[:32].astype(np.int32)))
        gpu_lib.rglru_paged_kv_write_q4(k, v, *want, slots)
        if step == 0:
            for w, g in zip(want, got):
                w.copy_(g)
            gpu_lib.rglru_paged_kv_write_q4(k, v, *want, slots)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        ek, ev = gpu_lib.rglru_paged_kv_read_q4(*want, slots)
        assert torch.equal(rk.view(torch.int16), ek.view(torch.int16)) and torch.equal(rv.view(torch.int16), ev.view(torch.int16))
