"""Limits of the paged-cache entry points, without a GPU: sizes as documented, and refusals that come before anything is launched."""
import ctypes

import pytest
import torch

import gated_linear_recurrence_amd as glr
from gated_linear_recurrence_amd import _lib


def shape(**kw):
    fields = dict(n_tokens=40, n_pages=100, n_seqs=3, max_pages=30, page_size=16, q_heads=8, kv_heads=2, head_dim=128,
                  io_dtype=_lib.RGLRU_IO_BF16, scale=0.1)
    return _lib.rglru_paged_shape_t(**{**fields, **kw})


def test_workspace_bytes_are_within_what_the_header_says():
    """153 MB, 40 bytes for every row tile (128 rows of float32, 256 of bf16) and 48 for every sequence; 153 MB is not too much by
    more than a hundredth."""
    most = 0
    for io, rows in ((_lib.RGLRU_IO_BF16, 256), (_lib.RGLRU_IO_F32, 128)):
        for dim in (64, 128, 256):
            for n in (1, 16, 17, 1000, 1 << 16):
                for t in (1, 300, 20000, 1 << 22, (1 << 27) - (1 << 13)):
                    for hq, hkv in ((1, 1), (16, 1), (16, 16)):
                        for new in (0, 1):
                            need = glr.rglru_paged_attn_workspace_bytes(shape(
                                n_tokens=t, n_seqs=n, q_heads=hq, kv_heads=hkv, head_dim=dim, io_dtype=io, max_new=new, max_pages=8000))
                            extra = 40 * -(-t * (hq // hkv) // rows) + 48 * n
                            assert 0 < need <= 153e6 + extra, (io, dim, n, t, hq, hkv, new)
                            most = max(most, need - extra)
    assert most > 0.99 * 153e6


def cpu_call(**kw):
    kc, vc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    return glr.rglru_paged_attn_fwd(torch.zeros(3, 4, 64, dtype=torch.bfloat16), kc, vc, i(0, 1).view(1, 2), i(0, 3), i(3), **kw)


def test_a_recurrent_workspace_is_not_taken():
    """The recurrent calls count on what their Workspace holds, so neither it nor its buffer serves as scratch memory here."""
    ws = glr.Workspace("cpu")
    with pytest.raises(TypeError, match="Workspace"):
        cpu_call(workspace=ws)
    buf = ws.get(1 << 20)
    for part in (buf, buf[4096:]):
        with pytest.raises(ValueError, match="Workspace"):
            cpu_call(workspace=part)
    with pytest.raises(ValueError, match="expected a GPU"):   # a buffer of its own passes that check
        cpu_call(workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def raw_attn(s):
    """The library's answer to a call with no workspace, which is refused at the latest for that."""
    at = ctypes.c_void_p(0x100000)
    return _lib.load().rglru_paged_attn_fwd(ctypes.byref(s), *[at] * 9, 0, None)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scales_past_float32_in_log2_units(sign):
    """scale log2 e has to be a float32: 3.4e38 / 1.4427 = 2.3586e38 is the largest."""
    for scale, status in ((2.35e38, 3), (2.37e38, 1), (3.4e38, 1)):
        s = shape(scale=sign * scale)
        assert raw_attn(s) == status
        assert (glr.rglru_paged_attn_workspace_bytes(s) > 0) == (status == 3)


@pytest.mark.parametrize("tokens,heads,dim,io,status", [
    (1 << 24, 128, 16, _lib.RGLRU_IO_BF16, 1), ((1 << 24) - 1, 128, 16, _lib.RGLRU_IO_BF16, 2),
    ((1 << 31) - 1, 2, 4, _lib.RGLRU_IO_F32, 1), ((1 << 31) - 128, 2, 4, _lib.RGLRU_IO_F32, 2), ((1 << 31) - 1, 1 << 14, 64, _lib.RGLRU_IO_F32, 1)])
def test_writes_of_more_threads_than_a_launch_has(tokens, heads, dim, io, status):
    """A thread moves 16 bytes of keys and of values, and a launch has less than 2^32 threads, in blocks of 256: 2^36 - 2^12 bytes of
    keys. A smaller call passes that check (and is refused for its alignment here)."""
    s = shape(n_tokens=tokens, kv_heads=heads, head_dim=dim, io_dtype=io)
    odd = ctypes.c_void_p(0x100008)
    assert _lib.load().rglru_paged_kv_write(ctypes.byref(s), *[odd] * 5, None) == status


def test_sizes_that_do_not_fit_32_bits():
    """Sizes that come from a tensor's shape are checked like those that are passed (they would wrap in the shape's 32-bit fields).
    Tensors without memory stand for the large ones."""
    m = lambda *a, dtype=torch.int32: torch.empty(a, dtype=dtype, device="meta")  # noqa: E731
    big, bf = (1 << 32) + 1, torch.bfloat16
    cache = m(4, 2, 16, 64, dtype=bf)
    attn = [m(3, 4, 64, dtype=bf), cache, cache, m(1, 2), m(2), m(1)]

    def with_(at, *values):
        out = list(attn)
        out[at:at + len(values)] = values
        return out

    for args in (with_(0, m(3, big * 2, 64, dtype=bf)), with_(1, *[m(4, 2, (1 << 32) + 16, 64, dtype=bf)] * 2),
                 with_(0, m(3, 4, (1 << 32) + 64, dtype=bf), *[m(4, 2, 16, (1 << 32) + 64, dtype=bf)] * 2),
                 with_(1, *[m(4, (1 << 32) + 2, 16, 64, dtype=bf)] * 2), with_(3, m(1, big)), with_(3, m(big, 2), m(big + 1), m(big))):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_paged_attn_fwd(*args)
    k = m(3, 2, 64, dtype=bf)
    for kk, c in ((k, m(4, 2, (1 << 32) + 16, 64, dtype=bf)), (m(3, big, 64, dtype=bf), m(4, big, 16, 64, dtype=bf)),
                  (m(3, 2, (1 << 32) + 64, dtype=bf), m(4, 2, 16, (1 << 32) + 64, dtype=bf))):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_paged_kv_write(kk, kk, c, c, m(3))
    for n, width in ((1, big), (big, 1)):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_page_plan(m(n), m(n + 1), m(n, width), m(8), m(1), n_tokens=1, page_size=16)
    with pytest.raises(ValueError, match="expected a GPU"):
        glr.rglru_paged_attn_fwd(*attn)


@pytest.mark.parametrize("io", [_lib.RGLRU_IO_BF16, _lib.RGLRU_IO_F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 4), (16, 16), (80, 2)])
def test_a_workspace_for_a_capacity_serves_smaller_batches(io, dim, hq, hkv):
    """A call of fewer tokens or sequences, or with a smaller bound on a sequence's new tokens, never needs more."""
    for n in (1, 2, 5, 9, 16, 17, 40):
        last = 0
        for t in (1, 2, 5, 16, 17, 33, 64, 100, 333, 1000, 4096, 30000):
            sizes = [glr.rglru_paged_attn_workspace_bytes(shape(n_tokens=t, n_seqs=m, q_heads=hq, kv_heads=hkv, head_dim=dim, io_dtype=io,
                                                                max_new=new, max_pages=600))
                     for m in range(1, n + 1) for new in (1, 2, 20, 300, 0)]
            assert max(sizes[:-1] + [0]) <= sizes[-1] and last <= sizes[-1], (n, t)
            last = sizes[-1]
