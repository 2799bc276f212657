"""The 4-bit cache and the page pool without a GPU: refusals and sizes under host sanitizers, limits, the binding's own checks."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import gated_linear_recurrence_amd as glr
from gated_linear_recurrence_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_linear_recurrence_amd", "csrc")
# sanitizers for the host side of the HIP compile only
HOST_SANITIZE = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]


def test_host_code_under_sanitizers(tmp_path):
    hip = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if hip is None:
        pytest.skip("hipcc not found")
    empty, exe = tmp_path / "empty.gpubin", tmp_path / "q4_check"
    empty.write_bytes(b"")
    cmd = [hip, "--offload-arch=gfx950", "--cuda-host-only", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", str(empty), "-O1",
           "-g", "-std=c++17", "-fno-omit-frame-pointer", *HOST_SANITIZE, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-o",
           str(exe), os.path.join(ROOT, "tests", "host_abi", "q4_check.cpp"),
           *[os.path.join(CSRC, f) for f in ("paged_q4.hip", "paged_attn_q4.hip", "page_pool.hip")]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all passed" in r.stdout, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]


def shape(**kw):
    fields = dict(n_tokens=40, n_pages=100, n_seqs=3, max_pages=30, page_size=16, q_heads=8, kv_heads=2, head_dim=128,
                  io_dtype=_lib.RGLRU_IO_BF16, scale=0.1)
    return _lib.rglru_paged_shape_t(**{**fields, **kw})


def test_workspace_bytes_are_within_what_the_header_says():
    """203 MB, 40 bytes for every row tile (128 rows of float32, 256 of bf16), 48 for every sequence and 8 for every key head of one."""
    most = 0
    for io, rows in ((_lib.RGLRU_IO_BF16, 256), (_lib.RGLRU_IO_F32, 128)):
        for dim in (64, 128, 256):
            for n in (1, 16, 17, 1000, 1 << 16):
                for t in (1, 300, 20000, 1 << 22, (1 << 27) - (1 << 13)):
                    for hq, hkv in ((1, 1), (16, 1), (16, 16)):
                        for new in (0, 1):
                            need = glr.rglru_paged_attn_q4_workspace_bytes(shape(
                                n_tokens=t, n_seqs=n, q_heads=hq, kv_heads=hkv, head_dim=dim, io_dtype=io, max_new=new, max_pages=8000))
                            extra = 40 * -(-t * (hq // hkv) // rows) + 48 * n + 8 * n * hkv
                            assert 0 < need <= 203e6 + extra, (io, dim, n, t, hq, hkv, new, need)
                            most = max(most, need - extra)
    assert most > 0.99 * 203e6, most


@pytest.mark.parametrize("io", [_lib.RGLRU_IO_BF16, _lib.RGLRU_IO_F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 4), (16, 16), (80, 2)])
def test_a_workspace_for_a_capacity_serves_smaller_batches(io, dim, hq, hkv):
    """A call of fewer tokens or sequences, or with a smaller bound on a sequence's new tokens, never needs more."""
    for n in (1, 2, 5, 9, 16, 17, 40):
        last = 0
        for t in (1, 2, 5, 16, 17, 33, 64, 100, 333, 1000, 4096, 30000):
            sizes = [glr.rglru_paged_attn_q4_workspace_bytes(shape(n_tokens=t, n_seqs=m, q_heads=hq, kv_heads=hkv, head_dim=dim,
                                                                   io_dtype=io, max_new=new, max_pages=600))
                     for m in range(1, n + 1) for new in (1, 2, 20, 300, 0)]
            assert max(sizes[:-1] + [0]) <= sizes[-1] and last <= sizes[-1], (n, t)
            last = sizes[-1]


def i32(*a):
    return torch.tensor(a, dtype=torch.int32)


def cache(n=4, heads=2, page=16, dim=64):
    return [torch.zeros(n, heads, page, dim // (32 if c % 2 else 2), dtype=torch.uint8) for c in range(4)]


def refuses(call, good, wrong, **kw):
    for at, x in wrong:
        with pytest.raises((TypeError, ValueError)):
            call(*good[:at], x, *good[at + 1:], **kw)


def test_binding_refuses_before_the_library():
    """Shapes, types and layouts are checked in Python; CPU tensors never reach the library."""
    q, c = torch.zeros(3, 4, 64, dtype=torch.bfloat16), cache()
    bad_cache = lambda at: [(at, x) for x in (None, c[0][0], c[0].float(), c[0].transpose(1, 2), cache(dim=128)[at - 1], cache(n=3)[at - 1])]  # noqa: E731
    good = (q, *c, i32(0, 1).view(1, 2), i32(0, 3), i32(3))
    refuses(glr.rglru_paged_attn_q4_fwd, good, [
        (0, q[:, :, :32]), (0, q.half()), (0, q[0]), (0, q.permute(1, 0, 2)), (0, None), *bad_cache(1)[:4], *bad_cache(2), *bad_cache(3), *bad_cache(4),
        (5, i32(0, 1)), (5, i32(0, 1, 2, 3).view(2, 2)), (5, good[5].long()), (6, i32(0)), (6, good[6].float()), (7, i32(3, 3)), (7, good[7].long())])
    for kw in (dict(window=1 << 32), dict(window=-1), dict(max_new=(1 << 32) + 1), dict(max_new=-1), dict(workspace=glr.Workspace("cpu")),
               dict(workspace=torch.zeros(8))):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_paged_attn_q4_fwd(*good, **kw)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    good = (k, k + 1, *c, i32(0, 1, 2))
    refuses(glr.rglru_paged_kv_write_q4, good, [
        (0, k.half()), (0, None), (0, k[:2]), (1, k.float()), (1, k[:, :1]), (0, k.transpose(0, 1)), (1, k.expand(3, 2, 64).transpose(1, 2)),
        *[(at + 1, x) for at, x in bad_cache(1)[:4] + bad_cache(2) + bad_cache(3) + bad_cache(4)], (6, i32(0, 1)), (6, good[6].long())])
    good = (*c, i32(0, 1, 2))
    refuses(glr.rglru_paged_kv_read_q4, good, [*[(at - 1, x) for at, x in bad_cache(1)[:4] + bad_cache(3)], (4, i32(0).view(1, 1)), (4, good[4].long()), (4, None)])
    for kw in (dict(dtype=torch.float16), dict(k=torch.zeros(3, 2, 64)), dict(v=k[:2])):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_paged_kv_read_q4(*good, **kw)
    with pytest.raises(ValueError, match="blocks of 32"):
        glr.rglru_paged_kv_read_q4(*[torch.zeros(4, 2, 16, 24, dtype=torch.uint8)] * 4, i32(0))
    n, p = 3, 10
    table, lens, pages = torch.zeros(n, 2, dtype=torch.int32), i32(0, 1, 2), torch.zeros(p, dtype=torch.int32)
    wrong_pool = [(1, lens[:2]), (1, lens.long()), (2, table[0]), (2, table[:2]), (2, table.long()), (3, pages[:5]), (3, None), (4, pages.view(2, 5)),
                  (4, pages[:5]), (5, i32(1, 1)), (5, None)]
    good = (lens, lens, table, pages, pages, i32(1))
    refuses(glr.rglru_page_fork, good, wrong_pool + [(0, lens[:2]), (0, None)], page_size=16)
    refuses(glr.rglru_page_free, good, wrong_pool + [(0, lens[:2]), (0, lens.long())], page_size=16)
    refuses(glr.rglru_page_compact, good[1:], [(at - 1, x) for at, x in wrong_pool], page_size=16, keep_pages=5)
    for kw in (dict(keep_pages=11), dict(keep_pages=-1), dict(keep_pages=5, pairs=torch.zeros(4, 2, dtype=torch.int32)), dict(keep_pages=5, n_pairs=i32(0, 0)),
               dict(keep_pages=5, block_table_out=table[:2]), dict(keep_pages=5, workspace=glr.Workspace("cpu"))):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_page_compact(*good[1:], page_size=16, **kw)
    for call, kw in ((glr.rglru_page_fork, dict(pairs=lens)), (glr.rglru_page_fork, dict(held_lens=lens[:1])), (glr.rglru_page_fork, dict(unserved=lens)),
                     (glr.rglru_page_free, dict(held_lens_out=lens[:1])), (glr.rglru_page_free, dict(workspace=lens))):
        with pytest.raises((TypeError, ValueError)):
            call(*good, page_size=16, **kw)
    pairs = torch.zeros(5, 2, dtype=torch.int32)
    for args, kw in (((pairs, []), {}), ((pairs, [c[0], None]), {}), ((pairs, [c[0], c[1][:2]]), {}), ((pairs, [c[0].transpose(0, 1)]), {}), ((pairs[:, :1], c), {}),
                     ((pairs.long(), c), {}), ((pairs.flatten(), c), {}), ((pairs, c), dict(n_pairs=i32(1, 2))), ((pairs, [c[0][:0]]), {}), ((pairs, [torch.tensor(1)]), {})):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_page_copy(*args, **kw)


def test_valid_arguments_on_the_cpu_are_refused():
    """A call that is right in everything but where its tensors live raises ValueError, with no GPU touched."""
    q, c, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), cache(), torch.zeros(3, 2, 64)
    table, lens, pages = torch.zeros(3, 2, dtype=torch.int32), i32(0, 1, 2), [torch.zeros(10, dtype=torch.int32) for _ in range(2)]
    for call in (lambda: glr.rglru_paged_attn_q4_fwd(q, *c, i32(0, 1).view(1, 2), i32(0, 3), i32(3)),
                 lambda: glr.rglru_paged_kv_write_q4(k, k + 1, *c, i32(0, 1, 2)), lambda: glr.rglru_paged_kv_read_q4(*c, i32(0, 1, 2)),
                 lambda: glr.rglru_page_fork(lens, lens, table, *pages, i32(1), page_size=16),
                 lambda: glr.rglru_page_free(lens, lens, table, *pages, i32(1), page_size=16),
                 lambda: glr.rglru_page_compact(lens, table, *pages, i32(1), page_size=16, keep_pages=4),
                 lambda: glr.rglru_page_copy(torch.zeros(5, 2, dtype=torch.int32), c)):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()


def test_sizes_that_do_not_fit_32_bits():
    """Sizes that come from a tensor's shape are checked like those that are passed. Tensors without memory stand for the large ones."""
    m = lambda *a, dtype=torch.int32: torch.empty(a, dtype=dtype, device="meta")  # noqa: E731
    u8 = torch.uint8
    mc = lambda n, h, p, d: [m(n, h, p, d // (32 if c % 2 else 2), dtype=u8) for c in range(4)]  # noqa: E731
    big = (1 << 32) + 1
    for c in (mc(4, big, 16, 64), mc(4, 2, (1 << 32) + 16, 64), mc(4, 2, 16, (1 << 32) + 64)):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_paged_kv_read_q4(*c, m(3))
    for n, width in ((1, big), (big, 1)):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_page_fork(m(n), m(n), m(n, width), m(8), m(8), m(1), page_size=16)
    for args in ((m(big, 2), [m(4, 8)]), (m(3, 2), [m(big, 8)])):
        with pytest.raises(ValueError, match=r"2\^31"):
            glr.rglru_page_copy(*args)


def test_status_of_a_raw_call():
    """The copy's arrays are read on the host: no GPU is needed to refuse one."""
    arrays, sizes = (ctypes.c_void_p * 1)(0x100000), (ctypes.c_int64 * 1)(24)
    assert _lib.load().rglru_page_copy(10, None, 0, None, 1, arrays, sizes, None) == 1
