"""The paged-cache entry points without a GPU: refusals and sizes under host sanitizers, and the binding's own checks."""
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
    empty, exe = tmp_path / "empty.gpubin", tmp_path / "paged_check"
    empty.write_bytes(b"")
    cmd = [hip, "--offload-arch=gfx950", "--cuda-host-only", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", str(empty), "-O1",
           "-g", "-std=c++17", "-fno-omit-frame-pointer", *HOST_SANITIZE, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-o",
           str(exe), os.path.join(ROOT, "tests", "host_abi", "paged_check.cpp"), os.path.join(CSRC, "paged_cache.hip"),
           os.path.join(CSRC, "paged_attn.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "all passed" in r.stdout, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]


def test_struct_matches_the_header():
    """Field order and size of the binding's struct: 8-byte fields first and last, ten 4-byte ones between."""
    s = _lib.rglru_paged_shape_t
    assert ctypes.sizeof(s) == 72
    assert [s.n_tokens.offset, s.n_pages.offset, s.n_seqs.offset, s.scale.offset, s.q_stride.offset, s.kv_stride.offset] == [0, 8, 16, 52, 56, 64]


def test_workspace_bytes():
    shape = _lib.rglru_paged_shape_t(64, 1000, 64, 512, 16, 32, 8, 128, _lib.RGLRU_IO_BF16, 1, 0, 0.1, 0, 0)
    decode = glr.rglru_paged_attn_workspace_bytes(shape)
    shape.max_new = 0
    assert 0 < decode < glr.rglru_paged_attn_workspace_bytes(shape)
    shape.head_dim = 80
    assert glr.rglru_paged_attn_workspace_bytes(shape) == 0


def test_binding_refuses_before_the_library():
    """Shapes, types and layouts are checked in Python; CPU tensors never reach the library."""
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    good = (q, kc, kc, i(0, 1).view(1, 2), i(0, 3), i(3))
    for n, wrong in ((0, q[:, :, :32]), (0, q.half()), (0, q[0]), (0, q.permute(1, 0, 2)), (0, None), (1, kc[0]), (1, kc.half()),
                     (1, kc.transpose(1, 2)), (2, kc[:2]), (2, kc.float()), (3, i(0, 1)), (3, i(0, 1, 2, 3).view(2, 2)),
                     (3, good[3].long()), (4, i(0)), (4, good[4].float()), (5, i(3, 3)), (5, good[5].long())):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_paged_attn_fwd(*good[:n], wrong, *good[n + 1:])
    for kw in (dict(window=1 << 32), dict(window=-1), dict(max_new=(1 << 32) + 1), dict(max_new=-1)):
        with pytest.raises(ValueError):
            glr.rglru_paged_attn_fwd(*good, **kw)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for args in ((k, k[:2], kc, kc, i(0, 1, 2)), (k, k.float(), kc, kc, i(0, 1, 2)), (k, k, kc, kc, i(0, 1)), (k[:, :1], k, kc, kc, i(0, 1, 2)),
                 (k.expand(3, 2, 64).transpose(1, 2), k, kc, kc, i(0, 1, 2)), (k[:1].expand(3, 2, 64), k[:1].expand(3, 2, 64), kc, kc, i(0, 1, 2))):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_paged_kv_write(*args)
    plan = dict(context_lens=i(0), cu_seqlens=i(0, 1), block_table=i(0).view(1, 1), free_pages=i(0), free_count=i(1), n_tokens=1, page_size=16)
    for bad in (dict(context_lens=i(0, 0)), dict(cu_seqlens=i(0)), dict(block_table=i(0)), dict(free_pages=i(0).view(1, 1)),
                dict(free_count=i(1, 1)), dict(held_lens=i(0, 0)), dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(page_size=1 << 32),
                dict(max_new=(1 << 32) + 1), dict(slot_map=i(0, 0))):
        with pytest.raises((TypeError, ValueError)):
            glr.rglru_page_plan(**{**plan, **bad})


def test_valid_arguments_on_the_cpu_are_refused():
    """A call that is right in everything but where its tensors live raises ValueError, with no GPU touched."""
    kc, vc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected a GPU"):
        glr.rglru_paged_attn_fwd(k, kc, vc, i(0, 1).view(1, 2), i(0, 3), i(3))
    with pytest.raises(ValueError, match="expected a GPU"):
        glr.rglru_paged_kv_write(k, k + 1, kc, vc, i(0, 1, 2))
    with pytest.raises(ValueError, match="expected a GPU"):
        glr.rglru_page_plan(i(0), i(0, 1), i(0).view(1, 1), i(0), i(1), n_tokens=1, page_size=16)
