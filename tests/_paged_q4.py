"""Shared by the 4-bit cache's tests: a random batch over a 4-bit cache, its device copy, the oracle's answer, error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as oracle_paged
from oracle import paged_q4

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def fast_quantise(x):
    """The oracle's rule over whole arrays (held to it in the tests), for inputs too many for its loops."""
    b = np.asarray(x, np.float64).reshape(-1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(b).max(-1)
        odd = ~np.isfinite(top)
        top[odd] = 0.0
        frac, exp = np.frexp(top)   # top = frac 2^exp, frac in [0.5, 1), or 0
        e = np.where(top == 0.0, -126, np.clip(exp - 3 + (frac > 0.75), -126, 125))
        y = np.abs(np.where(odd[:, None], 0.0, b)) / 2.0 ** e[:, None].astype(float)
    code = sum([y > 0.25, y >= 0.75, y > 1.25, y >= 1.75, y > 2.5, y >= 3.5, y > 5.0]).astype(np.uint8)
    code |= (np.signbit(b) & ~odd[:, None]).astype(np.uint8) << 3
    code = code.reshape(*np.shape(x)[:-1], np.shape(x)[-1] // 2, 2)
    return code[..., 0] | code[..., 1] << 4, np.where(odd, 255, e + 127).astype(np.uint8).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // 32)


class Q4Batch:
    """Sequences of (context, new) tokens over a 4-bit cache whose pages are in random order.

    Everything a sequence does not own (other pages, offsets past its length) holds random codes and scales of
    `garbage` (255: NaN).
    """

    def __init__(self, ctx, new, *, hq, hkv, dim, page, dtype=torch.bfloat16, pad=0, seed=0, garbage=255, kv_lens=None,
                 spare=2, q_extra=0, spread=1.0, device="cuda"):
        rng = np.random.default_rng(seed)
        n = len(ctx)
        self.new, self.page, self.hq, self.hkv, self.dim, self.dtype = list(new), page, hq, hkv, dim, dtype
        self.kv = [c + m for c, m in zip(ctx, new)] if kv_lens is None else list(kv_lens)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.cu[-1])
        rows = self.tokens + pad
        width = max(1, max(-(-max(x, 0) // page) for x in self.kv)) + 1
        n_pages = n * width + spare
        self.table = rng.permutation(n_pages)[: n * width].reshape(n, width).astype(np.int32)
        shape = (n_pages, hkv, page)
        self.cache = [rng.integers(0, 256, (*shape, dim // 2)).astype(np.uint8), np.full((*shape, dim // 32), garbage, np.uint8),
                      rng.integers(0, 256, (*shape, dim // 2)).astype(np.uint8), np.full((*shape, dim // 32), garbage, np.uint8)]
        for i in range(n):
            for which in (0, 2):
                # blocks of one head differ in size
                x = rng.standard_normal((max(self.kv[i], 0), hkv, dim // 32, 32)) * spread ** rng.standard_normal((1, hkv, dim // 32, 1))
                codes, scales = fast_quantise(x.reshape(-1, hkv, dim))
                for c in range(-(-max(self.kv[i], 0) // page)):
                    part = slice(c * page, min((c + 1) * page, self.kv[i]))
                    m = part.stop - part.start
                    self.cache[which][self.table[i, c], :, :m] = codes[part].transpose(1, 0, 2)
                    self.cache[which + 1][self.table[i, c], :, :m] = scales[part].transpose(1, 0, 2)
        wide = torch.from_numpy(rng.standard_normal((rows, hq * dim + q_extra))).to(dtype)
        self.q = wide[:, : hq * dim].view(rows, hq, dim)
        self.device = device
        self.d_q = wide.to(device)[:, : hq * dim].unflatten(1, (hq, dim))
        self.d_cache = [torch.from_numpy(c).to(device) for c in self.cache]
        self.d_table = torch.from_numpy(self.table).to(device)
        self.d_cu = torch.from_numpy(self.cu).to(device)
        self.d_kv = torch.tensor(self.kv, dtype=torch.int32, device=device)

    def put(self, i, j, *, k_scale=None, v_scale=None, k_codes=None, v_codes=None, heads=slice(None), blocks=slice(None)):
        """Overwrites scales or codes of token j of sequence i, on both sides."""
        at = (int(self.table[i, j // self.page]), heads, j % self.page)
        for which, val in ((0, k_codes), (1, k_scale), (2, v_codes), (3, v_scale)):
            if val is not None:
                where = (*at, blocks) if which % 2 else at
                self.cache[which][where] = val
                self.d_cache[which][where] = torch.as_tensor(val, dtype=torch.uint8, device=self.device)

    def call(self, glr, window=0, scale=None, **kw):
        rows = self.q.shape[0]
        o = torch.full((rows, self.hq, self.dim), 7.0, dtype=self.dtype, device=self.d_q.device)
        lse = torch.full((rows, self.hq), 7.0, device=self.d_q.device)
        kw.setdefault("max_new", max(1, max(self.new)))
        return glr.rglru_paged_attn_q4_fwd(self.d_q, *self.d_cache, self.d_table, self.d_cu, self.d_kv, window=window,
                                           scale=scale, o=o, lse=lse, **kw)

    def check(self, o, lse, window=0, scale=None):
        """Holds every row to the oracle (see hold)."""
        scale = self.dim ** -0.5 if scale is None else scale
        o64, lse64 = o.cpu().double().numpy(), lse.cpu().double().numpy()
        assert (o64[self.tokens:] == 7.0).all() and (lse64[self.tokens:] == 7.0).all(), "padding rows were written"
        for i, m in enumerate(self.new):
            if m == 0:
                continue
            rows = slice(int(self.cu[i]), int(self.cu[i + 1]))
            k, v = (paged_q4.values(oracle_paged.gather(self.cache[x], self.table[i], max(self.kv[i], 0)),
                                    oracle_paged.gather(self.cache[x + 1], self.table[i], max(self.kv[i], 0))) for x in (0, 2))
            hold(o64[rows], lse64[rows], self.q[rows].double().numpy(), k, v, self.kv[i], window, scale, self.dtype, i)


def hold(o, lse, q, k, v, kv, window, scale, dtype, name=""):
    """Holds the rows of one sequence, q [m, Hq, D] over k, v [Hkv, kv, D], to the oracle.

    Bound of a row that sees n keys, with A = sum p|v| per column and S the largest scale * sum |q||k|. Products of q
    (float32: of its three bf16 parts, whose sizes add up to |q| (1 + 2^-7) at most) and a value of the cache are exact, each of the
    c D sums (c = 1, float32 3) is off by at most 2^-24 of S: a score by e = (c D + 16) 2^-24 S, with scale, log2 e and the
    argument of exp2; a weight relative to its sum by 2 e plus (c n + 16) 2^-23 (both sums, exp2, rescaling, merging,
    division); bf16 adds half a step to every weight (2^-8 A; the block's power is exact) and to the result (2^-8 |o|),
    float32 half a step to the result.
    """
    half, c, dim = HALF[dtype], 1 if dtype == torch.bfloat16 else 3, q.shape[2]
    with np.errstate(invalid="ignore", over="ignore"):
        ref, ref_lse, weight, size, seen = oracle_paged.attention(q, k, v, kv, window, scale)
    fin = np.where(np.isfinite(size), size, 0.0)
    e = (c * dim + 16) * 2.0 ** -24 * fin
    rel = 2 * e + ((c * seen + 16) * 2.0 ** -23)[:, None]
    tol = rel[..., None] * weight + half * np.abs(ref) * 1.01 + 1e-38
    if dtype == torch.bfloat16:
        tol += half * weight * 1.01
    with np.errstate(invalid="ignore"):
        same = (np.abs(o - ref) <= tol) | (np.isnan(ref) & np.isnan(o)) | (ref == o)
    assert same.all(), (name, np.argwhere(~same)[:5], o[~same][:5], ref[~same][:5], tol[~same][:5])
    with np.errstate(invalid="ignore"):
        ltol = e + ((c * seen + 16) * 2.0 ** -23)[:, None] + np.abs(ref_lse) * 2.0 ** -22
        same = (np.abs(lse - ref_lse) <= ltol) | (np.isnan(ref_lse) & np.isnan(lse)) | (ref_lse == lse)
    assert same.all(), (name, "lse", np.argwhere(~same)[:5], lse[~same][:5], ref_lse[~same][:5])
