"""Shared by the paged-cache tests: a random batch on the host, its device copy, the oracle's answer and the error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as oracle_paged

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


class Batch:
    """Sequences of (context, new) tokens over a cache whose pages are in random order.

    Everything a sequence does not own (other pages, offsets past its length) holds `garbage`.
    """

    def __init__(self, ctx, new, *, hq, hkv, dim, page, dtype=torch.bfloat16, pad=0, seed=0, garbage=float("nan"),
                 kv_lens=None, spare=2, q_extra=0, device="cuda"):
        rng = np.random.default_rng(seed)
        n = len(ctx)
        self.new, self.page, self.hq, self.hkv, self.dim, self.dtype = list(new), page, hq, hkv, dim, dtype
        self.kv = [c + m for c, m in zip(ctx, new)] if kv_lens is None else list(kv_lens)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.cu[-1])
        rows = self.tokens + pad
        width = max(1, max(-(-max(x, 0) // page) for x in self.kv)) + 1
        n_pages = n * width + spare
        order = rng.permutation(n_pages)
        table = order[: n * width].reshape(n, width).astype(np.int32)
        t64 = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype)  # noqa: E731
        kc = torch.full((n_pages, hkv, page, dim), garbage, dtype=dtype)
        vc = torch.full((n_pages, hkv, page, dim), garbage, dtype=dtype)
        self.k, self.v = [], []
        for i in range(n):
            k, v = t64(max(self.kv[i], 0), hkv, dim), t64(max(self.kv[i], 0), hkv, dim)
            self.k.append(k)
            self.v.append(v)
            for c in range(-(-max(self.kv[i], 0) // page)):
                part = slice(c * page, min((c + 1) * page, self.kv[i]))
                m = part.stop - part.start
                kc[table[i, c], :, :m] = k[part].permute(1, 0, 2)
                vc[table[i, c], :, :m] = v[part].permute(1, 0, 2)
        wide = t64(rows, hq * dim + q_extra)
        self.q = wide[:, : hq * dim].view(rows, hq, dim)
        self.table = table
        self.d_q = wide.to(device)[:, : hq * dim].unflatten(1, (hq, dim))
        self.d_k, self.d_v = kc.to(device), vc.to(device)
        self.d_table = torch.from_numpy(table).to(device)
        self.d_cu = torch.from_numpy(self.cu).to(device)
        self.d_kv = torch.tensor(self.kv, dtype=torch.int32, device=device)

    def put(self, i, j, *, k=None, v=None, heads=slice(None), dims=slice(None)):
        """Overwrites key or value j of sequence i, on both sides."""
        page, off = int(self.table[i, j // self.page]), j % self.page
        for val, host, dev in ((k, self.k, self.d_k), (v, self.v, self.d_v)):
            if val is not None:
                host[i][j, heads, dims] = val
                dev[page, heads, off, dims] = val

    def call(self, glr, window=0, scale=None, **kw):
        rows = self.q.shape[0]
        o = torch.full((rows, self.hq, self.dim), 7.0, dtype=self.dtype, device=self.d_q.device)
        lse = torch.full((rows, self.hq), 7.0, device=self.d_q.device)
        kw.setdefault("max_new", max(1, max(self.new)))
        return glr.rglru_paged_attn_fwd(self.d_q, self.d_k, self.d_v, self.d_table, self.d_cu, self.d_kv, window=window,
                                        scale=scale, o=o, lse=lse, **kw)

    def check(self, o, lse, window=0, scale=None):
        """Holds every row to the oracle.

        Bound of a row that sees n keys, with A = sum p|v| per column and S the largest scale * sum |q||k|:
        a float32 score is off by at most e = (D + 8) 2^-24 S (products, sum, scale and log2 e, argument of exp2), a
        weight relative to its sum by 2 e plus (n + 8) 2^-23 (both sums, exp2, rescaling, division); bf16 adds half a step to every
        weight (2^-8 A) and to the result (2^-8 |o|), float32 half a step to the result.
        """
        scale = self.dim ** -0.5 if scale is None else scale
        half = HALF[self.dtype]
        o64, lse64 = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (o64[self.tokens:] == 7.0).all() and (lse64[self.tokens:] == 7.0).all(), "padding rows were written"
        for i, m in enumerate(self.new):
            if m == 0:
                continue
            rows = slice(int(self.cu[i]), int(self.cu[i + 1]))
            k, v = (t[i].double().numpy().transpose(1, 0, 2) for t in (self.k, self.v))
            q = self.q[rows].double().numpy()
            with np.errstate(invalid="ignore", over="ignore"):
                ref, ref_lse, weight, size, seen = oracle_paged.attention(q, k, v, self.kv[i], window, scale)
            fin = np.where(np.isfinite(size), size, 0.0)
            e = (self.dim + 8) * 2.0 ** -24 * fin
            rel = 2 * e + ((seen + 8) * 2.0 ** -23)[:, None]
            tol = rel[..., None] * weight + half * np.abs(ref) * 1.01 + 1e-38
            if self.dtype == torch.bfloat16:
                tol += half * weight * 1.01
            with np.errstate(invalid="ignore"):
                err = np.abs(o64[rows] - ref)
                same = (err <= tol) | (np.isnan(ref) & np.isnan(o64[rows])) | (ref == o64[rows])
            assert same.all(), (i, np.argwhere(~same)[:5], o64[rows][~same][:5], ref[~same][:5], tol[~same][:5])
            with np.errstate(invalid="ignore"):
                err = np.abs(lse64[rows] - ref_lse)
                ltol = e + ((seen + 8) * 2.0 ** -23)[:, None] + np.abs(ref_lse) * 2.0 ** -22
                same = (err <= ltol) | (np.isnan(ref_lse) & np.isnan(lse64[rows])) | (ref_lse == lse64[rows])
            assert same.all(), (i, "lse", np.argwhere(~same)[:5], lse64[rows][~same][:5], ref_lse[~same][:5])
