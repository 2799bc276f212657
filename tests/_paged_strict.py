"""A check of paged attention that also holds where the answer is not finite, or its inputs are near a type's largest value."""
from __future__ import annotations

import numpy as np
import torch

from _paged import HALF, Batch

FAINT = 2.0 ** -117   # weights of 2^-118 of a row's largest may count as nothing; a factor 2 for the scores' own error


def expected(q, k, v, kv_len, window, scale):
    """One sequence from the definition in float64: q [m, Hq, D], k and v [Hkv, kv_len, D].

    Returns a dict of o and lse; weight, size and seen as oracle.paged.attention has them, over the finite values; faint:
    what weights below FAINT add at most; loose: where o is infinite by a weight below FAINT, so that NaN stands for it too.
    """
    m, hq, d = q.shape
    g = hq // k.shape[0]
    r = {x: np.zeros((m, hq, d)) for x in ("o", "weight", "faint")}
    r.update(loose=np.zeros((m, hq, d), bool), lse=np.full((m, hq), -np.inf), size=np.zeros((m, hq)), seen=np.zeros(m, np.int64))
    for i in range(m):
        p = kv_len - m + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        r["seen"][i] = p + 1 - lo
        for h in range(hq):
            kk, vv = k[h // g, lo:p + 1], v[h // g, lo:p + 1]
            with np.errstate(invalid="ignore"):
                s = scale * (kk @ q[i, h])
                r["size"][i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            if (s == -np.inf).all():
                continue
            if np.isnan(s).any() or (s == np.inf).any():
                r["o"][i, h] = r["lse"][i, h] = np.nan
                continue
            w = np.exp(s - s.max())
            total = w.sum()
            r["lse"][i, h] = s.max() + np.log(total)
            fin = np.where(np.isfinite(vv), vv, 0.0)
            o = (w / total) @ fin
            r["weight"][i, h] = (w / total) @ np.abs(fin)
            r["faint"][i, h] = (np.where(w < FAINT, w, 0.0) / total) @ np.abs(fin)
            up, down, nan = vv == np.inf, vv == -np.inf, np.isnan(vv)
            o[up.any(0)] = np.inf
            o[down.any(0)] = -np.inf
            o[nan.any(0) | (up.any(0) & down.any(0))] = np.nan
            r["o"][i, h] = o
            r["loose"][i, h] = ((up | down) & (w < FAINT)[:, None]).any(0)
    return r


class StrictBatch(Batch):
    def check(self, o, lse, window=0, scale=None):
        """Holds every row to the definition.

        Finite answers: the bounds of Batch.check, and what weights of 2^-118 of the row's largest and less add. Others: the same
        infinity or NaN, and either where an infinite value has such a weight.
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
            r = expected(self.q[rows].double().numpy(), k, v, self.kv[i], window, scale)
            ref, ref_lse = r["o"], r["lse"]
            e = (self.dim + 8) * 2.0 ** -24 * np.where(np.isfinite(r["size"]), r["size"], 0.0)
            sums = ((r["seen"] + 8) * 2.0 ** -23)[:, None]
            fin, lfin = np.isfinite(ref), np.isfinite(ref_lse)
            size = np.where(fin, np.abs(ref), 0.0)
            tol = (2 * e + sums)[..., None] * r["weight"] + half * size * 1.01 + r["faint"] * 1.01 + 1e-38
            if self.dtype == torch.bfloat16:
                tol += half * r["weight"] * 1.01
            got, glse = o64[rows], lse64[rows]
            with np.errstate(invalid="ignore"):
                same = np.where(fin, np.abs(got - ref) <= tol,
                                (got == ref) | (np.isnan(got) & (np.isnan(ref) | r["loose"])))
                ltol = e + sums + np.where(lfin, np.abs(ref_lse), 0.0) * 2.0 ** -22
                lsame = np.where(lfin, np.abs(glse - ref_lse) <= ltol, (glse == ref_lse) | (np.isnan(glse) & np.isnan(ref_lse)))
            assert same.all(), (i, np.argwhere(~same)[:5], got[~same][:5], ref[~same][:5], tol[~same][:5])
            assert lsame.all(), (i, "lse", np.argwhere(~lsame)[:5], glse[~lsame][:5], ref_lse[~lsame][:5])
