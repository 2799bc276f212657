"""A check of paged attention that also holds where the answer is not finite, or its inputs are near a type's largest value."""
from __future__ import annotations

import numpy as np
import torch

from _paged import HALF, Batch

FAINT = 2.0 ** -117   # weights of 2^-118 of a row's largest may count as nothing; a factor 2 for the scores' own error


def expected(q, k, v, kv_len, window, scale):
    """One sequence from the definition in float64: q [m, Hq, D], k and v [Hkv, kv_len, D].

    Returns a dict of o and lse; weight, size and seen as oracle.paged.attention has them, over what is finite; faint:
    what weights below FAINT add at most; loose: where o is infinite by a weight below FAINT, so that NaN stands for it too.
    """
    m, hq, d = q.shape
    g = hq // k.shape[0]
    r = {x: np.zeros((m, hq, d)) for x in ("o", "weight", "faint")}
    r.update(loose=np.zeros((m, hq, d), bool), lse=np.full((m, hq), -np.inf), size=np.zeros((m, hq)))
    p = kv_len - m + np.arange(m)[:, None]
    j = np.arange(kv_len)
    sees = (j <= p) & (j > p - window if window else True)
    r["seen"] = sees.sum(1)
    some = r["seen"] > 0
    if not some.any():
        return r
    for h in range(hq):
        kk, vv = k[h // g], v[h // g]
        with np.errstate(invalid="ignore"):
            s = np.where(sees, scale * (q[:, h] @ kk.T), -np.inf)
            size = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
            top = s.max(1)
            w = np.exp(s - np.where(top == -np.inf, 0.0, top)[:, None])
            r["size"][:, h] = np.where(sees & np.isfinite(size), size, 0.0).max(1)
        alive = some & (top != -np.inf)
        bad = alive & (np.isnan(top) | (top == np.inf))
        w = np.where((alive & ~bad)[:, None], w, 0.0)
        total = np.where(alive & ~bad, w.sum(1), 1.0)
        odd = ~np.isfinite(vv)
        fin = np.where(odd, 0.0, vv)
        part = w / total[:, None]
        o, size = part @ fin, np.abs(fin)
        r["weight"][:, h] = part @ size
        r["faint"][:, h] = np.where(w < FAINT, part, 0.0) @ size
        hit = np.flatnonzero(odd.any(1))
        for n in hit:   # the few keys with such a value
            see, at = (sees[:, n] & alive)[:, None], odd[n] & ~np.isnan(vv[n])
            with np.errstate(invalid="ignore"):
                o = np.where(see & odd[n], np.where(np.isfinite(o), 0.0, o) + vv[n], o)
            r["loose"][:, h] |= see & at & (w[:, n] < FAINT)[:, None]
        o[bad] = np.nan
        r["o"][:, h] = o
        r["lse"][:, h] = np.where(bad, np.nan, np.where(alive, np.where(alive, top, 0.0) + np.log(total), -np.inf))
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
            e = (self.dim + 8) * 2.0 ** -24 * r["size"]
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
