"""The strict check of paged attention: it agrees with the oracle, and it rejects what is wrong where an answer is not finite."""
import numpy as np
import pytest
import torch

from _paged_strict import StrictBatch, expected
from oracle import paged as oracle_paged

INF, NAN = float("inf"), float("nan")


def answers(b, window=0):
    """What a call would return, from the definition, with the padding rows' 7."""
    o = torch.full((b.q.shape[0], b.hq, b.dim), 7.0, dtype=torch.float64)
    lse = torch.full((b.q.shape[0], b.hq), 7.0, dtype=torch.float64)
    for i, m in enumerate(b.new):
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        k, v = (t[i].double().numpy().transpose(1, 0, 2) for t in (b.k, b.v))
        r = expected(b.q[rows].double().numpy(), k, v, b.kv[i], window, b.dim ** -0.5)
        o[rows], lse[rows] = torch.from_numpy(r["o"]), torch.from_numpy(r["lse"])
    return o, lse


def batch():
    b = StrictBatch([40, 0], [3, 4], hq=4, hkv=2, dim=64, page=16, kv_lens=[43, 2], pad=2, dtype=torch.float32, seed=1, device="cpu")
    b.put(0, 5, v=INF, dims=3)
    b.put(0, 41, v=-INF, dims=9)
    b.put(0, 7, v=INF, dims=20)
    b.put(0, 8, v=-INF, dims=20)
    b.put(0, 9, v=NAN, heads=1, dims=30)
    return b


@pytest.mark.parametrize("window", [0, 30])
def test_the_definition_agrees_with_the_oracle(window):
    b = batch()
    for i in range(2):
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        q, (k, v) = b.q[rows].double().numpy(), (t[i].double().numpy().transpose(1, 0, 2) for t in (b.k, b.v))
        with np.errstate(invalid="ignore"):
            o, lse, _, size, seen = oracle_paged.attention(q, k, v, b.kv[i], window, 0.125)
        r = expected(q, k, v, b.kv[i], window, 0.125)
        assert np.allclose(r["o"], o, rtol=0, atol=1e-13, equal_nan=True)
        # the sums of both go in orders of their own: 64 products of a score of 20 at most and 43 weights, 2^-53 each
        assert (np.isinf(r["lse"]) == np.isinf(lse)).all() and size.max() < 20
        assert np.allclose(r["lse"], lse, rtol=0, atol=(64 * 20 + 43) * 2.0 ** -53)
        assert np.allclose(r["size"], size, rtol=64 * 2.0 ** -53) and (r["seen"] == seen).all()


def test_it_passes_the_answers_and_rejects_others():
    b = batch()
    o, lse = answers(b)
    assert torch.isinf(o).any() and torch.isnan(o).any() and (lse == -INF).sum() == 8
    b.check(o, lse)
    inf, nan, none = torch.isinf(o), torch.isnan(o), lse == -INF
    for wrong in (torch.where(inf, 0.5, o), torch.where(inf, -o, o), torch.where(inf, NAN, o), torch.where(nan, 0.5, o),
                  torch.where(nan, INF, o), torch.where(none[..., None], NAN, o), torch.where(none[..., None], 1e-3, o)):
        with pytest.raises(AssertionError):
            b.check(wrong, lse)
    for wrong in (torch.where(none, 3.0, lse), torch.where(none, INF, lse), torch.where(none, NAN, lse)):
        with pytest.raises(AssertionError):
            b.check(o, wrong)
    o[0, 0, 0] += 1e-3
    with pytest.raises(AssertionError):
        b.check(o, lse)


def test_faint_weights():
    """An infinite value whose weight underflows stands for infinity or NaN, never for a number; a finite one for nothing."""
    b = StrictBatch([63], [1], hq=1, hkv=1, dim=64, page=16, dtype=torch.float32, seed=2, device="cpu")
    b.q.fill_(1.0)
    b.put(0, 5, k=-200.0)             # a score of -1600
    b.put(0, 5, v=INF, dims=0)
    b.put(0, 6, k=20.0)               # 160, far above the others
    o, lse = answers(b)
    b.check(o, lse)
    for value, fine in ((NAN, True), (0.0, False), (-INF, False)):
        o[0, 0, 0] = value
        if fine:
            b.check(o, lse)
        else:
            with pytest.raises(AssertionError):
                b.check(o, lse)
