"""Limits of the tree-decoding operators that need no GPU: the softmax reference's raise rule restated
in fp32."""
from __future__ import annotations

import numpy as np
import pytest

pytest.importorskip("torch")

F = np.float32
LOG2E = 1.4426950408889634
UNSET, EXCEED, ROUND_FROM = F(-3.4028235e38), F(30), F(2 ** 24)


def fma(a, b, c):
    """fp32 fma: the product of two fp32 values is exact in 64 mantissa bits."""
    return (a.astype(np.longdouble) * np.longdouble(b) + c.astype(np.longdouble)).astype(F)


def run_of_jobs(z, zs, jobs):
    """The tensor-core path's rule on rows × keys logits, `jobs` keys at a time: a reference per row,
    raised where a logit passes it by 2^30; from references of 2^24 on, every job's references first and
    rounded products.  Returns the references, the sums of the weights, the largest exponent taken."""
    rows, keys = z.shape
    ref, total = np.full(rows, UNSET), np.zeros(rows)
    rounded, most = False, F(-np.inf)
    for k in range(0, keys, jobs):
        s = z[:, k:k + jobs]
        x = None if rounded else fma(s, zs, -ref[:, None])
        if rounded or (x > EXCEED).any():
            top = (s * zs).max(1)
            now = np.maximum(ref, top)
            total *= np.exp2((ref - now).astype(np.float64))
            ref = now
            rounded |= bool(((top > -np.inf) & (np.abs(ref) >= ROUND_FROM)).any())
            x = (s * zs - ref[:, None]) / zs * zs if rounded else fma(s, zs, -ref[:, None])
            assert not (x > EXCEED).any()   # (so no second raise)
        most = max(most, x.max())
        total += np.exp2(x.astype(np.float64)).sum(1)
    return ref, total, most


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("mag", [1.0, 1e3, 1e6, 1.2e7, 3e7, 1e8, 6e8, 6e9, 1e12, 1e20, 1e30, 1e37])
def test_one_raise_a_job_is_enough(mag, sign):
    """Weights stay within 2^30 and every row keeps one of at least 1/2, whatever the logits' size: the
    unrounded product may pass a rounded reference by half its step, hundreds at 1e10."""
    rng = np.random.default_rng(int(np.log2(mag)) + (sign > 0) * 1000)
    z = (F(sign * mag) * (1 + rng.random((64, 512)) ** 2)).astype(F)
    if sign < 0:
        z = z[:, ::-1]
    with np.errstate(over="ignore", under="ignore"):
        for order in (z, np.sort(z, 1)):
            ref, total, most = run_of_jobs(order.astype(F), F(0.08838835 * LOG2E), 128)
            assert most <= EXCEED, float(most)
            assert np.isfinite(total).all() and (total >= 0.5).all(), float(total.min())
            best = (order * F(0.08838835 * LOG2E)).max(1)
            got = ref + np.log2(total)
            assert (np.abs(got - best) <= 10 + np.abs(best) * 2.0 ** -22).all()
