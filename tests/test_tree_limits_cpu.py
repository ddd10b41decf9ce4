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


# ------------------------------------------------ buffers of the in-place calls

MB = 1 << 20
COMMIT = dict(kpool=512 * MB, vpool=640 * MB, n_slots=1 << 12, block_table=1 * MB, max_blocks=8,
              ctx_len=2 * MB, q_off=3 * MB, path=4 * MB, n_path=5 * MB, max_path=4, n_req=2, L=3, H=2,
              D=128, block_size=16, seq_out=6 * MB, row_idx=7 * MB, row_vis=8 * MB, dev_status=None,
              stream=None)
EVICT = dict(kpool=512 * MB, vpool=640 * MB, n_slots=1 << 12, block_table=1 * MB, max_blocks=8,
             seqused_k=2 * MB, n_pos=3 * MB, t_end=4 * MB, mass=5 * MB, pos=6 * MB, mass_out=7 * MB,
             pos_out=8 * MB, n_out=9 * MB, n_req=2, L=3, H=2, D=128, block_size=16, budget=64, n_sink=4,
             n_recent=8, ws=None, ws_bytes=0, dev_status=None, stream=None)
ROWS = 3 * 2 * 2 * 8 * 16 * 4   # bytes of a mass or pos buffer
POOL = 3 * 4096 * 2 * 128 * 2   # bytes of a pool


@pytest.mark.parametrize("call,change", [
    (COMMIT, dict(seq_out=2 * MB)), (COMMIT, dict(seq_out=2 * MB + 4)), (COMMIT, dict(seq_out=3 * MB + 8)),
    (COMMIT, dict(seq_out=5 * MB)), (COMMIT, dict(row_idx=4 * MB)), (COMMIT, dict(row_vis=4 * MB + 28)),
    (COMMIT, dict(row_vis=7 * MB)), (COMMIT, dict(seq_out=1 * MB + 60)), (COMMIT, dict(vpool=512 * MB)),
    (COMMIT, dict(vpool=512 * MB + POOL - 16)), (COMMIT, dict(seq_out=7 * MB, row_vis=None)),
    (EVICT, dict(n_out=2 * MB)), (EVICT, dict(n_out=2 * MB + 4)), (EVICT, dict(n_out=3 * MB)),
    (EVICT, dict(n_out=4 * MB)), (EVICT, dict(n_out=1 * MB)), (EVICT, dict(mass_out=5 * MB + 16)),
    (EVICT, dict(mass_out=5 * MB + ROWS - 16)), (EVICT, dict(pos_out=6 * MB - ROWS + 16)),
    (EVICT, dict(mass_out=6 * MB)), (EVICT, dict(pos_out=5 * MB)), (EVICT, dict(pos_out=7 * MB)),
    (EVICT, dict(vpool=512 * MB))])
def test_outputs_that_overlap_are_refused(call, change):
    """A launch writes its outputs while other blocks of it still read the inputs: lengths updated in
    place would evict nothing, or move the wrong rows, in some layers."""
    import __graft_entry__
    __graft_entry__.build()
    import query_conditioned_kv_gb300 as kvc
    name = "kvc_tree_commit" if call is COMMIT else "kvc_mass_evict"
    args = dict(call, **change)
    assert list(args) == list(call)
    assert getattr(kvc.lib, name)(*args.values()) == 1
