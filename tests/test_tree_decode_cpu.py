"""Host-side validation of the tree-decoding entry points: every refusal is answered before any
launch (no call here reaches a kernel), and the plain 64-bit forms the GPU tests use hold the
definitions' own identities."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import tree_ref as ref  # noqa: E402

P, U = 1 << 20, (1 << 20) + 2  # an aligned non-NULL address, never dereferenced; a misaligned one
BIG = 1 << 62
INVALID, SHAPE, BUDGET, ALIGN, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import query_conditioned_kv_gb300 as k
    return k


ATTN = dict(q=P, kpool=P, vpool=P, n_slots=1 << 12, block_table=P, max_blocks=8, ctx_len=P, q_off=P,
            tree_mask=P, mask_words=2, n_req=2, n_q=20, max_tree=40, H=2, Hq=8, D=128, block_size=16,
            scale=ctypes.c_float(0.1), out=P, lse=P, ws=P, ws_bytes=BIG, dev_status=None, stream=None)
COMMIT = dict(kpool=P, vpool=P, n_slots=1 << 12, block_table=P, max_blocks=8, ctx_len=P, q_off=P,
              path=P, n_path=P, max_path=4, n_req=2, L=3, H=2, D=128, block_size=16, seq_out=P,
              row_idx=P, row_vis=P, dev_status=None, stream=None)
MASS = dict(q=P, lse=P, n_q=20, row_idx=P, row_vis=P, row_off=P, n_rows=8, max_rows=4, kpool=P,
            n_slots=1 << 12, block_table=P, max_blocks=8, seqused_k=P, n_mass=P, n_req=2, L=3, H=2,
            Hq=8, D=128, block_size=16, scale=ctypes.c_float(0.1), decay=ctypes.c_float(1.0), mass=P,
            ws=P, ws_bytes=BIG, dev_status=None, stream=None)
EVICT = dict(kpool=P, vpool=P, n_slots=1 << 12, block_table=P, max_blocks=8, seqused_k=P, n_pos=P,
             t_end=P, mass=P, pos=P, mass_out=P, pos_out=P, n_out=P, n_req=2, L=3, H=2, D=128,
             block_size=16, budget=64, n_sink=4, n_recent=8, ws=P, ws_bytes=BIG, dev_status=None,
             stream=None)
CALLS = {"kvc_tree_attn": ATTN, "kvc_tree_commit": COMMIT, "kvc_attn_mass": MASS,
         "kvc_mass_evict": EVICT}
F = ctypes.c_float

PAGED = [(dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(block_size=65), SHAPE),
         (dict(block_size=0), INVALID), (dict(H=0), INVALID), (dict(n_req=0), INVALID),
         (dict(max_blocks=0), INVALID), (dict(n_slots=8), INVALID), (dict(n_slots=1 << 31), INVALID),
         (dict(max_blocks=(1 << 20) + 1), SHAPE), (dict(n_req=65536), SHAPE), (dict(kpool=None), INVALID),
         (dict(block_table=None), INVALID), (dict(kpool=U), ALIGN)]
HEADS = [(dict(Hq=7), SHAPE), (dict(Hq=258, H=2), SHAPE), (dict(Hq=1), SHAPE)]
REFUSED = {
    "kvc_tree_attn": PAGED + HEADS + [
        (dict(q=None), INVALID), (dict(vpool=None), INVALID), (dict(ctx_len=None), INVALID),
        (dict(q_off=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID),
        (dict(ws=None), INVALID), (dict(n_q=0), INVALID), (dict(max_tree=0), INVALID),
        (dict(max_tree=1025, mask_words=64), SHAPE), (dict(mask_words=1), SHAPE),
        (dict(scale=F(math.nan)), INVALID), (dict(scale=F(math.inf)), INVALID),
        (dict(q=U), ALIGN), (dict(vpool=U), ALIGN), (dict(out=U), ALIGN), (dict(lse=U), ALIGN),
        (dict(ws=U), ALIGN), (dict(ws_bytes=0), WORKSPACE)],
    "kvc_tree_commit": PAGED + [
        (dict(vpool=None), INVALID), (dict(path=None), INVALID), (dict(n_path=None), INVALID),
        (dict(seq_out=None), INVALID), (dict(max_path=0), INVALID), (dict(max_path=1025), SHAPE),
        (dict(L=0), INVALID), (dict(L=65536), SHAPE), (dict(vpool=U), ALIGN)],
    "kvc_attn_mass": PAGED + HEADS + [
        (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(row_vis=None), INVALID),
        (dict(row_off=None), INVALID), (dict(seqused_k=None), INVALID), (dict(n_mass=None), INVALID),
        (dict(mass=None), INVALID), (dict(n_rows=0), INVALID), (dict(max_rows=0), INVALID),
        (dict(n_q=0), INVALID), (dict(row_idx=None, n_q=7), INVALID), (dict(L=0), INVALID),
        (dict(scale=F(math.nan)), INVALID), (dict(decay=F(1.5)), INVALID), (dict(decay=F(-0.1)), INVALID),
        (dict(decay=F(math.nan)), INVALID), (dict(q=U), ALIGN), (dict(lse=U), ALIGN),
        (dict(mass=U), ALIGN), (dict(ws=U), ALIGN)],
    "kvc_mass_evict": PAGED + [
        (dict(vpool=None), INVALID), (dict(mass=None), INVALID), (dict(pos=None), INVALID),
        (dict(mass_out=None), INVALID), (dict(pos_out=None), INVALID), (dict(n_out=None), INVALID),
        (dict(t_end=None), INVALID), (dict(budget=0), BUDGET), (dict(n_sink=-1), BUDGET),
        (dict(n_recent=-1), BUDGET), (dict(n_sink=60, n_recent=5), BUDGET), (dict(L=0), INVALID),
        (dict(mass=U), ALIGN), (dict(pos_out=U), ALIGN),
        (dict(max_blocks=4096, ws=None, ws_bytes=0), WORKSPACE),
        (dict(max_blocks=4096, ws_bytes=64), WORKSPACE)],
}


@pytest.mark.parametrize("name,change,status",
                         [(n, c, s) for n, cases in REFUSED.items() for c, s in cases],
                         ids=lambda v: None if isinstance(v, int) else str(v))
def test_refused_before_any_launch(kvc, name, change, status):
    args = dict(CALLS[name], **change)
    assert set(args) == set(CALLS[name])
    assert getattr(kvc.lib, name)(*args.values()) == status


def test_workspace_queries(kvc):
    assert kvc.kvc_tree_attn_workspace_size(2, 8, 40, 2, 8, 128, 16) > 0
    for bad in [(0, 8, 40, 2, 8, 128, 16), (2, 8, 1025, 2, 8, 128, 16), (2, 8, 40, 3, 8, 128, 16),
                (2, 8, 40, 2, 8, 80, 16), (2, 8, 40, 2, 8, 128, 65)]:
        assert kvc.kvc_tree_attn_workspace_size(*bad) == 0
    assert kvc.kvc_attn_mass_workspace_size(2, 8, 0, 1, 2, 8, 128, 16) == 0
    assert kvc.kvc_mass_evict_workspace_size(2, 8, 36, 8, 16, 64) == 0        # staged on chip
    assert kvc.kvc_mass_evict_workspace_size(2, 4096, 36, 8, 16, 64) > 0      # 65,536 rows
    with open(kvc._HERE + "/../include/kvc.h") as f:
        head = f.read()
    assert f"#define KVC_EVICT_STAGED_ROWS {kvc.EVICT_STAGED_ROWS}\n" in head
    assert f"#define KVC_TREE_MAX_NODES {kvc.TREE_MAX_NODES}\n" in head


def test_binding_refuses_strided_and_host_tensors(kvc):
    t = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="contiguous"):
        kvc.kvc_mass_evict(t.t(), t, 4, t, 1, t, t, t, t, t, t, t, t, 1, 1, 1, 64, 16, 4, 0, 0)
    with pytest.raises(ValueError, match="device"):
        kvc.kvc_tree_commit(t, t, 4, t, 1, t, t, t, t, 1, 1, 1, 1, 64, 16, t)


def test_reference_attention_identities():
    """A chain's last row attends like plain softmax attention; weights of all rows of a request
    add up to one per row and head."""
    g = torch.Generator().manual_seed(1)
    H, G, D, BS, c, T = 2, 3, 64, 8, 19, 4
    bt = np.array([[3, 0, 2]])
    kp, vp = torch.randn(32, H, D, generator=g), torch.randn(32, H, D, generator=g)
    q = torch.randn(T, H * G, D, generator=g)
    out, lse, _, _ = ref.attn(q, kp, vp, bt, BS, [c], [0, T], None, H, 0.125)
    s = ref.slots(bt[0], BS, c + T)
    for hq in range(H * G):
        z = kp[s, hq // G].double() @ q[-1, hq].double() * 0.125
        assert torch.allclose(out[-1, hq], torch.softmax(z, 0) @ vp[s, hq // G].double())
    old = torch.zeros(1, 1, H, 24)
    m, _ = ref.mass(q[None], lse[None], None, c + 1 + np.arange(T), [0, T], kp[None], bt, BS, [c + T],
                    [0], old, H, 0.125, 1.0)
    assert torch.allclose(m.sum(-1), torch.full((1, 1, H), float(T * G), dtype=torch.float64))
    full = ref.tree_masks(np.random.default_rng(0), 5, 1, "full")
    assert np.array_equal(full[:, 0], np.full(5, 31, np.uint32))
    assert np.all(ref.tree_masks(np.random.default_rng(0), 5, 1, "empty") == 0)


def test_reference_eviction_keeps_the_heaviest():
    rng = np.random.default_rng(3)
    n, B, H, BS = 21, 9, 2, 8
    bt = np.array([[1, 0, 2]])
    w = rng.random((1, 1, H, 24)).astype(np.float32)
    k = rng.integers(0, 1000, (1, 24, H, 4))
    pos = np.zeros((1, 1, H, 24), np.int32)
    ko, vo, mo, po, m = ref.evict(k, k, bt, BS, [n], [0], [n], w, pos, H, B, 2, 3)
    assert m[0] == B
    for h in range(H):
        free = np.sort(w[0, 0, h, 2:n - 3])[::-1][:B - 5]
        want = np.concatenate([w[0, 0, h, :2], w[0, 0, h, n - 3:n], free])
        assert np.array_equal(np.sort(mo[0, 0, h, :B]), np.sort(want))
        s = ref.slots(bt[0], BS, n).numpy()
        for i in range(B):  # every kept row carries its own K row, weight and position
            assert np.array_equal(ko[0, s[i], h], k[0, s[po[0, 0, h, i]], h])
            assert mo[0, 0, h, i] == w[0, 0, h, po[0, 0, h, i]]
