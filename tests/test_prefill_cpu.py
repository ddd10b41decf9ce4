"""Host-side validation of the entry points that fill the paged cache and read its 8-bit part: every
refusal is answered before any launch (no call here reaches a kernel), and the plain 64-bit forms the
GPU tests use hold the definitions' own identities."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import prefill_ref as ref  # noqa: E402
import tree_ref  # noqa: E402

M = 1 << 32  # far-apart aligned non-NULL addresses, never dereferenced
BIG = 1 << 62
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 4, 5
F = ctypes.c_float


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    import query_conditioned_kv_gb300 as k
    return k


ROPE = dict(q=1 * M, q_stride=1536, k=2 * M, k_stride=1536, v=3 * M, v_stride=1536, n_tok=20, wq=4 * M,
            wk=5 * M, eps=F(1e-6), rope_tab=6 * M, n_pos=100, pos=7 * M, q_off=8 * M, ctx_len=9 * M,
            n_req=2, block_table=10 * M, max_blocks=8, kpool=11 * M, vpool=12 * M, n_slots=1 << 12, H=2,
            Hq=8, D=128, block_size=16, q_out=13 * M, k_raw=14 * M, raw_stride=20 * 128, dev_status=None,
            stream=None)
PROMPT = dict(q=1 * M, kpool=2 * M, vpool=3 * M, n_slots=1 << 12, block_table=4 * M, max_blocks=8,
              ctx_len=5 * M, q_off=6 * M, n_req=2, n_q=20, max_rows=20, H=2, Hq=8, D=128, block_size=16,
              scale=F(0.1), out=7 * M, lse=8 * M, dev_status=None, stream=None)
PACK = dict(kpool=1 * M, vpool=2 * M, n_slots=1 << 12, k8=3 * M, v8=4 * M, kscale=5 * M, vscale=6 * M,
            n_blocks8=9, src_block=7 * M, dst_block=8 * M, n=5, L=3, H=2, D=128, block_size=16,
            dev_status=None, stream=None)
ATTN = dict(q=1 * M, k8=2 * M, v8=3 * M, kscale=4 * M, vscale=5 * M, n_blocks8=9, table8=6 * M,
            max_blocks8=4, len8=7 * M, kpool=8 * M, vpool=9 * M, n_slots=1 << 12, block_table=10 * M,
            max_blocks=8, ctx_len=11 * M, q_off=12 * M, tree_mask=13 * M, mask_words=2, n_req=2, n_q=20,
            max_tree=40, H=2, Hq=8, D=128, block_size=16, scale=F(0.1), out=14 * M, lse=15 * M,
            ws=16 * M, ws_bytes=BIG, dev_status=None, stream=None)
CALLS = {"kvc_qkv_rope": ROPE, "kvc_prompt_attn": PROMPT, "kvc_q8_pack": PACK, "kvc_q8_attn": ATTN}

PAGED = [(dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(block_size=65), SHAPE),
         (dict(block_size=0), INVALID), (dict(H=0), INVALID), (dict(n_slots=8), INVALID),
         (dict(n_slots=1 << 31), INVALID), (dict(kpool=None), INVALID), (dict(vpool=None), INVALID),
         (dict(kpool=1 * M + 2), ALIGN), (dict(vpool=2 * M + 8), ALIGN)]
TABLE = [(dict(n_req=0), INVALID), (dict(max_blocks=0), INVALID), (dict(max_blocks=(1 << 20) + 1), SHAPE),
         (dict(n_req=65536), SHAPE), (dict(block_table=None), INVALID), (dict(q_off=None), INVALID),
         (dict(ctx_len=None), INVALID), (dict(q=None), INVALID), (dict(q=1 * M + 4), ALIGN)]
HEADS = [(dict(Hq=7), SHAPE), (dict(Hq=258, H=2), SHAPE), (dict(Hq=1), SHAPE),
         (dict(H=257, Hq=257), SHAPE)]
ATTENTION = [(dict(n_q=0), INVALID), (dict(scale=F(math.nan)), INVALID), (dict(scale=F(math.inf)), INVALID),
             (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(out=7 * M + 8), ALIGN),
             (dict(lse=8 * M + 2), ALIGN)]
REFUSED = {
    "kvc_qkv_rope": PAGED + TABLE + HEADS + [
        (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(rope_tab=None), INVALID),
        (dict(q_out=None), INVALID), (dict(n_tok=0), INVALID), (dict(n_pos=0), INVALID),
        (dict(eps=F(-1e-6)), INVALID), (dict(eps=F(math.nan)), INVALID), (dict(eps=F(math.inf)), INVALID),
        (dict(q_stride=1016), SHAPE), (dict(k_stride=248), SHAPE), (dict(v_stride=1537), SHAPE),
        (dict(q_stride=1 << 62), SHAPE), (dict(raw_stride=19 * 128), SHAPE), (dict(raw_stride=2564), SHAPE),
        (dict(k=2 * M + 2), ALIGN), (dict(v=3 * M + 2), ALIGN), (dict(wq=4 * M + 2), ALIGN),
        (dict(wk=5 * M + 2), ALIGN), (dict(rope_tab=6 * M + 4), ALIGN), (dict(q_out=13 * M + 2), ALIGN),
        (dict(k_raw=14 * M + 2), ALIGN),
        # outputs over inputs or over each other
        (dict(q_out=1 * M), INVALID), (dict(q_out=2 * M + 512), INVALID), (dict(kpool=3 * M), INVALID),
        (dict(vpool=11 * M + 1024), INVALID), (dict(k_raw=13 * M + 64), INVALID), (dict(k_raw=6 * M), INVALID)],
    "kvc_prompt_attn": PAGED + TABLE + HEADS + ATTENTION + [
        (dict(max_rows=0), INVALID), (dict(max_rows=(1 << 24) + 1), SHAPE),
        (dict(out=1 * M), INVALID), (dict(out=3 * M - 16), INVALID), (dict(lse=7 * M + 4), INVALID),
        (dict(lse=4 * M + 60), INVALID)],
    "kvc_q8_pack": PAGED + [
        (dict(H=257), SHAPE),        (dict(k8=None), INVALID), (dict(v8=None), INVALID), (dict(kscale=None), INVALID),
        (dict(vscale=None), INVALID), (dict(src_block=None), INVALID), (dict(dst_block=None), INVALID),
        (dict(n=0), INVALID), (dict(n_blocks8=0), INVALID), (dict(n_blocks8=1 << 31), SHAPE),
        (dict(n=(1 << 31) - 1), SHAPE), (dict(L=0), INVALID), (dict(L=65536), SHAPE),
        (dict(k8=3 * M + 8), ALIGN), (dict(v8=4 * M + 1), ALIGN), (dict(kscale=5 * M + 2), ALIGN),
        (dict(vscale=6 * M + 1), ALIGN), (dict(k8=1 * M), INVALID), (dict(v8=3 * M + 64), INVALID),
        (dict(kscale=6 * M + 4), INVALID), (dict(vscale=8 * M), INVALID)],
    "kvc_q8_attn": PAGED + TABLE + HEADS + ATTENTION + [
        (dict(k8=None), INVALID), (dict(v8=None), INVALID), (dict(kscale=None), INVALID),
        (dict(vscale=None), INVALID), (dict(table8=None), INVALID), (dict(len8=None), INVALID),
        (dict(max_blocks8=0), INVALID), (dict(max_blocks8=(1 << 20) + 1), SHAPE), (dict(n_blocks8=0), INVALID),
        (dict(n_blocks8=1 << 31), SHAPE), (dict(max_tree=0), INVALID),
        (dict(max_tree=1025, mask_words=64), SHAPE), (dict(mask_words=1), SHAPE), (dict(ws=None), INVALID),
        (dict(ws=16 * M + 8), ALIGN), (dict(ws_bytes=64), WORKSPACE), (dict(k8=2 * M + 4), ALIGN),
        (dict(v8=3 * M + 8), ALIGN), (dict(kscale=4 * M + 2), ALIGN), (dict(vscale=5 * M + 3), ALIGN),
        (dict(out=1 * M + 256), INVALID), (dict(out=3 * M + 64), INVALID), (dict(lse=5 * M + 8), INVALID),
        (dict(ws=14 * M + 64), INVALID), (dict(lse=16 * M + 32), INVALID), (dict(out=13 * M), INVALID)],
}


@pytest.mark.parametrize("name,change,status",
                         [(n, c, s) for n, cases in REFUSED.items() for c, s in cases],
                         ids=lambda v: None if isinstance(v, int) else str(v))
def test_refused_before_any_launch(kvc, name, change, status):
    args = dict(CALLS[name], **change)
    assert set(args) == set(CALLS[name])
    assert getattr(kvc.lib, name)(*args.values()) == status


@pytest.mark.parametrize("name", ["kvc_prompt_attn", "kvc_q8_attn"])
@pytest.mark.parametrize("scale", [3e38, -2.5e38])
def test_scales_that_pass_fp32_in_log2_are_refused(kvc, name, scale):
    args = dict(CALLS[name], scale=F(scale))
    assert getattr(kvc.lib, name)(*args.values()) == INVALID


def test_workspace_query(kvc):
    assert kvc.kvc_q8_attn_workspace_size(2, 4, 8, 40, 2, 8, 128, 16) > 0
    for bad in [(0, 4, 8, 40, 2, 8, 128, 16), (2, 0, 8, 40, 2, 8, 128, 16), (2, 4, 0, 40, 2, 8, 128, 16),
                (2, 4, 8, 1025, 2, 8, 128, 16), (2, 4, 8, 0, 2, 8, 128, 16), (2, 4, 8, 40, 3, 8, 128, 16),
                (2, 4, 8, 40, 2, 8, 80, 16), (2, 4, 8, 40, 2, 8, 128, 65)]:
        assert kvc.kvc_q8_attn_workspace_size(*bad) == 0


def test_workspace_of_fewer_rows_is_no_larger(kvc):
    """A buffer made for a call of many rows serves calls of fewer (what a step's sizes rely on)."""
    for n_req, mb8, mb, H, G, D in [(1, 8, 4, 1, 1, 64), (3, 200, 20, 2, 4, 128), (64, 512, 64, 8, 4, 128),
                                    (2, 1, 1, 4, 33, 64), (500, 3, 2, 1, 256, 128), (1, 8192, 9, 8, 6, 128)]:
        sizes = [kvc.kvc_q8_attn_workspace_size(n_req, mb8, mb, t, H, H * G, D, 16) for t in range(1, 1025)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_binding_refuses_wrong_rows(kvc):
    """Rows of a fused projection may be strided; columns may not, and host tensors are refused."""
    t = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="device"):
        kvc.kvc_qkv_rope(t, t, t, 4, None, None, 1e-6, t, 4, None, t, t, 1, t, 1, t, t, 16, 2, 2, 128, 16, t)
    with pytest.raises(ValueError, match="device"):
        kvc.kvc_prompt_attn(t, t, t, 16, t, 1, t, t, 1, 4, 4, 2, 2, 128, 16, 0.1, t, t)
    with pytest.raises(ValueError, match="contiguous"):
        kvc.kvc_q8_pack(t.t(), t, 16, t, t, t, t, 1, t, t, 1, 1, 2, 64, 16)


@pytest.mark.parametrize("change", [dict(recent=-1), dict(max_move=0), dict(max_move=-3)])
def test_history_event_refuses(kvc, change):
    from query_conditioned_kv_gb300.event import HistoryEvent
    with pytest.raises(ValueError, match="HistoryEvent"):
        HistoryEvent(1, 4, 4, 16, 1, 1, 1, 64, 64, 4, 4, 4, 8, **change)


def test_reference_rotation_keeps_lengths_and_offsets():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 3, 64, generator=g, dtype=torch.float64)
    tab = ref.rope_table(50, 64)
    at7, _ = ref.rotated(x, 0.0, tab[[7, 7]])
    at9, _ = ref.rotated(x, 0.0, tab[[9, 9]])
    at40, _ = ref.rotated(x, 0.0, tab[[40, 40]])
    at42, _ = ref.rotated(x, 0.0, tab[[42, 42]])
    assert torch.allclose(at7.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
    assert torch.allclose((at7 * at9.flip(0)).sum(-1), (at40 * at42.flip(0)).sum(-1), atol=1e-4)
    y, _ = ref.normed(x, torch.ones(64), 0.0)
    assert torch.allclose(y.pow(2).mean(-1), torch.ones(2, 3, dtype=torch.float64))


def test_reference_prompt_is_the_chain():
    g = torch.Generator().manual_seed(5)
    H, G, D, BS = 2, 3, 64, 8
    bt = np.array([[3, 0, 2], [1, 4, 5]])
    k, v = torch.randn(48, H, D, generator=g), torch.randn(48, H, D, generator=g)
    q = torch.randn(11, H * G, D, generator=g)
    a = ref.prompt(q, k, v, bt, BS, [13, 0], [0, 4, 11], H, 0.2)
    b = tree_ref.attn(q, k, v, bt, BS, [13, 0], [0, 4, 11], None, H, 0.2)
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-9, atol=1e-12)


def test_reference_e4m3():
    """Every e4m3 value is its own; midpoints go to the even one; the largest value is the scale's."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fine = codes[np.isfinite(codes)]
    assert np.array_equal(ref.e4m3(fine), fine)
    pos = np.unique(fine[fine >= 0])
    mid = (pos[:-1] + pos[1:]) / 2
    got = ref.e4m3(mid)
    even = np.where(np.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])
    assert np.array_equal(got, even)
    x = torch.tensor([448.0, 1.0, 449.0, 0.0]).view(1, 4, 1, 1).expand(1, 4, 1, 64).clone().bfloat16()
    x[0, 0, 0, 0] = 450.0  # rounds to bf16 450
    y, s = ref.pack(x, [0, 1, 3], 1)
    assert s[:, 0, 0].tolist() == [2.0, 2.0 ** -8, 1.0] and y[1, 0, 0, 0, 0] == 256.0


def test_reference_q8_without_history_is_tree_attention():
    g = torch.Generator().manual_seed(7)
    H, G, D, BS = 2, 2, 64, 8
    bt, t8 = np.array([[3, 0, 2]]), np.array([[1, 0]])
    k, v = torch.randn(32, H, D, generator=g), torch.randn(32, H, D, generator=g)
    q = torch.randn(4, H * G, D, generator=g)
    k8, v8 = torch.randn(2, H, BS, D, generator=g), torch.randn(2, H, BS, D, generator=g)
    one = torch.ones(2, H)
    a = ref.q8(q, k8, v8, one, one, t8, [0], k, v, bt, BS, [13], [0, 4], None, H, 0.2)
    b = tree_ref.attn(q, k, v, bt, BS, [13], [0, 4], None, H, 0.2)
    assert torch.allclose(a[0], b[0]) and torch.allclose(a[1], b[1])
    # a history of the same rows in bf16 gives the same as one cache
    hist = torch.stack([k8[b_, :, p] for b_ in (1, 0) for p in range(BS)][:11])
    vals = torch.stack([v8[b_, :, p] for b_ in (1, 0) for p in range(BS)][:11])
    s = tree_ref.slots(bt[0], BS, 17)
    kk, vv = torch.cat([hist, k[s]]), torch.cat([vals, v[s]])
    a = ref.q8(q, k8, v8, one, one, t8, [11], k, v, bt, BS, [13], [0, 4], None, H, 0.2)
    b = tree_ref.attn(q, kk, vv, np.arange(28)[None], 1, [24], [0, 4], None, H, 0.2)
    assert torch.allclose(a[0], b[0]) and torch.allclose(a[1], b[1])
