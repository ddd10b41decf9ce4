"""Tree decoding on the GPU at the limits of its types, against 64-bit forms: logits far past the range
in which fp32 resolves single units."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import tree_ref as ref  # noqa: E402
from test_gpu_tree_decode import Evict, Mass, Tree, check_evict, i32, inside, kvc  # noqa: E402,F401

DEV = "cuda"
NAN = float("nan")


def evenly(t):
    """Attention with the maximum taken off the logits first (an lse of 2^66 does not hold ln n in 64
    bits)."""
    o = torch.zeros(t.n_q, t.Hq, t.D, dtype=torch.float64)
    for r in range(t.n_req):
        s = ref.slots(t.bt[r], t.BS, t.ctx[r] + t.T[r])
        for i in range(t.T[r]):
            row = int(t.q_off[r]) + i
            nodes = ref.sees(None if t.mask is None else t.mask[row], i, t.T[r], t.mask is None)
            at = s[torch.from_numpy(np.flatnonzero(np.concatenate([np.ones(t.ctx[r], bool), nodes])))]
            for h in range(t.Hq):
                z = t.k[at, h // t.G].double() @ t.q[row, h].double() * t.scale
                o[row, h] = torch.softmax(z, 0) @ t.v[at, h // t.G].double()
    return o


@pytest.mark.parametrize("T,G,D", [(3, 4, 128), (12, 4, 64), (20, 5, 128), (64, 4, 128), (50, 4, 64)])
@pytest.mark.parametrize("exponent", [20, 27, 33, 40, 66, 99])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "equal"])
def test_attn_huge_logits(kvc, T, G, D, exponent, order):  # noqa: F811
    """Logits of ±2^20 to ±2^99, exact in fp32, whose distinct levels lie 2^-7 of them apart: the rows
    attend to their highest level's keys alone, evenly.  Few rows and many, several tiles and CTAs."""
    for sign in (1.0, -1.0):
        t = Tree(exponent + T, [1100, 70], [T, T - 1], 1, G, D, 16, "tree")
        t.scale = 1.0
        t.q.zero_()
        t.q[..., 0] = 1.0
        rng = np.random.default_rng(exponent)
        for r in range(2):
            n = t.ctx[r] + t.T[r]
            j = {"rising": np.arange(n) * 100 // n, "falling": 100 - np.arange(n) * 100 // n,
                 "mixed": rng.integers(0, 100, n), "equal": np.full(n, 77)}[order]
            level = torch.from_numpy(sign * 2.0 ** exponent * (1 + j / 128.0)).to(torch.bfloat16)
            t.k[ref.slots(t.bt[r], 16, n), 0, 0] = level
        out, lse = t.gpu().call(kvc)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(t.d["status"]) == 0
        _, ls, _, _ = t.want()
        o = evenly(t)
        # weights of 1 and 0 (of 2^r, |r| < 1, in bf16 where references are below 2^24), n keys summed
        # in fp32, one rounding of out; the lse: scale·log2e, the product, the sum, ·ln2
        wv = torch.where(torch.isfinite(t.v), t.v.double().abs(), torch.zeros_like(t.v.double())).max()
        ob = 2 * ref.UBF * o.abs() + (ref.UBF + 1200 * ref.U32 + 2 ** -21) * wv
        inside(out, o, ob, f"out {sign}")
        inside(lse, ls, 8 * ref.U32 * ls.abs() + 1200 * ref.U32 + 2 ** -20, f"lse {sign}")


# ------------------------------------------------------- NaN among the logits

@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (3, 4, 64), (12, 4, 128), (20, 4, 128), (64, 4, 64)])
@pytest.mark.parametrize("ctx", [[700, 3, 40], [0, 9, 16], [6000, 5000, 30], [40000, 64, 9]])
def test_attn_nan_logits(kvc, T, G, D, ctx):  # noqa: F811
    """A NaN in a query, a whole page of NaN keys, the only keys of a request NaN, a NaN node: NaN in
    exactly the rows that see it, whichever path takes them (a row that sees nothing has 0 and -inf)."""
    if max(ctx) > 10000 and T > 3:
        pytest.skip("long caches with short trees only")
    t = Tree(sum(ctx) + T, ctx, [T] * 3, 2, G, D, 16, "tree", poison=False)
    t.q[1 % (3 * T), 1, 5] = NAN                       # one head of one row
    t.q[T + T // 2, 2] = NAN
    s2 = ref.slots(t.bt[2], 16, ctx[2] + T)
    t.k[s2[:min(16, ctx[2])], 0] = NAN                 # a page (or less) of the last request, one KV head
    s0 = ref.slots(t.bt[0], 16, ctx[0] + T)
    t.k[s0[ctx[0] + T - 1], 1, 7] = NAN                # the last node of the first, the other KV head
    out, lse = t.gpu().call(kvc)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(t.d["status"]) == 0
    o, ls, ob, lb = t.want()
    assert torch.isnan(ls).any() and not torch.isnan(ls).all()
    inside(out, o, ob, "out")
    inside(lse, ls, lb, "lse")


def test_attn_nan_next_to_rows_that_see_nothing(kvc):  # noqa: F811
    """Nothing cached and masks of holes: 0 and -inf where a row sees nothing, NaN where its only node
    is NaN."""
    for T, G in [(4, 4), (40, 4)]:
        t = Tree(3, [0, 0], [T, T], 1, G, 128, 16, "self", poison=False)
        t.mask[1] = 0
        t.k[ref.slots(t.bt[0], 16, T)[2]] = NAN
        out, lse = t.gpu().call(kvc)
        o, ls, ob, lb = t.want()
        assert torch.isinf(ls[1]).all() and torch.isnan(ls[2]).all()
        inside(out, o, ob, "out")
        inside(lse, ls, lb, "lse")


@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (8, 4), (20, 4), (64, 4)])
@pytest.mark.parametrize("value", [NAN, float("inf")])
@pytest.mark.parametrize("place", ["cached", "node"])
def test_attn_values_that_are_not_finite_reach_far_rows(kvc, T, G, value, place):  # noqa: F811
    """A NaN or infinite V whose weight is below the smallest fp32 is still a value the row sees: its
    result is not finite."""
    t = Tree(5, [900], [T], 1, G, 128, 16, "chain", poison=False)
    s = ref.slots(t.bt[0], 16, 900 + T)
    t.q.zero_()
    t.q[..., 0] = 1.0
    t.k[s, 0, 0] = 0.0
    at = 100 if place == "cached" else 900
    t.k[s[at], 0, 0] = -300.0 / t.scale
    t.v[s[at], 0, 9] = value
    out, lse = t.gpu().call(kvc)
    o, ls, ob, lb = t.want()
    out = out.float().cpu()
    assert not torch.isfinite(out[:, :, 9]).any()
    keep = torch.arange(128) != 9
    inside(out[..., keep], o[..., keep], ob[..., keep], "out")
    inside(lse, ls, lb, "lse")


@pytest.mark.parametrize("tile", [0, 1])
def test_attn_values_that_are_not_finite_in_a_tile_of_no_weight(kvc, tile):  # noqa: F811
    """The same where all of a tile's weights are below the smallest fp32: whole units of two tiles, so
    that one of a block's two groups of warps holds nothing else."""
    T, G, n = 10, 4, 100
    t = Tree(6, [246] * n, [T] * n, 2, G, 128, 16, "chain", poison=False)
    t.q.zero_()
    t.q[..., 0] = 1.0
    t.k[:, :, 0] = 0.0
    for r in range(n):
        s = ref.slots(t.bt[r], 16, 256)
        t.k[s[128 * tile:128 * tile + 128], :, 0] = -300.0 / t.scale
        t.v[s[128 * tile + 7], r % 2, 11] = NAN
    out, lse = t.gpu().call(kvc)
    o, ls, ob, lb = t.want()
    inside(out, o, ob, "out")
    inside(lse, ls, lb, "lse")


# --------------------------------------------- infinite keys under the weights

@pytest.mark.parametrize("m,G,kind", [(3, 4, "path"), (1, 1, "path"), (7, 3, "path"), (9, 4, "path"),
                                      (20, 8, "path"), (48, 4, "window"), (33, 1, "window"),
                                      (100, 3, "window"), (130, 4, "path")])
def test_mass_infinite_keys(kvc, m, G, kind):  # noqa: F811
    """A key with an infinite component that every row's query meets with the same sign: weight 0 where
    that makes all logits -inf, infinite where +inf, and nothing else is touched."""
    for sign in (-1.0, 1.0):
        t = Mass(m + G, [300, 290], [m, m], 2, 2, G, 128, 16, kind, decay=0.5)
        t.q[..., 0] = sign
        want, bound = t.want()
        cached = [5, 100, 150, 0]                     # (all rows of windows up to 130 see these)
        for r in range(2):
            s = ref.slots(t.bt[r], 16, t.seq[r])
            t.k[:, s[cached], :, 0] = float("inf")
            old = t.old[:, r, :, cached].double() * t.decay
            want[:, r, :, cached] = old if sign < 0 else float("inf")
            bound[:, r, :, cached] = 2 * ref.U32
        got = t.gpu().call(kvc)
        torch.cuda.synchronize()
        inside(got, want, bound, f"mass {sign}")


# --------------------------------------------------------- streams by handle

@pytest.mark.parametrize("raw", [True, False])
def test_event_takes_a_stream_or_its_handle(kvc, raw):  # noqa: F811
    from test_gpu_tree_event import Serving
    a, b = Serving(5, [50, 7], 9, observe=4), Serving(5, [50, 7], 9, observe=4)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else 0           # (0: the default stream)
    q = torch.randn(2, 8, a.Hq, a.D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    lse = torch.full((2, 8, a.Hq), 5.0, device=DEV)
    vis, off = i32([47, 48, 49, 50, 4, 5, 6, 7]), i32([0, 4, 8])
    torch.cuda.synchronize()
    for sv, stream in ((a, None), (b, handle)):
        sv.ev.observe(q, lse, vis, off, sv.kd, sv.btd, stream)
        for _ in range(2):
            s = sv.draw()
            torch.cuda.synchronize()
            sv.write_nodes(s)
            torch.cuda.synchronize()
            sv.step({"q": s["q"].to(DEV), "mask_d": i32(s["mask"].view(np.int32)), "path_d": i32(s["path"]),
                     "m_d": i32(s["m"])}, stream)
            torch.cuda.synchronize()
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


# --------------------------------------------------------------- host threads

def test_calls_of_several_sizes_from_several_threads(kvc):  # noqa: F811
    """Two host threads evict from tables of different lengths at once: the shared-memory limit that one
    sets never refuses the other's launch."""
    import threading
    errors, results = [], {}

    def work(name, n, budget):
        try:
            e = Evict(n, [n], budget, 1, 1, 64, 16)
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                kd, vd = (torch.from_numpy(x).to(DEV).view(torch.bfloat16) for x in (e.k, e.v))
                m, p = torch.from_numpy(e.mass).to(DEV), torch.from_numpy(e.pos).to(DEV)
                mo, po, no = torch.empty_like(m), torch.empty_like(p), i32([0])
                bt, seq, n_pos, t_end = i32(e.bt), i32(e.seq), i32(e.n_pos), i32(e.t_end)
                status = i32([0])
                st.synchronize()
                for _ in range(3000):
                    kvc.kvc_mass_evict(kd, vd, e.n_slots, bt, e.max_blocks, seq, n_pos, t_end, m, p, mo, po,
                                       no, 1, 1, 1, 64, 16, budget, e.n_sink, e.n_recent, None, status, st)
                st.synchronize()
                results[name] = int(no)
        except Exception as x:  # noqa: BLE001
            errors.append(f"{name}: {x}")

    threads = [threading.Thread(target=work, args=a) for a in
               [("long", 15000, 4000), ("short", 200, 100), ("other", 900, 100)]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert results == {"long": 4000, "short": 100, "other": 100}


# ------------------------------------------------------ forms few calls reach

@pytest.mark.parametrize("rows,G,max_blocks", [(640, 8, 1 << 18), (2100, 2, 300000)])
def test_mass_of_more_rows_than_one_pass_holds(kvc, rows, G, max_blocks):  # noqa: F811
    """Partial sums past their 512 MB (a long table): the rows' tiles take several passes that add to
    one another, the first on top of the decayed weight."""
    t = Mass(rows, [rows, rows // 3], [rows, rows // 3], 1, 1, G, 64, 32, "window", decay=0.75)
    old_cap, old = t.cap, t.old
    t.max_blocks = max_blocks
    t.cap = max_blocks * 32
    bt = np.full((2, max_blocks), -1)
    bt[:, :t.bt.shape[1]] = t.bt
    t.bt = bt
    t.old = torch.zeros(1, 2, 1, t.cap)
    t.old[..., :old_cap] = old
    per = 1 * 2 * 1 * 2 * t.cap * 4
    pairs = -(-rows // (2 * (256 // G)))
    assert pairs > max(8, (1 << 29) // per)
    n = kvc.kvc_attn_mass_workspace_size(2, max_blocks, rows, 1, 1, G, 64, 32)
    assert per * 8 <= n < per * pairs
    got = t.gpu().call(kvc)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(t.d["status"]) == 0
    t.old = old
    want, bound = t.want()
    inside(got[..., :old_cap], want, bound, "mass")
    assert not got[..., old_cap:].any()


@pytest.mark.parametrize("weights,sink,recent,carried", [("equal", 2, 3, 0.5), ("random", 2, 3, 1.0),
                                                         ("mixed", 0, 64, 0.0), ("mixed", 64, 0, 1.0),
                                                         ("nan", 2, 3, 0.5), ("mixed", 10, 54, 0.7)])
def test_evict_past_the_staged_length(kvc, weights, sink, recent, carried):  # noqa: F811
    """Tables past the length whose keys fit the chip, requests of many rows, few, and under the budget;
    in place and into other buffers."""
    for in_place in (True, False):
        e = Evict(sink + recent, [50000, 3000, 900, 0], 1000, 1, 1, 64, 16, sink, recent, carried, weights)
        assert e.cap > kvc.EVICT_STAGED_ROWS
        check_evict(kvc, e, in_place, status=8 if weights == "nan" else 0)


@pytest.mark.parametrize("H,G,D,BS", [(8, 4, 128, 16), (2, 3, 64, 8)])
def test_the_lse_is_what_the_recovery_score_takes(kvc, H, G, D, BS):  # noqa: F811
    """Plain decoding's LSE against a 64-bit one, through kvc_recover_score."""
    ctx, L = [70, 3, 500], 2
    seq = np.array(ctx) + 1
    trees = [Tree(7 + layer, ctx, [1, 1, 1], H, G, D, BS, "chain", poison=False) for layer in range(L)]
    for t in trees[1:]:
        t.bt = trees[0].bt
    lses, wants, bounds = [], [], []
    for t in trees:
        lses.append(t.gpu().call(kvc)[1])
        _, ls, _, lb = t.want()
        wants.append(ls.float().to(DEV))
        bounds.append(lb)
    t0 = trees[0]
    k = torch.stack([t.k for t in trees]).to(DEV)
    q = torch.stack([t.q for t in trees], 1).contiguous().to(DEV)        # [n_req][L][Hq][D]
    state = []
    for lse in (lses, wants):
        st = torch.zeros(3, t0.max_blocks * BS, device=DEV)
        status = i32([0])
        kvc.kvc_recover_score(q, torch.stack(lse, 1).contiguous(), k, t0.n_slots, i32(t0.bt), t0.max_blocks,
                              i32(seq), i32([1, 1, 1]), 3, L, H, H * G, D, BS, st, None, status)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(status) == 0
        state.append(st.double().cpu())
    # the same kernel on both: each weight moves by its lse's error and by the exponent's rounding
    tol = float(torch.stack(bounds).max()) + 64 * ref.U32 + 2 ** -20
    for r in range(3):
        a, b = state[0][r, :seq[r]], state[1][r, :seq[r]]
        assert float(b.max()) > 0 and float(((a - b).abs() / b.clamp(min=1e-30)).max()) <= tol
