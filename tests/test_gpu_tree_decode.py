"""Tree decoding on the GPU against 64-bit forms (tests/tree_ref.py): attention of drafted trees over
a paged cache, accumulated attention weight, the commit of an accepted path and eviction by weight,
at the sizes, masks and values where each can go wrong.  Tolerances are counted in half steps of the
types (tree_ref); integers, copies and orders are exact."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import tree_ref as ref  # noqa: E402

DEV = "cuda"
NAN = float("nan")


@pytest.fixture(scope="module")
def kvc():
    import query_conditioned_kv_gb300 as k
    return k


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(torch.bfloat16)


def table(rng, n_req, max_blocks, spare=2):
    n_blocks = n_req * max_blocks + spare
    return rng.permutation(n_blocks)[:n_req * max_blocks].reshape(n_req, max_blocks), n_blocks


def inside(got, want, bound, what):
    got, want = got.double().cpu(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    over = (got - want).abs()[fin] / bound[fin].clamp(min=1e-300)
    assert over.numel() == 0 or float(over.max()) <= 1.0, \
        f"{what}: {float(over.max()):.3g} times the bound, {int((over > 1).sum())} values"


class Tree:
    """A batch of requests with trees over a paged pool, on the host."""

    def __init__(self, seed, ctx, T, H, G, D, BS, kind="tree", kscale=1.0, poison=True, pad_words=0):
        rng = np.random.default_rng(seed)
        self.ctx, self.T, self.H, self.G, self.D, self.BS = list(ctx), list(T), H, G, D, BS
        self.n_req, self.Hq = len(ctx), H * G
        self.max_tree = max(max(T), 1)
        self.max_blocks = max(1, max(-(-(c + t) // BS) for c, t in zip(ctx, T)))
        self.bt, n_blocks = table(rng, self.n_req, self.max_blocks)
        self.n_slots = n_blocks * BS
        self.q_off = np.concatenate([[0], np.cumsum(T)])
        self.n_q = max(1, int(self.q_off[-1]))
        self.words = (self.max_tree + 31) // 32 + pad_words
        self.mask = None if kind == "chain" else np.concatenate(
            [ref.tree_masks(rng, t, self.words, kind) for t in T] + [np.zeros((0, self.words), np.uint32)])
        if self.mask is not None and len(self.mask) == 0:
            self.mask = np.zeros((1, self.words), np.uint32)
        self.q = rows(seed + 1, self.n_q, self.Hq, D, scale=kscale)
        self.k, self.v = rows(seed + 2, self.n_slots, H, D), rows(seed + 3, self.n_slots, H, D)
        self.scale = 1.0 / math.sqrt(D)
        if poison:  # everything no row sees holds NaN: other slots, and nodes outside every mask
            seen = np.zeros(self.n_slots, bool)
            for r in range(self.n_req):
                s = ref.slots(self.bt[r], BS, self.ctx[r] + self.T[r]).numpy()
                seen[s[:self.ctx[r]]] = True
                for i in range(self.T[r]):
                    m = ref.sees(None if self.mask is None else self.mask[self.q_off[r] + i], i,
                                 self.T[r], self.mask is None)
                    seen[s[self.ctx[r]:][m]] = True
            self.k[~seen], self.v[~seen] = NAN, NAN

    def gpu(self):
        self.d = dict(q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV), bt=i32(self.bt),
                      ctx=i32(self.ctx), q_off=i32(self.q_off),
                      mask=None if self.mask is None else i32(self.mask.view(np.int32)),
                      out=torch.full((self.n_q, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV),
                      lse=torch.full((self.n_q, self.Hq), 7.0, device=DEV),
                      status=torch.zeros(1, dtype=torch.int32, device=DEV))
        return self

    def call(self, kvc, ws=None, stream=None):
        d = self.d
        if ws is None:
            n = kvc.kvc_tree_attn_workspace_size(self.n_req, self.max_blocks, self.max_tree, self.H,
                                                 self.Hq, self.D, self.BS)
            ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        self.ws = ws
        kvc.kvc_tree_attn(d["q"], d["k"], d["v"], self.n_slots, d["bt"], self.max_blocks, d["ctx"],
                          d["q_off"], d["mask"], self.words, self.n_req, self.n_q, self.max_tree,
                          self.H, self.Hq, self.D, self.BS, self.scale, d["out"], d["lse"], ws,
                          d["status"], stream)
        return d["out"], d["lse"]

    def want(self, bad_blocks=()):
        return ref.attn(self.q, self.k, self.v, self.bt, self.BS, self.ctx, self.q_off, self.mask,
                        self.H, self.scale, bad_blocks)


def check(kvc, t, what=""):
    out, lse = t.gpu().call(kvc)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(t.d["status"]) == 0
    o, ls, ob, lb = t.want()
    inside(out, o, ob, f"out {what}")
    inside(lse, ls, lb, f"lse {what}")


# -------------------------------------------------------------- attention

EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (8, 4), (3, 6), (2, 8), (1, 3), (2, 16)])
@pytest.mark.parametrize("T", [1, 2, 5])
def test_attn_edges(kvc, D, H, G, T):
    """Context lengths on and off every tile edge, short trees."""
    check(kvc, Tree(D + H * 10 + G + T, EDGE, [T] * len(EDGE), H, G, D, 16))


@pytest.mark.parametrize("BS", [1, 2, 5, 8, 12, 16, 32, 48, 64])
@pytest.mark.parametrize("T", [3, 40])
def test_attn_page_sizes(kvc, BS, T):
    check(kvc, Tree(BS, [0, 33, 100, 181], [T, 1, T, max(1, T - 2)], 2, 4, 128, BS))


@pytest.mark.parametrize("kind", ["chain", "tree", "empty", "self", "noself", "full", "holes"])
@pytest.mark.parametrize("ctx,T,G", [([0, 5, 70], [37, 9, 64], 4), ([0, 130], [7, 3], 2),
                                     ([0, 64, 1], [64, 33, 48], 8)])
def test_attn_masks(kvc, kind, ctx, T, G):
    check(kvc, Tree(11, ctx, T, 2, G, 128, 16, kind, pad_words=1), kind)


@pytest.mark.parametrize("T,G,H,D", [(64, 4, 2, 128), (65, 4, 1, 128), (33, 6, 2, 64), (100, 1, 2, 128),
                                     (200, 2, 1, 64), (17, 8, 2, 128), (130, 3, 1, 128), (31, 16, 1, 128)])
def test_attn_many_rows(kvc, T, G, H, D):
    check(kvc, Tree(T, [90, 0, 300], [T, max(1, T // 2), T - 1], H, G, D, 16))


@pytest.mark.parametrize("T,G,kind", [(1, 4, "chain"), (6, 4, "tree"), (30, 4, "tree")])
@pytest.mark.parametrize("BS", [16, 24])
def test_attn_long_context(kvc, T, G, kind, BS):
    """Long and very different lengths in one batch: work split over the positions and joined."""
    check(kvc, Tree(5, [5000, 3, 1700, 0, 9000], [T] * 5, 2, G, 128, BS, kind))


@pytest.mark.parametrize("ctx,H,T,G,D,kind", [
    ([40000], 1, 1, 4, 128, "chain"), ([40000], 1, 7, 2, 64, "tree"), ([20000, 0, 9000, 33], 2, 8, 4, 128, "tree"),
    ([11500, 700, 11000, 40], 13, 2, 3, 128, "tree")])
def test_attn_few_rows_over_long_caches(kvc, ctx, H, T, G, D, kind):
    """Caches so long that their positions are dealt out over the whole GPU, a unit cut into many parts
    or into a few."""
    check(kvc, Tree(9, ctx, [T] * len(ctx), H, G, D, 16, kind, poison=False))


@pytest.mark.parametrize("n_req,ctx", [(1, 30), (1, 1000), (2, 4000), (9, 2100), (40, 70)])
@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (3, 5, 64), (8, 4, 128)])
def test_attn_few_rows_over_short_caches(kvc, n_req, ctx, T, G, D):
    """Units shared by clusters of 1 to 16 CTAs, some of them without a tile."""
    c = [ctx] + [(ctx * (r % 7)) // 7 for r in range(1, n_req)]
    check(kvc, Tree(8, c, [T] * n_req, 2, G, D, 8, "tree" if T > 1 else "chain"))


@pytest.mark.parametrize("D,BS,G,T", [(128, 16, 4, (64, 20, 33, 9)), (64, 8, 8, (30, 12, 17, 5)),
                                      (128, 12, 4, (40, 64, 10, 25)), (128, 32, 4, (30, 9, 16, 31))])
def test_attn_many_units(kvc, D, BS, G, T):
    """More (request, head) units than CTAs, trees of very different size: a CTA works on several in
    turn, with one or two teams' rows each."""
    ctx = [300 + 37 * r for r in range(16)]
    check(kvc, Tree(D + BS, ctx, [T[r % 4] for r in range(16)], 12, G, D, BS))


def test_attn_longest_tree(kvc):
    check(kvc, Tree(3, [10], [1024], 1, 1, 64, 16, "chain"))


@pytest.mark.parametrize("T,G", [(1, 4), (12, 4), (64, 4)])
@pytest.mark.parametrize("kscale", [0.0, 8.0, 60.0])
def test_attn_extreme_logits(kvc, T, G, kscale):
    """All logits equal, and logits of hundreds: one key takes all."""
    check(kvc, Tree(17, [700, 64], [T, T], 2, G, 128, 16, "chain", kscale), f"scale {kscale}")


@pytest.mark.parametrize("T,G", [(1, 4), (12, 4), (64, 4)])
@pytest.mark.parametrize("order", ["rising", "falling", "late"])
def test_attn_moving_maximum(kvc, T, G, order):
    """The maximum climbs by hundreds from tile to tile, falls, or jumps at the last positions."""
    t = Tree(23, [1500], [T], 1, G, 128, 16, "chain", poison=False)
    n = 1500 + T
    s = ref.slots(t.bt[0], 16, n)
    level = {"rising": torch.linspace(-300, 300, n), "falling": torch.linspace(300, -300, n),
             "late": torch.where(torch.arange(n) > n - 3, 250.0, -250.0)}[order]
    t.q[..., 0] = 1.0
    t.k[s, 0, 0] = (level / t.scale).to(torch.bfloat16)
    check(kvc, t, order)


def test_attn_non_finite_values(kvc):
    """Infinite and NaN V of a node reach exactly the rows that see the node."""
    for T, G in [(5, 2), (40, 4)]:
        t = Tree(29, [50, 0], [T, T], 2, G, 128, 16, "tree")
        for r, j, h, d, val in [(0, 2, 0, 7, math.inf), (0, T - 1, 1, 100, -math.inf), (1, 1, 0, 3, NAN)]:
            t.v[ref.slots(t.bt[r], 16, t.ctx[r] + T)[t.ctx[r] + j], h, d] = val
        out, lse = t.gpu().call(kvc)
        torch.cuda.synchronize()
        o, ls, ob, lb = t.want()
        ob = torch.where(torch.isfinite(ob), ob, torch.ones_like(ob))
        inside(out, o, ob, "out")
        inside(lse, ls, lb, "lse")


def test_attn_bad_requests_are_skipped(kvc):
    """Each kind of bad size: recorded, the request's rows untouched, the others right."""
    base = Tree(31, [20, 30, 40, 50], [4, 4, 4, 4], 2, 4, 128, 16)
    o, ls, ob, lb = base.want()
    for field, at, val in [("ctx", 1, -1), ("ctx", 1, 61), ("ctx", 1, 1 << 30), ("q_off", 4, 17),
                           ("q_off", 4, 11), ("q_off", 4, 1 << 30), ("q_off", 0, -3)]:
        base.gpu()
        base.d[field][at] = val
        skipped = {("ctx", 1): 1, ("q_off", 4): 3, ("q_off", 0): 0}[(field, at)]
        out, lse = base.call(kvc)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(base.d["status"]) == 7, (field, val)
        sl = slice(4 * skipped, 4 * skipped + 4)
        assert torch.all(out[sl] == 7.0) and torch.all(lse[sl] == 7.0)
        keep = [i for i in range(16) if i // 4 != skipped]
        inside(out[keep], o[keep], ob[keep], "out")
        inside(lse[keep], ls[keep], lb[keep], "lse")


@pytest.mark.parametrize("bad", [-1, 1 << 20, 2147483647])
@pytest.mark.parametrize("T", [3, 40])
def test_attn_bad_block_is_not_visible(kvc, bad, T):
    t = Tree(37, [100, 60], [T, T], 2, 4, 128, 16, poison=False)
    t.bt[0][2] = bad
    t.bt[1][0] = bad
    out, lse = t.gpu().call(kvc)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(t.d["status"]) == 7
    o, ls, ob, lb = t.want(bad_blocks=(bad,))
    inside(out, o, ob, "out")
    inside(lse, ls, lb, "lse")


def test_attn_repeats_streams_and_graphs(kvc):
    """The same bits again, on another stream, and from a captured graph after the inputs changed;
    the workspace's contents do not matter."""
    t = Tree(41, [2000, 77, 0], [20, 7, 3], 2, 4, 128, 16).gpu()
    a, la = (x.clone() for x in t.call(kvc))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    t.ws.fill_(0x55)
    st.wait_stream(torch.cuda.current_stream())
    t.call(kvc, t.ws, st)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), t.d["out"].view(torch.int16)) and torch.equal(la, t.d["lse"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.call(kvc, t.ws)
    t.d["q"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    t.q = t.d["q"].cpu()
    o, ls, ob, lb = t.want()
    inside(t.d["out"], o, ob, "out from the graph")
    inside(t.d["lse"], ls, lb, "lse from the graph")


def test_offsets_past_32_bits(kvc):
    """Pages whose element offsets pass 2^32: attention, weight, commit and eviction."""
    H, G, D, BS, n_blocks = 8, 1, 128, 64, 68000          # 4.46e9 elements a pool
    c, T = 100, 3
    k = torch.zeros(n_blocks * BS, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    bt = np.array([[n_blocks - 1, n_blocks - 5, 1]])
    s = ref.slots(bt[0], BS, c + T)
    kr, vr = rows(1, c + T, H, D), rows(2, c + T, H, D)
    k[s.to(DEV)], v[s.to(DEV)] = kr.to(DEV), vr.to(DEV)
    q = rows(3, T, H * G, D)
    # the same rows in a small pool for the reference
    small = np.arange(3)[None]
    k2, v2 = torch.zeros(3 * BS, H, D, dtype=torch.bfloat16), torch.zeros(3 * BS, H, D, dtype=torch.bfloat16)
    k2[ref.slots(small[0], BS, c + T)], v2[ref.slots(small[0], BS, c + T)] = kr, vr
    o, ls, ob, lb = ref.attn(q, k2, v2, small, BS, [c], [0, T], None, H, 0.1)
    out = torch.empty(T, H * G, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, H * G, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(kvc.kvc_tree_attn_workspace_size(1, 3, T, H, H * G, D, BS), dtype=torch.uint8, device=DEV)
    kvc.kvc_tree_attn(q.to(DEV), k, v, n_blocks * BS, i32(bt), 3, i32([c]), i32([0, T]), None, 1, 1, T, T,
                      H, H * G, D, BS, 0.1, out, lse, ws, st)
    inside(out, o, ob, "out")
    inside(lse, ls, lb, "lse")
    m = torch.zeros(1, 1, H, 192, device=DEV)
    wsb = kvc.kvc_attn_mass_workspace_size(1, 3, T, 1, H, H * G, D, BS)
    kvc.kvc_attn_mass(q.to(DEV)[None], lse[None], T, None, i32([101, 102, 103]), i32([0, T]), T, T, k[None],
                      n_blocks * BS, i32(bt), 3, i32([c + T]), i32([0]), 1, 1, H, H * G, D, BS, 0.1, 1.0, m,
                      torch.empty(max(16, wsb), dtype=torch.uint8, device=DEV), st)
    want, bound = ref.mass(q[None], lse.cpu()[None], None, [101, 102, 103], [0, T], k2[None], small, BS,
                           [c + T], [0], torch.zeros(1, 1, H, 192), H, 0.1, 1.0)
    inside(m, want, bound, "mass")
    so = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvc.kvc_tree_commit(k[None], v[None], n_blocks * BS, i32(bt), 3, i32([c]), i32([0, T]), i32([[0, 2]]),
                        i32([2]), 2, 1, 1, H, D, BS, so, None, None, st)
    assert torch.equal(k[s[c + 1]].cpu(), kr[c + 2]) and torch.equal(v[s[c + 1]].cpu(), vr[c + 2])
    mo, po = torch.zeros_like(m), torch.zeros(1, 1, H, 192, dtype=torch.int32, device=DEV)
    m[..., :c] = torch.arange(c, device=DEV).float()       # the last rows are the heaviest
    kvc.kvc_mass_evict(k[None], v[None], n_blocks * BS, i32(bt), 3, i32([c]), i32([0]), i32([c]), m, po, mo,
                       po, so, 1, 1, H, D, BS, 40, 0, 0, None, st)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(st) == 0
    assert torch.equal(k[s[:40]].cpu(), kr[60:100]) and torch.equal(v[s[:40]].cpu(), vr[60:100])


# ---------------------------------------------------- accumulated weight

class Mass:
    def __init__(self, seed, seq, m, L, H, G, D, BS, kind="path", decay=1.0, kscale=1.0, extra=0):
        rng = np.random.default_rng(seed)
        self.seq, self.L, self.H, self.G, self.D, self.BS = list(seq), L, H, G, D, BS
        self.n_req, self.Hq, self.decay = len(seq), H * G, decay
        m = [min(a, b) for a, b in zip(m, seq)]
        self.max_rows = max(max(m), 1)
        self.max_blocks = max(1, max(-(-(n + extra) // BS) for n in seq))
        self.cap = self.max_blocks * BS
        self.bt, n_blocks = table(rng, self.n_req, self.max_blocks)
        self.n_slots = n_blocks * BS
        vis = [seq[r] - m[r] + 1 + np.arange(m[r]) for r in range(self.n_req)]
        if kind == "path":
            per = 2 * self.max_rows + 3
            self.n_q = self.n_req * per
            self.row_off = np.arange(self.n_req + 1) * self.max_rows
            self.row_idx = np.zeros((self.n_req, self.max_rows), np.int64)
            self.row_vis = np.zeros((self.n_req, self.max_rows), np.int64)
            for r in range(self.n_req):
                self.row_idx[r, :m[r]] = r * per + np.sort(rng.permutation(per)[:m[r]])
                self.row_vis[r, :m[r]] = vis[r]
            self.row_idx, self.row_vis = self.row_idx.reshape(-1), self.row_vis.reshape(-1)
        else:
            self.row_off = np.concatenate([[0], np.cumsum(m)])
            self.row_idx, self.row_vis = None, np.concatenate(vis)
            if len(self.row_vis) == 0:
                self.row_vis = np.zeros(1, np.int64)
            self.n_q = len(self.row_vis)
            if kind == "any":   # no order among the rows' limits, some see nothing, some too much
                self.row_vis = rng.integers(-2, max(seq) + 5, self.n_q)
        self.n_mass = np.array([max(0, a - b) for a, b in zip(seq, m)])
        self.q = rows(seed + 1, L, self.n_q, self.Hq, D, scale=kscale)
        self.k = rows(seed + 2, L, self.n_slots, H, D)
        self.scale = 1.0 / math.sqrt(D)
        self.lse = (torch.rand(L, self.n_q, self.Hq, generator=gen(seed + 3)) * 3 + 4 * kscale).float()
        self.old = torch.rand(L, self.n_req, H, self.cap, generator=gen(seed + 4))

    def gpu(self):
        self.d = dict(q=self.q.to(DEV), lse=self.lse.to(DEV), k=self.k.to(DEV), bt=i32(self.bt),
                      idx=None if self.row_idx is None else i32(self.row_idx), vis=i32(self.row_vis),
                      off=i32(self.row_off), seq=i32(self.seq), n_mass=i32(self.n_mass),
                      mass=self.old.to(DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))
        return self

    def call(self, kvc, stream=None):
        d = self.d
        n = kvc.kvc_attn_mass_workspace_size(self.n_req, self.max_blocks, self.max_rows, self.L, self.H,
                                             self.Hq, self.D, self.BS)
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
        self.ws = ws
        kvc.kvc_attn_mass(d["q"], d["lse"], self.n_q, d["idx"], d["vis"], d["off"], len(self.row_vis),
                          self.max_rows, d["k"], self.n_slots, d["bt"], self.max_blocks, d["seq"],
                          d["n_mass"], self.n_req, self.L, self.H, self.Hq, self.D, self.BS, self.scale,
                          self.decay, d["mass"], ws, d["status"], stream)
        return d["mass"]

    def want(self, bad_blocks=()):
        return ref.mass(self.q, self.lse, self.row_idx, self.row_vis, self.row_off, self.k, self.bt,
                        self.BS, self.seq, self.n_mass, self.old, self.H, self.scale, self.decay,
                        bad_blocks)


def check_mass(kvc, m, what="", status=0, bad_blocks=()):
    got = m.gpu().call(kvc)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(m.d["status"]) == status
    want, bound = m.want(bad_blocks)
    for r in range(m.n_req):  # positions past the sequence are untouched, to the bit
        assert torch.equal(got[:, r, :, m.seq[r]:].cpu(), m.old[:, r, :, m.seq[r]:]), "untouched part"
    inside(got, want, bound, f"mass {what}")


SEQ = [1, 2, 15, 16, 17, 64, 65, 128, 129, 200, 0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (8, 4), (3, 6), (2, 8), (1, 5), (1, 16)])
@pytest.mark.parametrize("m", [1, 5])
def test_mass_path(kvc, D, H, G, m):
    check_mass(kvc, Mass(D + H + G, SEQ, [m] * len(SEQ), 2, H, G, D, 16, decay=0.9))


@pytest.mark.parametrize("BS", [1, 5, 8, 16, 24, 32, 64])
@pytest.mark.parametrize("m", [4, 40])
def test_mass_page_sizes(kvc, BS, m):
    check_mass(kvc, Mass(BS, [33, 100, 181], [m] * 3, 1, 2, 4, 128, BS, "window", extra=70))


@pytest.mark.parametrize("m,G,H,D", [(32, 4, 2, 128), (33, 4, 1, 128), (64, 1, 2, 64), (21, 6, 2, 128),
                                     (16, 8, 1, 128), (100, 3, 1, 64), (17, 16, 1, 128)])
def test_mass_windows(kvc, m, G, H, D):
    check_mass(kvc, Mass(m, [700, 130, 5], [m] * 3, 2, H, G, D, 16, "window", decay=0.5))


@pytest.mark.parametrize("n,G,BS", [(300, 4, 16), (257, 1, 32), (520, 3, 16), (400, 8, 64), (333, 4, 20)])
def test_mass_prompt(kvc, n, G, BS):
    """Whole prompts, causal: every row against the positions up to its own."""
    check_mass(kvc, Mass(n, [n, n // 2], [n, n // 2], 1, 2, G, 128, BS, "window"))


@pytest.mark.parametrize("m", [3, 50, 300])
def test_mass_unordered_limits(kvc, m):
    check_mass(kvc, Mass(m, [310, 320, 1], [m, m, 1], 1, 2, 4, 128, 16, "any"))


@pytest.mark.parametrize("m,kind", [(3, "path"), (48, "window"), (260, "window")])
def test_mass_masked_places(kvc, m, kind):
    """Keys no row sees hold NaN and infinities; rows whose LSE is −inf (nothing visible to attention)
    and rows without a limit add nothing."""
    t = Mass(7, [300, 290], [m, m], 1, 2, 4, 128, 16, kind)
    cut = 280
    t.row_vis = np.minimum(t.row_vis, cut)
    for r in range(2):
        s = ref.slots(t.bt[r], 16, t.seq[r])
        t.k[:, s[cut:]] = NAN
        t.k[:, s[cut + 1:cut + 4]] = math.inf
    t.lse[:, ::3] = -math.inf
    t.row_vis[1] = 0
    check_mass(kvc, t)


@pytest.mark.parametrize("m,kind", [(3, "path"), (40, "window")])
def test_mass_bad_inputs(kvc, m, kind):
    base = dict(seq=[60, 70, 80], m=[m] * 3, L=1, H=2, G=4, D=128, BS=16, kind=kind)
    t = Mass(3, **base)
    t.bt[1][2] = 1 << 25                                # a block outside the pool gains nothing
    check_mass(kvc, t, "bad block", 7, (1 << 25,))
    for field, at, val, r in [("seq", 1, -1, 1), ("seq", 1, 81, 1), ("off", 3, 1 << 30, 2), ("off", 0, -1, 0),
                              ("off", 3, 0, 2)]:
        t = Mass(3, **base)
        want, bound = t.want()
        t.gpu()
        t.d[field][at] = val
        got = t.call(kvc)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(t.d["status"]) == 7
        assert torch.equal(got[:, r].cpu(), t.old[:, r]), (field, val)
        keep = [i for i in range(3) if i != r]
        inside(got[:, keep], want[:, keep], bound[:, keep], "others")
    if kind == "path":
        t = Mass(3, **base)
        t.row_idx[0] = t.n_q
        t.gpu()
        got = t.call(kvc)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(t.d["status"]) == 7
        t.row_idx[0], t.row_vis[0] = 0, 0               # the row is left out
        inside(got, *t.want(), "row left out")


@pytest.mark.parametrize("m,kind,G", [(4, "path", 4), (32, "window", 4), (400, "window", 4)])
def test_mass_repeats_and_long_caches(kvc, m, kind, G):
    t = Mass(9, [4000, 900], [m, m], 1, 1, G, 128, 16, kind)
    check_mass(kvc, t)
    a = t.d["mass"].clone()
    t.d["mass"].copy_(t.old)
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        t.call(kvc)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, t.d["mass"])


def test_mass_of_attention_adds_up(kvc):
    """With attention's own LSE every row's weights add up to one per query head."""
    T, G, H = 6, 4, 2
    t = Tree(51, [900], [T], H, G, 128, 16, "chain", poison=False).gpu()
    out, lse = t.call(kvc)
    cap = t.max_blocks * 16
    m = torch.zeros(1, 1, H, cap, device=DEV)
    n = kvc.kvc_attn_mass_workspace_size(1, t.max_blocks, T, 1, H, H * G, 128, 16)
    kvc.kvc_attn_mass(t.d["q"][None], lse[None], T, None, i32(901 + np.arange(T)), i32([0, T]), T, T,
                      t.d["k"][None], t.n_slots, t.d["bt"], t.max_blocks, i32([900 + T]), i32([0]), 1, 1, H,
                      H * G, 128, 16, t.scale, 1.0, m, torch.empty(max(n, 16), dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert float((m.sum(-1) - T * G).abs().max()) < T * G * 1e-5


# ------------------------------------------------------ commit, eviction

@pytest.mark.parametrize("D,H,BS", [(64, 1, 5), (128, 8, 16), (128, 3, 64), (64, 16, 1)])
@pytest.mark.parametrize("max_path", [1, 4, 21])
def test_commit(kvc, D, H, BS, max_path):
    rng = np.random.default_rng(D + H + max_path)
    L, n_req, T = 2, 5, 30
    ctx = np.array([0, 1, 17, 64, 100])
    max_blocks = -(-(100 + T) // BS)
    bt, nb = table(rng, n_req, max_blocks)
    n = np.array([max_path, 0, 1, max_path, max(1, max_path // 2)])
    path = np.full((n_req, max_path), -7)
    for r in range(n_req):
        path[r, :n[r]] = np.sort(rng.permutation(T)[:n[r]])
    path[3, :n[3]] = np.arange(n[3])                    # nothing to move
    k, v = rows(1, L, nb * BS, H, D), rows(2, L, nb * BS, H, D)
    kd, vd = k.to(DEV), v.to(DEV)
    so, ri, rv = (torch.full(s, 9, dtype=torch.int32, device=DEV) for s in ((n_req,), (n_req, max_path),
                                                                            (n_req, max_path)))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_off = np.arange(n_req + 1) * T
    kvc.kvc_tree_commit(kd, vd, nb * BS, i32(bt), max_blocks, i32(ctx), i32(q_off), i32(path), i32(n), max_path,
                        n_req, L, H, D, BS, so, ri, rv, st)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(st) == 0
    kw, vw = k.clone(), v.clone()
    for r in range(n_req):
        s = ref.slots(bt[r], BS, ctx[r] + T)
        for i in range(n[r]):
            kw[:, s[ctx[r] + i]], vw[:, s[ctx[r] + i]] = k[:, s[ctx[r] + path[r, i]]], v[:, s[ctx[r] + path[r, i]]]
    assert torch.equal(kd.cpu(), kw) and torch.equal(vd.cpu(), vw)
    assert np.array_equal(so.cpu().numpy(), ctx + n)
    on = np.arange(max_path) < n[:, None]
    assert np.array_equal(ri.cpu().numpy(), np.where(on, q_off[:-1, None] + path, 0))
    assert np.array_equal(rv.cpu().numpy(), np.where(on, ctx[:, None] + np.arange(max_path) + 1, 0))


def test_commit_bad_inputs(kvc):
    """A path that does not ascend or leaves the tree moves nothing; the other request's rows move."""
    rng = np.random.default_rng(5)
    H, D, BS, T = 2, 64, 16, 8
    bt, nb = table(rng, 2, 4)
    k, v = rows(1, 1, nb * BS, H, D), rows(2, 1, nb * BS, H, D)
    for path, n, ctx, bad_bt in [([0, 0, 2], 3, 20, None), ([0, 3, 2], 3, 20, None), ([0, 3, 8], 3, 20, None),
                                 ([-1, 3, 5], 3, 20, None), ([0, 1, 2], 4, 20, None), ([0, 1, 2], -1, 20, None),
                                 ([0, 2, 3], 3, -4, None), ([0, 2, 3], 3, 57, None), ([0, 2, 3], 3, 20, 1 << 20)]:
        kd, vd = k.to(DEV), v.to(DEV)
        so, rv = (torch.full(s, 9, dtype=torch.int32, device=DEV) for s in ((2,), (2, 3)))
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        tab = bt.copy()
        if bad_bt is not None:
            tab[0, 1] = bad_bt
        kvc.kvc_tree_commit(kd, vd, nb * BS, i32(tab), 4, i32([ctx, 10]), i32([0, T, 2 * T]),
                            i32([path, [1, 2, 4]]), i32([n, 3]), 3, 2, 1, H, D, BS, so, None, rv, st)
        torch.cuda.synchronize()
        assert kvc.kvc_device_status(st) == 7
        s0, s1 = ref.slots(bt[0], BS, 64), ref.slots(bt[1], BS, 64)
        assert torch.equal(kd[:, s0].cpu(), k[:, s0]) and torch.equal(vd[:, s0].cpu(), v[:, s0])
        assert torch.equal(kd[:, s1[[10, 11, 12]]].cpu(), k[:, s1[[11, 12, 14]]])
        if bad_bt is None:
            assert int(so[0]) == max(ctx, 0) and torch.all(rv[0] == 0)


class Evict:
    def __init__(self, seed, seq, budget, L, H, D, BS, n_sink=2, n_recent=3, carried=0.5, weights="mixed",
                 max_blocks=None):
        rng = np.random.default_rng(seed)
        self.seq, self.budget, self.L, self.H, self.D, self.BS = list(seq), budget, L, H, D, BS
        self.n_sink, self.n_recent, self.n_req = n_sink, n_recent, len(seq)
        self.max_blocks = max_blocks or max(1, max(-(-n // BS) for n in seq))
        self.cap = self.max_blocks * BS
        self.bt, nb = table(rng, self.n_req, self.max_blocks)
        self.n_slots = nb * BS
        self.n_pos = np.array([int(n * carried) for n in seq])
        self.t_end = np.array([n + 5 * int(n * carried) for n in seq])
        shape = (L, self.n_req, H, self.cap)
        self.mass = rng.random(shape).astype(np.float32)
        if weights == "mixed":
            self.mass = np.where(rng.random(shape) < 0.3, 0, np.exp(20 * self.mass - 15)).astype(np.float32)
            self.mass[rng.random(shape) < 0.05] *= -0.0
        elif weights == "equal":
            self.mass[:] = 0.5
        elif weights == "nan":
            self.mass[rng.random(shape) < 0.4] = np.nan
            self.mass[rng.random(shape) < 0.1] = np.inf
            self.mass[rng.random(shape) < 0.1] = -np.inf
        self.pos = np.zeros(shape, np.int32)
        for r in range(self.n_req):
            first = self.t_end[r] - (seq[r] - self.n_pos[r])   # original position of the first fresh row
            for layer in range(L):
                for h in range(H):
                    self.pos[layer, r, h, :self.n_pos[r]] = rng.permutation(int(first))[:self.n_pos[r]]
        self.k = rng.integers(-3000, 3000, (L, self.n_slots, H, D)).astype(np.int16)
        self.v = rng.integers(-3000, 3000, (L, self.n_slots, H, D)).astype(np.int16)

    def run(self, kvc, in_place=False):
        kd, vd = (torch.from_numpy(x).to(DEV).view(torch.bfloat16) for x in (self.k, self.v))
        m, p = torch.from_numpy(self.mass).to(DEV), torch.from_numpy(self.pos).to(DEV)
        mo, po = (m, p) if in_place else (m.clone(), p.clone())
        n_out = torch.full((self.n_req,), -5, dtype=torch.int32, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        n = kvc.kvc_mass_evict_workspace_size(self.n_req, self.max_blocks, self.L, self.H, self.BS, self.budget)
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
        kvc.kvc_mass_evict(kd, vd, self.n_slots, i32(self.bt), self.max_blocks, i32(self.seq), i32(self.n_pos),
                           i32(self.t_end), m, p, mo, po, n_out, self.n_req, self.L, self.H, self.D, self.BS,
                           self.budget, self.n_sink, self.n_recent, ws, st)
        torch.cuda.synchronize()
        return (kd.view(torch.int16).cpu().numpy(), vd.view(torch.int16).cpu().numpy(), mo.cpu().numpy(),
                po.cpu().numpy(), n_out.cpu().numpy()), kvc.kvc_device_status(st)

    def want(self, bad_blocks=()):
        return ref.evict(self.k, self.v, self.bt, self.BS, self.seq, self.n_pos, self.t_end, self.mass, self.pos,
                         self.H, self.budget, self.n_sink, self.n_recent, bad_blocks)


def check_evict(kvc, e, in_place=False, status=0, bad_blocks=()):
    got, st = e.run(kvc, in_place)
    assert st == status
    for name, a, b in zip(("k", "v", "mass", "pos", "n_out"), got, e.want(bad_blocks)):
        assert np.array_equal(a.view(np.int32) if a.dtype == np.float32 else a,
                              b.view(np.int32) if b.dtype == np.float32 else b), name


@pytest.mark.parametrize("weights", ["mixed", "equal", "random"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,H,BS", [(128, 2, 16), (64, 3, 5)])
def test_evict(kvc, weights, in_place, D, H, BS):
    check_evict(kvc, Evict(1, [130, 64, 65, 300, 10, 0, 1], 64, 2, H, D, BS, weights=weights), in_place)


@pytest.mark.parametrize("n,B", [(2, 1), (100, 99), (100, 1), (512, 256), (1000, 37), (4160, 4096), (6144, 4096),
                                 (33000, 20000)])
def test_evict_sizes(kvc, n, B):
    check_evict(kvc, Evict(n + B, [n], B, 1, 2, 64, 16, min(2, B // 4), min(8, B // 4)), in_place=True)


@pytest.mark.parametrize("sink,recent", [(0, 0), (64, 0), (0, 64), (10, 54)])
@pytest.mark.parametrize("carried", [0.0, 1.0, 0.7])
def test_evict_pinned_rows(kvc, sink, recent, carried):
    check_evict(kvc, Evict(sink + recent, [200, 64, 150], 64, 1, 2, 64, 16, sink, recent, carried))


def test_evict_more_pinned_than_budget(kvc):
    """Repeated positions can pin more rows than the budget holds: the lowest rows stay."""
    e = Evict(2, [120], 16, 1, 2, 64, 16, 4, 4, carried=1.0)
    e.pos[..., 40:100] = 1
    check_evict(kvc, e)


def test_evict_nan_is_recorded_and_last(kvc):
    check_evict(kvc, Evict(3, [150, 90], 64, 1, 2, 64, 16, weights="nan"), status=8)


def test_evict_long_segments(kvc):
    """Past the staged length the weights are read from global memory on each pass."""
    check_evict(kvc, Evict(4, [52000, 300], 8000, 1, 1, 64, 16), in_place=True)


def test_evict_many_segments(kvc):
    check_evict(kvc, Evict(5, [60] * 40, 32, 10, 4, 64, 16))


def test_evict_bad_inputs(kvc):
    e = Evict(6, [150, 160], 64, 1, 2, 64, 16)
    good = int(e.bt[0][0])
    e.bt[0][7] = -3                                       # K and V of its rows stay where they are
    check_evict(kvc, e, status=7, bad_blocks=(-3,))
    assert good >= 0
    for val in (-1, 161, 1 << 30):
        e = Evict(6, [150, 160], 64, 1, 2, 64, 16)
        want = e.want()
        e.seq[0] = val
        got, st = e.run(kvc)
        assert st == 7 and got[4][0] == 0 and got[4][1] == 64
        assert np.array_equal(got[2][:, 0], e.mass[:, 0]) and np.array_equal(got[2][:, 1], want[2][:, 1])
        s1 = ref.slots(e.bt[1], 16, 160).numpy()
        assert np.array_equal(got[0][:, s1], want[0][:, s1])
        s0 = ref.slots(e.bt[0], 16, 150).numpy()
        assert np.array_equal(got[0][:, s0], e.k[:, s0])
