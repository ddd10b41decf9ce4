"""Filling the paged cache and reading its 8-bit part on the GPU, against 64-bit forms
(tests/prefill_ref.py), at the sizes, masks and values where each can go wrong.  Tolerances are counted
in half steps of the types there; integers, copies and codes are exact."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import prefill_ref as ref  # noqa: E402
import tree_ref  # noqa: E402

DEV = "cuda"
NAN, INF = float("nan"), float("inf")
BOUNDS, NAN_CODE = 7, 8
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def kvc():
    import query_conditioned_kv_gb300 as k
    return k


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def rows(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


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


def status(kvc, t):
    torch.cuda.synchronize()
    return kvc.kvc_device_status(t)


class Batch:
    """Requests with ctx cached rows and T new ones, over a paged pool, on the host.  `room`: pages of
    a request's table past what it needs."""

    def __init__(self, seed, ctx, T, H, G, D, BS, pad=0, kscale=1.0, poison=True, room=0):
        self.rng = np.random.default_rng(seed)
        self.ctx, self.T, self.H, self.G, self.D, self.BS = list(ctx), list(T), H, G, D, BS
        self.n_req, self.Hq = len(ctx), H * G
        self.max_rows = max(max(T), 1)
        self.max_blocks = max(1, max(-(-(c + t) // BS) for c, t in zip(ctx, T))) + room
        self.bt, n_blocks = table(self.rng, self.n_req, self.max_blocks)
        self.n_slots = n_blocks * BS
        self.q_off = np.concatenate([[0], np.cumsum(T)])
        self.n_q = int(self.q_off[-1]) + pad
        self.q = rows(seed + 1, max(self.n_q, 1), self.Hq, D, scale=kscale)
        self.k, self.v = rows(seed + 2, self.n_slots, H, D), rows(seed + 3, self.n_slots, H, D)
        self.scale = 1.0 / math.sqrt(D)
        if poison:  # every slot that holds no position of a request
            held = np.zeros(self.n_slots, bool)
            for r in range(self.n_req):
                held[tree_ref.slots(self.bt[r], BS, self.ctx[r] + self.T[r]).numpy()] = True
            self.k[~held], self.v[~held] = NAN, NAN

    def common(self):
        return dict(bt=i32(self.bt), ctx=i32(self.ctx), q_off=i32(self.q_off),
                    status=torch.zeros(1, dtype=torch.int32, device=DEV))


# ------------------------------------------------- norms, rotation, storing

class Rope(Batch):
    def __init__(self, *a, norm=(True, True), raw=True, shift=0, fused=True, **k):
        super().__init__(*a, **k)
        self.n = self.n_q
        D, w = self.D, (self.Hq + 2 * self.H) * self.D
        self.qkv = rows(77, self.n, w + (8 if fused else 0), scale=2.0)
        self.wq, self.wk = ((1 + 0.3 * rows(78 + i, D).float()).bfloat16() if norm[i] else None for i in range(2))
        self.pos = np.concatenate([c + np.arange(t) for c, t in zip(self.ctx, self.T)] +
                                  [np.zeros(self.n - int(self.q_off[-1]), np.int64)]).astype(np.int64) + shift
        self.n_pos = int(self.pos.max()) + 1
        self.tab = ref.rope_table(self.n_pos, D)
        self.raw, self.shift, self.eps = raw, shift, 1e-6

    def parts(self, x):
        a, b = self.Hq * self.D, (self.Hq + self.H) * self.D
        return x[:, :a], x[:, a:b], x[:, b:b + self.H * self.D]

    def gpu(self):
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.d = dict(self.common(), x=self.qkv.to(DEV), wq=dev(self.wq), wk=dev(self.wk),
                      tab=self.tab.to(DEV), pos=i32(self.pos) if self.shift else None,
                      k=self.k.to(DEV), v=self.v.to(DEV),
                      out=torch.full((self.n, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV),
                      raw=torch.full((self.H, self.n + 3, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
                      if self.raw else None)
        return self

    def call(self, kvc, stream=None, **over):
        d = dict(self.d, **over)
        q, k, v = self.parts(d["x"])
        kvc.kvc_qkv_rope(d.get("q", q), k, v, self.n, d["wq"], d["wk"], self.eps, d["tab"], self.n_pos,
                         d["pos"], d["q_off"], d["ctx"], self.n_req, d["bt"], self.max_blocks, d["k"],
                         d["v"], self.n_slots, self.H, self.Hq, self.D, self.BS, d["out"], d["raw"],
                         d["status"], stream)

    def check(self, skip=(), no_store=()):
        """All outputs; `skip`: tokens left out, `no_store`: tokens whose page is bad."""
        D, n_live = self.D, int(self.q_off[-1])
        q, k, v = (p.reshape(self.n, -1, D) for p in self.parts(self.qkv))
        y, rel = ref.normed(q, self.wq, self.eps)
        want, bound = ref.rotated(y, rel, self.tab[self.pos])
        live = np.array([i for i in range(n_live) if i not in skip], dtype=np.int64)
        dead = np.setdiff1d(np.arange(self.n), live)
        out = self.d["out"].cpu()
        inside(out[live], want[live], bound[live], "q")
        assert bool((out[dead] == 7.0).all())
        y, rel = ref.normed(k, self.wk, self.eps)
        want, bound = ref.rotated(y, rel, self.tab[self.pos])
        kk, vv, bb = self.k.double(), self.v.clone(), torch.zeros(self.k.shape, dtype=torch.float64)
        for r in range(self.n_req):
            s = tree_ref.slots(self.bt[r] % (self.n_slots // self.BS), self.BS, self.ctx[r] + self.T[r])
            for i in range(self.T[r]):
                x = int(self.q_off[r]) + i
                if x in skip or x in no_store:
                    continue
                at = s[self.ctx[r] + i]
                kk[at], bb[at], vv[at] = want[x], bound[x], v[x]
        inside(self.d["k"], kk, bb, "K")
        got = self.d["v"].cpu()
        assert torch.equal(got.view(torch.int16), vv.view(torch.int16))
        if self.raw:
            got = self.d["raw"].cpu()
            inside(got[:, live], y.transpose(0, 1)[:, live],
                   ((rel + ref.UBF * (1 + rel)) * y.abs() + 1e-38).transpose(0, 1)[:, live], "raw K")
            assert bool((got[:, dead] == 7.0).all()) and bool((got[:, self.n:] == 7.0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (8, 4), (3, 6), (1, 3), (16, 1), (5, 2)])
def test_rope_heads(kvc, D, H, G):
    t = Rope(D + H + G, [0, 5, 31, 0], [1, 17, 0, 40], H, G, D, 16, pad=3).gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


@pytest.mark.parametrize("BS", [1, 5, 8, 16, 48, 64])
@pytest.mark.parametrize("norm", [(True, True), (False, False), (True, False), (False, True)])
def test_rope_pages_and_norms(kvc, BS, norm):
    t = Rope(BS, [3, 64, 0], [33, 1, 7], 2, 4, 128, BS, norm=norm, raw=norm[0], shift=1234, fused=norm[1]).gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


@pytest.mark.parametrize("n_req", [1, 31, 32, 33, 1000, 1025])
def test_rope_finds_requests(kvc, n_req):
    rng = np.random.default_rng(n_req)
    T = rng.integers(0, 3, n_req)
    T[-1] = 2
    t = Rope(n_req, rng.integers(0, 9, n_req), T, 1, 2, 64, 4, pad=1).gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


def test_rope_many_tokens_and_offset_start(kvc):
    """Enough tokens for a warp each; the first request begins past token 0."""
    t = Rope(9, [0, 100], [2500, 1201], 2, 3, 128, 16, shift=7)
    t.q_off = t.q_off.copy()
    t.gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()
    t = Rope(10, [4, 9], [20, 6], 2, 3, 128, 16)
    t.q_off = np.array([3, 23, 26])  # (three tokens before it, the second request cut to three)
    t.T = [20, 3]
    t.pos = np.concatenate([[0] * 3, 4 + np.arange(20), 9 + np.arange(3)])
    t.gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    out = t.d["out"].clone()
    assert bool((out[:3] == 7).all())
    t.check(skip=(0, 1, 2))


def test_rope_in_place_and_extreme_values(kvc):
    t = Rope(11, [0, 6], [30, 5], 2, 2, 128, 8, fused=False)
    t.qkv[0, :128] = 0                      # a zero head: eps keeps it 0
    t.qkv[1, 0] = INF
    t.qkv[2, 3] = NAN
    t.qkv[3, :128] = 3e38                   # the squares pass fp32: y = 0
    t.gpu()
    q = t.parts(t.qkv)[0].contiguous().view(-1, t.Hq, t.D).to(DEV)
    t.call(kvc)
    first = t.d["out"].clone()
    t.d["out"] = q
    t.call(kvc, q=q)
    assert status(kvc, t.d["status"]) == 0
    assert torch.equal(first.view(torch.int16), q.view(torch.int16))
    assert bool((first[0, 0] == 0).all()) and bool((first[3, 0] == 0).all())
    assert bool(torch.isnan(first[2, 0]).any())
    t.d["out"] = first
    ok = [i for i in range(t.n) if i not in (1, 2, 3)]
    y, rel = ref.normed(t.parts(t.qkv)[0].reshape(t.n, -1, 128), t.wq, t.eps)
    want, bound = ref.rotated(y, rel, t.tab[t.pos])
    inside(first[ok], want[ok], bound[ok], "q")


def test_rope_bad_pages_positions_and_requests(kvc):
    def go(change, skip=(), no_store=()):
        t = Rope(13, [0, 7, 3], [20, 9, 4], 2, 2, 64, 8, shift=5)
        change(t)
        t.gpu()
        t.call(kvc)
        assert status(kvc, t.d["status"]) == BOUNDS
        t.check(skip, no_store)

    def page(t):
        t.bt[0, 1] = t.n_slots // 8

    def negative(t):
        t.bt[1, 1] = -1

    go(page, no_store=range(8, 16))
    go(negative, no_store=range(21, 29))

    def place(t):
        t.pos[4], t.pos[25] = t.n_pos, -1
    t = Rope(13, [0, 7, 3], [20, 9, 4], 2, 2, 64, 8, shift=5)
    place(t)
    t.gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == BOUNDS
    t.pos = t.pos.clip(0, t.n_pos - 1)
    t.check(skip=(4, 25))

    t = Rope(14, [0, 7, 3], [20, 9, 4], 2, 2, 64, 8).gpu()
    t.d["ctx"] = i32([0, 1 << 20, -1])
    t.call(kvc)
    assert status(kvc, t.d["status"]) == BOUNDS
    t.check(skip=range(20, 33))
    t = Rope(14, [0, 7, 3], [20, 9, 4], 2, 2, 64, 8).gpu()
    t.d["q_off"] = i32([0, 20, 29, 1 << 30])
    t.call(kvc)
    assert status(kvc, t.d["status"]) == BOUNDS
    t.check(skip=range(29, 33))


@pytest.mark.parametrize("D", [64, 128])
def test_rope_raw_keys_make_the_block_means(kvc, D):
    """k_raw as kvc_build_meank takes it: the means of the keys that the projection's norm gives."""
    t = Rope(69, [0], [96], 3, 2, D, 16, fused=False).gpu()
    t.d["raw"] = torch.empty(3, 96, D, dtype=torch.bfloat16, device=DEV)
    t.call(kvc)
    mean = torch.empty(1, 3, 3, D, dtype=torch.bfloat16, device=DEV)
    kvc.kvc_build_meank(t.d["raw"][None], mean, 1, 3, D, 96, t.d["status"])
    assert status(kvc, t.d["status"]) == 0
    y, rel = ref.normed(t.parts(t.qkv)[1].reshape(96, 3, D), t.wk, t.eps)
    y = y.transpose(0, 1).reshape(3, 3, 32, D)
    want = y.mean(2)
    bound = (rel + ref.UBF * (1 + rel)) * y.abs().mean(2)
    inside(mean[0], want, bound + ref.UBF * (want.abs() + bound) + 1e-38, "block means")


def test_rope_repeats_replays_and_streams(kvc):
    t = Rope(15, [40, 3], [1, 1], 8, 4, 128, 16).gpu()
    t.call(kvc)
    want = [t.d[n].clone() for n in ("out", "k", "v", "raw")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t.gpu()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.call(kvc)
    g.replay()
    torch.cuda.synchronize()
    for n, w in zip(("out", "k", "v", "raw"), want):
        assert torch.equal(t.d[n].view(torch.int16), w.view(torch.int16))
    t.gpu()
    torch.cuda.synchronize()
    t.call(kvc, stream=side)
    torch.cuda.synchronize()
    for n, w in zip(("out", "k", "v", "raw"), want):
        assert torch.equal(t.d[n].view(torch.int16), w.view(torch.int16))


# ------------------------------------------------------------------ prompts

class Prompt(Batch):
    def gpu(self):
        n = max(self.n_q, 1)
        self.d = dict(self.common(), q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV),
                      out=torch.full((n, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV),
                      lse=torch.full((n, self.Hq), 7.0, device=DEV))
        return self

    def call(self, kvc, stream=None):
        d = self.d
        kvc.kvc_prompt_attn(d["q"], d["k"], d["v"], self.n_slots, d["bt"], self.max_blocks, d["ctx"],
                            d["q_off"], self.n_req, max(self.n_q, 1), self.max_rows, self.H, self.Hq,
                            self.D, self.BS, self.scale, d["out"], d["lse"], d["status"], stream)
        return d["out"], d["lse"]

    def want(self, bad_blocks=()):
        return ref.prompt(self.q, self.k, self.v, self.bt, self.BS, self.ctx, self.q_off, self.H,
                          self.scale, bad_blocks)

    def compare(self, bad_blocks=(), live=None):
        o, ls, ob, lb = self.want(bad_blocks)
        n = int(self.q_off[-1])
        live = np.arange(n) if live is None else np.asarray(live, dtype=np.int64)
        dead = np.setdiff1d(np.arange(max(self.n_q, 1)), live)
        out, lse = self.d["out"].cpu(), self.d["lse"].cpu()
        inside(out[live], o[live], ob[live], "out")
        inside(lse[live], ls[live], lb[live], "lse")
        assert bool((out[dead] == 7.0).all()) and bool((lse[dead] == 7.0).all())


def go(kvc, t, want=0, **k):
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == want
    t.compare(**k)


EDGE = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (3, 6), (2, 8), (1, 3), (1, 5), (2, 16)])
def test_prompt_edges(kvc, D, H, G):
    """Whole prompts of lengths on and off every tile edge, one empty, rows behind the last."""
    go(kvc, Prompt(D + H * 10 + G, [0] * len(EDGE), EDGE, H, G, D, 16, pad=2))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_prompt_behind_a_cache(kvc, D, G):
    """Chunks behind cached rows, on and off the tile edges."""
    ctx = [1, 17, 63, 64, 127, 128, 129, 255, 256, 300, 511, 0]
    go(kvc, Prompt(D + G, ctx, [70, 1, 64, 65, 3, 128, 129, 2, 31, 300, 5, 9], 2, G, D, 16, pad=1))


@pytest.mark.parametrize("BS", [1, 2, 5, 8, 12, 16, 24, 32, 48, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_page_sizes(kvc, BS, D):
    go(kvc, Prompt(BS, [0, 133, 7], [300, 140, 129], 2, 4, D, BS))


@pytest.mark.parametrize("H,G", [(1, 64), (1, 100), (1, 128), (1, 130), (1, 256), (2, 128), (2, 65), (4, 33),
                                 (32, 1), (256, 1)])
def test_prompt_wide_groups(kvc, H, G):
    """Groups that fill a tile, do not divide it, or are wider than one."""
    go(kvc, Prompt(H + G, [0, 20], [40, 3], H, G, 64, 16))


@pytest.mark.parametrize("T,ctx,H,G,D", [(1500, 0, 1, 2, 128), (700, 900, 2, 1, 64), (1030, 3, 1, 4, 128)])
def test_prompt_long(kvc, T, ctx, H, G, D):
    go(kvc, Prompt(T, [ctx], [T], H, G, D, 16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,ctx", [([5], [700]), ([130, 3], [300, 1900]), ([40, 0, 64, 1], [0, 900, 127, 2049]),
                                   ([65, 200], [1000, 0])])
@pytest.mark.parametrize("G", [1, 4, 5])
def test_prompt_few_rows_behind_long_caches(kvc, D, T, ctx, G):
    """Few units, whose keys a cluster's CTAs share; some parts hold no key that a row sees."""
    go(kvc, Prompt(D + G + T[0], ctx, T, 2, G, D, 16, pad=1))


@pytest.mark.parametrize("room", [1, 6, 40, 200])
def test_prompt_room_in_the_table(kvc, room):
    """Tables longer than the requests: clusters of every size over few keys, most parts empty."""
    for D, G, BS in ((128, 4, 16), (64, 2, 5)):
        t = Prompt(room, [0, 31], [70, 140], 1, G, D, BS, room=room * 16 // BS, pad=1)
        go(kvc, t)


@pytest.mark.parametrize("T,ctx,H,G,D", [([3, 20, 7], [3000, 2900, 3100], 64, 1, 64), ([9, 0, 40, 1], [2500, 9, 2400, 0], 80, 2, 64),
                                         ([70, 33], [4000, 4100], 40, 4, 128)])
def test_prompt_more_units_than_sms(kvc, T, ctx, H, G, D):
    """More units of about a size than the GPU holds at once."""
    go(kvc, Prompt(83, ctx, T, H, G, D, 16, pad=2))


def test_prompt_equals_chain_rows(kvc):
    """The rows of a whole prompt are those of its pieces (within both bounds)."""
    t = Prompt(31, [0], [400], 2, 4, 128, 16).gpu()
    whole, lse = (x.clone() for x in t.call(kvc))
    o, ls, ob, lb = t.want()
    for a, b in ((0, 1), (1, 130), (130, 399), (399, 400)):
        p = Prompt(31, [a], [b - a], 2, 4, 128, 16)
        p.bt, p.k, p.v, p.n_slots, p.max_blocks = t.bt, t.k, t.v, t.n_slots, t.max_blocks
        p.q = t.q[a:b].contiguous()
        p.gpu().call(kvc)
        assert status(kvc, p.d["status"]) == 0
        inside(p.d["out"], o[a:b], ob[a:b], f"rows {a}:{b}")
        inside(p.d["lse"], ls[a:b], lb[a:b], f"lse {a}:{b}")
        assert float((p.d["lse"] - lse[a:b]).abs().max()) <= 2 * float(lb.max())


@pytest.mark.parametrize("kscale", [0.0, 1e-20, 30.0, 3000.0, 1e18])
def test_prompt_logit_ranges(kvc, kscale):
    """Flat, peaked and huge logits, whose maxima move from tile to tile."""
    for room in (0, 100):
        go(kvc, Prompt(41, [3, 0], [333, 290], 2, 2, 128, 16, kscale=kscale, room=room))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0 ** -100])
def test_prompt_scales(kvc, scale):
    t = Prompt(43, [3, 0], [150, 290], 2, 2, 64, 16)
    t.scale = scale
    go(kvc, t)


def test_prompt_rising_maxima(kvc):
    """Every key is more attended to than all before it, by steps that pass any one-time reference."""
    t = Prompt(47, [0], [600], 1, 2, 64, 16, poison=False)
    s = tree_ref.slots(t.bt[0], 16, 600)
    t.q[:] = 1.0
    t.k[s, 0] = (torch.arange(600, dtype=torch.float32) / 4).to(torch.bfloat16)[:, None]
    t.scale = 1.0
    go(kvc, t)
    t.k[s, 0] = -t.k[s, 0]
    go(kvc, t)


@pytest.mark.parametrize("T,ctx", [([600], [0]), ([40], [900]), ([5], [3000])])
def test_prompt_largest_values(kvc, T, ctx):
    """Values of 2^72 of one sign under logits that rise by up to 2^29 within a reference, and past it."""
    for step in (0.05, 4.0):
        t = Prompt(89, ctx, T, 1, 4, 64, 16, poison=False)
        n = ctx[0] + T[0]
        s = tree_ref.slots(t.bt[0], 16, n)
        t.q[:] = 1.0
        t.scale = 1.0
        t.k[s, 0] = (torch.arange(n, dtype=torch.float32) * (step / 64)).to(torch.bfloat16)[:, None]
        t.v[s] = (t.v[s].abs() + 0.5) * 2.0 ** 71
        go(kvc, t)


def test_prompt_values_not_seen_never_reach_a_row(kvc):
    """Infinite and NaN keys and values of later tokens reach exactly the rows that see them."""
    for D, G, room in ((128, 4, 0), (64, 1, 0), (128, 3, 0), (128, 4, 60), (64, 2, 200)):
        t = Prompt(53 + D, [10, 0], [200, 150], 2, G, D, 16, room=room)
        for r, at, val in ((0, 90, NAN), (0, 150, INF), (1, 40, -INF), (1, 149, NAN)):
            s = tree_ref.slots(t.bt[r], 16, t.ctx[r] + t.T[r])
            t.v[s[t.ctx[r] + at], 1, 5] = val
        s = tree_ref.slots(t.bt[1], 16, 150)
        t.k[s[100], 0, 3] = NAN
        t.gpu().call(kvc)
        assert status(kvc, t.d["status"]) == 0
        o, ls, ob, lb = t.want()
        # in 64 bits a hidden value's weight 0 times NaN is NaN too: per row instead
        for r in range(2):
            c, a = t.ctx[r], int(t.q_off[r])
            for i in (0, 39, 40, 89, 90, 99, 100, 149, 150, 199):
                if i >= t.T[r]:
                    continue
                s = tree_ref.slots(t.bt[r], 16, c + i + 1)
                for h in range(2):
                    k, v = t.k[s, h].double(), t.v[s, h].double()
                    for g in range(h * G, h * G + G):
                        qq = t.q[a + i, g].double()[None]
                        see = torch.ones(1, c + i + 1, dtype=torch.bool)
                        want, ls1, ob1, lb1 = ref._rows(qq, k, v, see, t.scale, ref.UBF)
                        inside(t.d["out"][a + i, g][None], want, ob1, f"row {r} {i} {g}")
                        inside(t.d["lse"][a + i, g][None], ls1, lb1, f"lse {r} {i} {g}")


@pytest.mark.parametrize("n_req", [1, 90])
def test_prompt_infinities_of_no_weight(kvc, n_req):
    """An infinite value of a new row is the result of the rows that see it, also where their weights lie
    elsewhere, whether one CTA takes a request's keys or a cluster."""
    t = Prompt(83, [700] * n_req, [5] * n_req, 2, 2, 64, 16)
    t.q[:] = 1.0
    for r in range(n_req):
        s = tree_ref.slots(t.bt[r], 16, 705)
        t.k[s] = 0.0
        t.k[s[:384]] = 37.5             # logits of 300, all others 0
        t.v[s[702], 1, 5], t.v[s[703], 1, 6] = INF, -INF
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == 0
    o = t.d["out"].float().cpu().view(n_req, 5, 2, 2, 64)
    assert bool((o[:, 2:, 1, :, 5] == INF).all()) and bool((o[:, 3:, 1, :, 6] == -INF).all())
    o[:, 2:, 1, :, 5], o[:, 3:, 1, :, 6] = 0.0, 0.0
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(t.d["lse"]).all())


def test_prompt_bad_pages(kvc):
    for BS, room in ((16, 0), (5, 0), (16, 100)):
        t = Prompt(59, [40, 0, 16], [100, 64, 1], 2, 2, 128, BS, room=room)
        t.bt[0, 1], t.bt[1, 0], t.bt[1, 2] = t.n_slots // BS, -1, 1 << 30
        go(kvc, t, BOUNDS, bad_blocks={t.n_slots // BS, -1, 1 << 30})
    t = Prompt(61, [0], [30], 1, 2, 64, 16)     # nothing to see at all
    t.bt[0, :] = -1
    go(kvc, t, BOUNDS, bad_blocks={-1})
    assert bool((t.d["out"] == 0).all()) and bool((t.d["lse"] == -INF).all())


def test_prompt_bad_requests(kvc):
    def start():
        return Prompt(67, [5, 9, 0], [30, 40, 50], 2, 2, 64, 16).gpu()
    for key, value, live in (("ctx", [5, -1, 0], [*range(30), *range(70, 120)]),
                             ("ctx", [1 << 24, 9, 0], range(30, 120)),
                             ("q_off", [0, 30, 70, 121], range(70)),
                             ("q_off", [-1, 30, 70, 120], range(30, 120)),
                             ("q_off", [0, 30, 29, 120], [])):
        t = start()
        t.d[key] = i32(value)
        t.call(kvc)
        assert status(kvc, t.d["status"]) == BOUNDS
        if len(live):
            t.compare(live=live)
    t = start()
    t.max_rows = 45
    t.call(kvc)
    assert status(kvc, t.d["status"]) == BOUNDS
    t.compare(live=range(70))


def test_prompt_out_off_a_sector(kvc):
    """out on a 16-byte boundary that is no 32-byte one, lse on a 4-byte one."""
    t = Prompt(69, [0, 40], [140, 33], 2, 4, 128, 16).gpu()
    room = torch.full((t.n_q * t.Hq * t.D + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
    t.d["out"] = room[8:].view(t.n_q, t.Hq, t.D)
    t.d["lse"] = torch.full((t.n_q * t.Hq + 1,), 7.0, device=DEV)[1:].view(t.n_q, t.Hq)
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.compare()
    assert bool((room[:8] == 7).all())


def test_calls_from_several_threads(kvc):
    """Calls of different sizes from several host threads on streams of their own."""
    import threading
    jobs = [Prompt(200, [0], [600], 2, 4, 128, 16), Prompt(201, [900], [40], 1, 2, 64, 8),
            Q8(202, [700], [20], [1], 4, 4, 128, 16), Q8(203, [100, 40], [3, 90], [4, 2], 2, 8, 64, 16),
            Rope(204, [5, 0], [40, 9], 2, 4, 128, 16), Prompt(205, [0, 3], [100, 257], 1, 3, 128, 5)]
    want = []
    for t in jobs:
        t.gpu().call(kvc)
        torch.cuda.synchronize()
        want.append([t.d["out"].clone()] + ([t.d["lse"].clone()] if "lse" in t.d else []))
        t.gpu()
    torch.cuda.synchronize()
    failed = []

    def work(t, w):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    t.call(kvc, stream=s)
            s.synchronize()
            got = [t.d["out"]] + ([t.d["lse"]] if "lse" in t.d else [])
            if not all(torch.equal(a, b) for a, b in zip(got, w)):
                failed.append(type(t).__name__)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=x) for x in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_prompt_repeats_replays_and_streams(kvc):
    t = Prompt(71, [0, 33, 5], [260, 100, 3], 2, 4, 128, 16).gpu()
    want = [x.clone() for x in t.call(kvc)]
    for _ in range(3):
        t.gpu()
        torch.cuda.synchronize()
        got = t.call(kvc)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    t.gpu()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t.call(kvc)
    u = Prompt(73, [0, 11], [500, 77], 2, 4, 128, 16).gpu()
    other = [x.clone() for x in u.call(kvc)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):  # a replay on one stream beside calls on another
        g.replay()
        u.call(kvc, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(t.d["out"], want[0]) and torch.equal(t.d["lse"], want[1])
    assert torch.equal(u.d["out"], other[0]) and torch.equal(u.d["lse"], other[1])


# ------------------------------------------------------------------ packing

class Pack:
    def __init__(self, seed, n, L, H, D, BS):
        rng = np.random.default_rng(seed)
        self.n, self.L, self.H, self.D, self.BS = n, L, H, D, BS
        self.n_src, self.n_dst = n + 2, n + 3
        self.src, self.dst = rng.permutation(self.n_src)[:n], rng.permutation(self.n_dst)[:n]
        self.k, self.v = (rows(seed + i, L, self.n_src * BS, H, D) for i in (1, 2))
        # magnitudes of every size from block to block
        for i, p in enumerate((self.k, self.v)):
            e = torch.from_numpy(rng.integers(-20, 20, (L, self.n_src * BS // BS, 1, H, 1)))
            p.view(L, -1, BS, H, D).mul_(torch.exp2(e.float()).bfloat16())

    def gpu(self):
        shape = (self.L, self.n_dst, self.H, self.BS, self.D)
        self.d = dict(k=self.k.to(DEV), v=self.v.to(DEV), src=i32(self.src), dst=i32(self.dst),
                      k8=torch.full(shape, 3, dtype=torch.uint8, device=DEV),
                      v8=torch.full(shape, 3, dtype=torch.uint8, device=DEV),
                      ks=torch.full(shape[:3], 7.0, device=DEV), vs=torch.full(shape[:3], 7.0, device=DEV),
                      status=torch.zeros(1, dtype=torch.int32, device=DEV))
        return self

    def call(self, kvc, stream=None):
        d = self.d
        kvc.kvc_q8_pack(d["k"], d["v"], self.n_src * self.BS, d["k8"], d["v8"], d["ks"], d["vs"], self.n_dst,
                        d["src"], d["dst"], self.n, self.L, self.H, self.D, self.BS, d["status"], stream)

    def check(self, left_out=()):
        go_in = [i for i in range(self.n) if i not in left_out]
        for pool, x8, sc in ((self.k, "k8", "ks"), (self.v, "v8", "vs")):
            y, s = ref.pack(pool, self.src[go_in], self.BS)
            got, gs = self.d[x8].cpu(), self.d[sc].cpu()
            at = self.dst[go_in]
            assert np.array_equal(gs[:, at].numpy().transpose(1, 0, 2), s)
            vals = got[:, at].view(F8).double().numpy().transpose(1, 0, 2, 3, 4)
            assert np.array_equal(vals, y, equal_nan=True)
            rest = np.setdiff1d(np.arange(self.n_dst), at)
            assert bool((got[:, rest] == 3).all()) and bool((gs[:, rest] == 7).all())


@pytest.mark.parametrize("BS", [1, 2, 5, 8, 12, 16, 17, 32, 33, 48, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_pack_sizes(kvc, BS, D):
    t = Pack(BS + D, 7, 2, 3, D, BS).gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


@pytest.mark.parametrize("H", [1, 2, 8, 9, 16, 40])
def test_pack_heads_and_layers(kvc, H):
    t = Pack(H, 3, 5, H, 128, 16).gpu()
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


def test_pack_ties_zeros_and_small_values(kvc):
    """Every e4m3 midpoint, blocks of zeros, largest values on both sides of 448·2^e, subnormals."""
    t = Pack(5, 6, 1, 2, 128, 16)
    codes = torch.arange(127, dtype=torch.uint8).view(F8).float()
    mid = ((codes[:-1] + codes[1:]) / 2)
    for b, f in ((0, 1.0), (1, 2.0 ** -30), (2, 2.0 ** 90)):
        x = t.k.view(1, -1, 16, 2, 128)[0, b, :, 0]
        x.copy_(torch.cat([mid, -mid, codes, -codes, torch.full((2048,), 448.0)])[:2048].view(16, 128).bfloat16() * f)
    blocks = t.k.view(1, -1, 16, 2, 128)[0]
    blocks[3] = 0
    blocks[4] = -0.0
    blocks[4, 0, 1, 0] = 2.0 ** -133            # the least subnormal
    blocks[5] = blocks[5].clamp(-400, 400)
    blocks[5, 3, 0, 7], blocks[5, 3, 1, 7] = 450.0, -3.38e38
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check()


def test_pack_not_finite(kvc):
    t = Pack(6, 3, 1, 2, 64, 16)
    x = t.k.view(1, -1, 16, 2, 64)[0, int(t.src[1])]
    x[2, 0, 5], x[3, 0, 6], x[4, 0, 7], x[:, 1] = INF, -INF, NAN, INF
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == NAN_CODE
    t.check()


def test_pack_left_out_and_bad_pairs(kvc):
    t = Pack(7, 6, 2, 2, 64, 8).gpu()
    src, dst = t.src.copy(), t.dst.copy()
    src[1] = dst[1] = -1
    t.d["src"], t.d["dst"] = i32(src), i32(dst)
    t.call(kvc)
    assert status(kvc, t.d["status"]) == 0
    t.check(left_out={1})
    for bad in ((t.n_src, 0), (-1, 0), (0, t.n_dst), (0, -1)):
        t = Pack(7, 6, 2, 2, 64, 8).gpu()
        src, dst = t.src.copy(), t.dst.copy()
        src[4], dst[4] = (bad[0] if bad[0] else src[4]), (bad[1] if bad[1] else dst[4])
        t.d["src"], t.d["dst"] = i32(src), i32(dst)
        t.call(kvc)
        assert status(kvc, t.d["status"]) == BOUNDS
        t.check(left_out={4})


@pytest.mark.parametrize("spare", [1, 3, 15])
@pytest.mark.parametrize("L", [1, 2, 5])
def test_pack_spare_rows_behind_the_blocks(kvc, L, spare):
    """Pools whose rows make no whole number of blocks: a layer begins n_slots rows after the last."""
    t = Pack(11 + L, 4, L, 3, 64, 16).gpu()
    n = t.n_src * t.BS
    for name in ("k", "v"):
        pool = torch.full((L, n + spare, t.H, t.D), NAN, dtype=torch.bfloat16, device=DEV)
        pool[:, :n] = t.d[name]
        t.d[name] = pool
    d = t.d
    kvc.kvc_q8_pack(d["k"], d["v"], n + spare, d["k8"], d["v8"], d["ks"], d["vs"], t.n_dst, d["src"], d["dst"],
                    t.n, L, t.H, t.D, t.BS, d["status"])
    assert status(kvc, d["status"]) == 0
    t.check()


# ---------------------------------------------------------- 8-bit attention

class Q8(Batch):
    def __init__(self, seed, len8, ctx, T, H, G, D, BS, kind="chain", spread=6, **k):
        super().__init__(seed, ctx, T, H, G, D, BS, **k)
        self.len8 = list(len8)
        self.max_blocks8 = max(1, max(-(-n // BS) for n in len8))
        self.t8, self.n_blocks8 = table(self.rng, self.n_req, self.max_blocks8)
        rs = np.random.RandomState(seed)
        shape = (self.n_blocks8, H, BS, D)
        self.k8, self.v8 = ((torch.randn(shape, generator=torch.Generator().manual_seed(seed + 20 + i)) * 60)
                            .clamp(-448, 448).to(F8) for i in range(2))
        self.ks, self.vs = (torch.from_numpy(np.exp2(rs.randint(-5 - spread, spread - 4, shape[:2])).astype(np.float32))
                            for _ in range(2))
        self.words = (self.max_rows + 31) // 32
        self.mask = None if kind == "chain" else np.concatenate(
            [tree_ref.tree_masks(self.rng, t, self.words, kind) for t in T] + [np.zeros((1, self.words), np.uint32)])
        # what no row sees holds NaN
        held = np.zeros((self.n_blocks8, BS), bool)
        for r in range(self.n_req):
            for p in range(self.len8[r]):
                held[self.t8[r][p // BS], p % BS] = True
        dead = torch.from_numpy(~held)[:, None].expand(-1, H, -1)
        for x in (self.k8, self.v8):
            x.view(torch.uint8)[dead] = 0x7F

    def gpu(self):
        n = max(self.n_q, 1)
        self.d = dict(self.common(), q=self.q.to(DEV), k=self.k.to(DEV), v=self.v.to(DEV),
                      k8=self.k8.view(torch.uint8).to(DEV), v8=self.v8.view(torch.uint8).to(DEV),
                      ks=self.ks.to(DEV), vs=self.vs.to(DEV), t8=i32(self.t8), len8=i32(self.len8),
                      mask=None if self.mask is None else i32(self.mask.view(np.int32)),
                      out=torch.full((n, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV),
                      lse=torch.full((n, self.Hq), 7.0, device=DEV))
        return self

    def call(self, kvc, ws=None, stream=None):
        d = self.d
        if ws is None:
            n = kvc.kvc_q8_attn_workspace_size(self.n_req, self.max_blocks8, self.max_blocks, self.max_rows,
                                               self.H, self.Hq, self.D, self.BS)
            ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        self.ws = ws
        kvc.kvc_q8_attn(d["q"], d["k8"], d["v8"], d["ks"], d["vs"], self.n_blocks8, d["t8"],
                        self.max_blocks8, d["len8"], d["k"], d["v"], self.n_slots, d["bt"], self.max_blocks,
                        d["ctx"], d["q_off"], d["mask"], self.words, self.n_req, max(self.n_q, 1),
                        self.max_rows, self.H, self.Hq, self.D, self.BS, self.scale, d["out"], d["lse"], ws,
                        d["status"], stream)
        return d["out"], d["lse"]

    def compare(self, live=None, **bad):
        o, ls, ob, lb = ref.q8(self.q, self.k8.float(), self.v8.float(), self.ks, self.vs, self.t8, self.len8,
                               self.k, self.v, self.bt, self.BS, self.ctx, self.q_off, self.mask, self.H,
                               self.scale, **bad)
        live = np.arange(int(self.q_off[-1])) if live is None else np.asarray(live, dtype=np.int64)
        dead = np.setdiff1d(np.arange(max(self.n_q, 1)), live)
        out, lse = self.d["out"].cpu(), self.d["lse"].cpu()
        inside(out[live], o[live], ob[live], "out")
        inside(lse[live], ls[live], lb[live], "lse")
        assert bool((out[dead] == 7.0).all()) and bool((lse[dead] == 7.0).all())


L8 = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 200, 300]
C8 = [5, 0, 64, 1, 63, 0, 17, 128, 0, 31, 2, 65, 0]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (8, 4), (3, 6), (1, 3), (2, 16)])
@pytest.mark.parametrize("T", [1, 3])
def test_q8_edges(kvc, D, H, G, T):
    """Histories and bf16 rows on and off every tile edge, either of them empty."""
    go(kvc, Q8(D + H + G + T, L8, C8, [T] * len(L8), H, G, D, 16, pad=1))


@pytest.mark.parametrize("BS", [1, 2, 5, 8, 12, 16, 32, 48, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_q8_page_sizes(kvc, BS, D):
    go(kvc, Q8(BS, [150, 3, 64], [20, 0, 70], [2, 1, 2], 2, 4, D, BS))


@pytest.mark.parametrize("kind", ["tree", "full", "self", "noself", "empty", "holes"])
@pytest.mark.parametrize("T", [5, 40])
def test_q8_masks(kvc, kind, T):
    """Drafted trees behind the history; with no history and no cached row, some rows see nothing."""
    go(kvc, Q8(T, [70, 0, 33], [9, 0, 0], [T, T, T - 2], 2, 4, 128, 16, kind=kind, poison=False))


def test_q8_no_history_at_all_and_empty_requests(kvc):
    go(kvc, Q8(3, [0, 0], [30, 0], [1, 2], 2, 2, 64, 16))
    go(kvc, Q8(4, [50, 20], [0, 4], [0, 2], 2, 2, 64, 16))


@pytest.mark.parametrize("n_req,len8,H,G,D", [(1, 20000, 2, 4, 128), (1, 9000, 8, 1, 64), (3, 4000, 4, 6, 128),
                                              (70, 150, 2, 2, 64)])
def test_q8_long_and_many(kvc, n_req, len8, H, G, D):
    """Units cut into many parts, and units by the hundred."""
    rng = np.random.default_rng(len8)
    n = [len8] + list(rng.integers(len8 // 2, len8, n_req - 1))
    go(kvc, Q8(len8, n, [33] * n_req, [1] * n_req, H, G, D, 16))


@pytest.mark.parametrize("len8", [40, 130, 600, 1500, 5000])
@pytest.mark.parametrize("n_req,H,G,T,D", [(1, 2, 4, 1, 128), (3, 8, 2, 2, 64), (2, 4, 16, 1, 128), (5, 1, 1, 9, 64)])
def test_q8_clusters(kvc, len8, n_req, H, G, T, D):
    """Units that clusters of every size share, some parts without a tile; one row tile and more."""
    n = [len8] + [max(0, len8 - 300 * i) for i in range(1, n_req)]
    go(kvc, Q8(len8 + T, n, [20, 0, 65, 3, 130][:n_req], [T] * n_req, H, G, D, 16, pad=1))


@pytest.mark.parametrize("spread,kscale", [(0, 1.0), (1, 0.0), (3, 30.0), (20, 1e-6), (5, 1e12)])
def test_q8_scales(kvc, spread, kscale):
    """Blocks' scales 2^±spread apart under flat and peaked logits."""
    t = Q8(spread + 5, [300, 77], [40, 3], [2, 1], 2, 3, 128, 16, spread=max(spread, 1), kscale=kscale)
    if spread == 20:  # any positive scales, powers of two or not
        t.ks *= 1.37
        t.vs *= 0.71
    go(kvc, t)


def test_q8_extreme_scales_and_queries(kvc):
    """Scales near the ends of fp32, one block's values 2^60 times another's, queries of 2^±100."""
    t = Q8(21, [64], [5], [1], 1, 4, 64, 16)
    t.ks[:] = 2.0 ** -20
    t.vs[t.t8[0][0]], t.vs[t.t8[0][1]], t.vs[t.t8[0][2]], t.vs[t.t8[0][3]] = 2.0 ** -60, 1.0, 2.0 ** -100, 2.0 ** 20
    # the block of the largest values has all but no weight
    t.ks[t.t8[0][3]] = 0.5
    t.k8.view(torch.uint8)[t.t8[0][3]] = torch.tensor([-448.0]).to(F8).view(torch.uint8)
    t.q[:] = t.q.abs()
    go(kvc, t)
    t = Q8(22, [64], [5], [3], 1, 4, 64, 16)
    t.q[0] *= 2.0 ** 100
    t.q[1] *= 2.0 ** -100
    t.ks *= 2.0 ** -100
    t.k *= 2.0 ** -100
    go(kvc, t)


@pytest.mark.parametrize("T,G", [(1, 4), (4, 2), (5, 6)])
def test_q8_largest_values_of_bf16_rows(kvc, T, G):
    """Values of 2^72 in the cached rows and nodes, whose logits rise past the history's."""
    for step in (0.05, 4.0):
        t = Q8(91, [200], [150], [T], 2, G, 64, 16)
        n = 150 + T
        s = tree_ref.slots(t.bt[0], 16, n)
        t.q[:] = 1.0
        t.scale = 1.0
        t.ks[:] = 2.0 ** -20
        t.k[s] = (torch.arange(n, dtype=torch.float32) * (step / 64)).to(torch.bfloat16)[:, None, None]
        t.v[s] = (t.v[s].abs() + 0.5) * 2.0 ** 71
        go(kvc, t)


@pytest.mark.parametrize("D", [64, 128])
def test_q8_queries_far_below_a_rows_largest(kvc, D):
    """q enters the products exactly from 2^-31 of a row's largest value on, and to within 2^-39 of it
    below: the largest meets keys of 0, so that the logits are the others'."""
    for low, off in ((-31, 0.0), (-34, 2.0 ** -39), (-40, 2.0 ** -39)):
        t = Q8(93, [150], [0], [1], 1, 4, D, 16)
        t.scale = 1.0
        t.q[:] = (torch.rand(t.q.shape, generator=torch.Generator().manual_seed(1)) + 1).bfloat16() * 2.0 ** low
        t.q[..., 0] = 1.0
        t.k8.view(torch.uint8)[..., 0] = 0
        t.ks[:] = 2.0 ** (-low - 10)        # (logits of some units)
        t.k[:] = 0.0
        t.gpu().call(kvc)
        assert status(kvc, t.d["status"]) == 0
        o, ls, ob, lb = ref.q8(t.q, t.k8.float(), t.v8.float(), t.ks, t.vs, t.t8, t.len8, t.k, t.v, t.bt, 16,
                               t.ctx, t.q_off, None, 1, 1.0)
        # a logit's error, and what that makes of weights and values
        blk = torch.from_numpy(t.t8[0])
        k = t.k8.float()[blk].transpose(1, 2).reshape(-1, D)[:150].double()
        v = (t.v8.float()[blk].double() * t.vs[blk].double()[..., None, None]).transpose(1, 2).reshape(-1, D)[:150]
        ez = off * float((k.abs().sum(1) * t.ks[0, 0]).max())
        # (every weight within exp(±2·ez) of its own, and any two means of the values within twice the top)
        top = torch.cat([v.abs(), t.v[tree_ref.slots(t.bt[0], 16, 1)].double()[:, 0].abs()]).amax(0)
        inside(t.d["lse"], ls, lb + ez, "lse")
        inside(t.d["out"], o, ob + min(math.expm1(2 * ez), 2.0) * top, "out")


def test_q8_no_weight_on_far_larger_scales(kvc):
    """A CTA's first tile has the least scale of values, its next one scales 2^146 times as large at
    positions of no weight: they add nothing."""
    t = Q8(37, [160] * 16, [5] * 16, [1] * 16, 32, 1, 64, 16)
    t.q[:] = t.q.abs()
    for r in range(16):
        t.ks[t.t8[r][:8]] = 2.0 ** -20
        t.vs[t.t8[r][:8]] = 2.0 ** -126
        t.ks[t.t8[r][8:]] = 0.5
        t.vs[t.t8[r][8:]] = 2.0 ** 20
        t.k8.view(torch.uint8)[t.t8[r][8:]] = torch.tensor([-448.0]).to(F8).view(torch.uint8)
    go(kvc, t)


@pytest.mark.parametrize("top", [104, 115, 118])
@pytest.mark.parametrize("n_req,len8,H,G,T,D", [(1, 200, 2, 4, 1, 128), (1, 20000, 2, 4, 1, 64), (3, 700, 4, 2, 1, 64),
                                                 (1, 5000, 1, 4, 5, 128), (40, 600, 8, 4, 5, 64), (2, 130, 1, 8, 4, 128)])
def test_q8_values_near_the_end_of_fp32(kvc, n_req, len8, H, G, T, D, top):
    """Blocks of values under scales that kvc_q8_pack makes of bf16's largest: out is finite, however
    many positions and parts add to it."""
    t = Q8(top + len8, [len8 - 3 * r for r in range(n_req)], [3] * n_req, [T] * n_req, H, G, D, 16)
    t.ks[:] = 2.0 ** -7
    t.vs[:] = 2.0 ** top
    t.vs[::5] = 2.0 ** -100
    # (all of one sign, so that sums grow; none past 400·2^118)
    t.v8.copy_(t.v8.float().abs().clamp(max=400).nan_to_num(0).to(F8))
    go(kvc, t)


def test_q8_bad_pages_and_requests(kvc):
    for BS in (16, 5):
        t = Q8(25, [100, 64, 40], [40, 0, 16], [2, 2, 1], 2, 2, 128, BS)
        t.t8[0, 1], t.t8[1, 0], t.t8[2, 2] = t.n_blocks8, -1, 1 << 30
        t.bt[0, 1] = t.n_slots // BS
        go(kvc, t, BOUNDS, bad_blocks={t.n_slots // BS}, bad_blocks8={t.n_blocks8, -1, 1 << 30})
    for key, value, live in (("len8", [100, -1, 40], [0, 1, 4]), ("len8", [1 << 24, 64, 40], [2, 3, 4]),
                             ("ctx", [40, 0, -1], [0, 1, 2, 3]), ("q_off", [0, 2, 4, 9], [0, 1, 2, 3])):
        t = Q8(26, [100, 64, 40], [40, 0, 16], [2, 2, 1], 2, 2, 128, 16).gpu()
        t.d[key] = i32(value)
        t.call(kvc)
        assert status(kvc, t.d["status"]) == BOUNDS
        t.compare(live=live)


def test_q8_values_not_seen_never_reach_a_row(kvc):
    """A node's infinite and NaN values reach the rows that see it; NaN in the history reaches all."""
    t = Q8(27, [50, 30], [7, 3], [4, 4], 1, 2, 64, 16)
    s = tree_ref.slots(t.bt[0], 16, 11)
    t.v[s[9], 0, 3] = INF
    t.v8.view(torch.uint8)[t.t8[1][0], 0, 4, 9] = 0x7F
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == 0
    out = t.d["out"].float().cpu()
    assert bool(torch.isfinite(out[:2]).all()) and bool((out[2:4, :, 3] == INF).all())
    assert bool(torch.isnan(out[4:, :, 9]).all()) and bool(torch.isfinite(out[4:, :, :9]).all())


@pytest.mark.parametrize("n_req,G,len8", [(1, 1, 300), (1, 2, 3000), (1, 8, 900), (200, 1, 300), (40, 8, 300)])
def test_q8_infinities_of_no_weight(kvc, n_req, G, len8):
    """As in the prompt: rows whose weights lie in the history, by single CTAs, clusters and joined parts."""
    t = Q8(85, [len8] * n_req, [5] * n_req, [4] * n_req, 2, G, 64, 16)
    t.q[:] = 1.0
    t.ks[:], t.vs[:] = 1.0, 2.0 ** -6
    t.k8.view(torch.uint8)[:] = torch.tensor([40.0]).to(F8).view(torch.uint8)   # logits of 320
    for r in range(n_req):
        s = tree_ref.slots(t.bt[r], 16, 9)
        t.k[s] = 0.0
        t.v[s[7], 1, 5], t.v[s[8], 1, 6] = INF, -INF
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == 0
    o = t.d["out"].float().cpu().view(n_req, 4, 2, G, 64)
    assert bool((o[:, 2:, 1, :, 5] == INF).all()) and bool((o[:, 3:, 1, :, 6] == -INF).all())
    o[:, 2:, 1, :, 5], o[:, 3:, 1, :, 6] = 0.0, 0.0
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(t.d["lse"]).all())


def test_q8_infinity_before_a_key_that_takes_all_weight(kvc):
    """A node's infinite value, and a later node whose logit raises the reference past it."""
    t = Q8(87, [40], [0], [200], 1, 1, 64, 16)
    s = tree_ref.slots(t.bt[0], 16, 200)
    t.q[:] = 1.0
    t.ks[:], t.vs[:] = 2.0 ** -20, 2.0 ** -6
    t.k[s] = 0.0
    t.k[s[130]] = 37.5
    t.v[s[2], 0, 5] = INF
    t.gpu().call(kvc)
    assert status(kvc, t.d["status"]) == 0
    o = t.d["out"].float().cpu()
    assert bool((o[2:, 0, 5] == INF).all())
    o[2:, 0, 5] = 0.0
    assert bool(torch.isfinite(o).all())


def test_q8_repeats_replays_and_streams(kvc):
    t = Q8(29, [700, 33], [20, 90], [1, 2], 4, 4, 128, 16).gpu()
    want = [x.clone() for x in t.call(kvc)]
    ws = t.ws
    g = torch.cuda.CUDAGraph()
    t.gpu()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t.call(kvc, ws)
    for _ in range(3):
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.d["out"], want[0]) and torch.equal(t.d["lse"], want[1])
    u = Q8(31, [500], [9], [1], 4, 4, 128, 16).gpu()
    other = [x.clone() for x in u.call(kvc)]
    own_ws, side = u.ws, torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        g.replay()
        u.call(kvc, own_ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(t.d["out"], want[0]) and torch.equal(u.d["out"], other[0])


# ------------------------------------------------------------ a run of them

def test_prompt_pack_and_decode(kvc):
    """A prompt enters the cache, its rows attend, its full blocks move to 8 bits, and the next token
    attends to history and rest: each step against the 64-bit form of what the last one left."""
    H, G, D, BS, T = 2, 4, 128, 16, [100, 61]
    r = Rope(97, [0, 0], T, H, G, D, BS, pad=0).gpu()
    r.call(kvc)
    assert status(kvc, r.d["status"]) == 0
    r.check()
    p = Prompt(97, [0, 0], T, H, G, D, BS)
    p.q, p.k, p.v, p.bt, p.n_slots = (r.d["out"].cpu(), r.d["k"].cpu(), r.d["v"].cpu(), r.bt, r.n_slots)
    p.max_blocks = r.max_blocks
    go(kvc, p)
    full = [t // BS for t in T]
    src = np.concatenate([r.bt[i, :n] for i, n in enumerate(full)])
    k = Pack(1, len(src), 1, H, D, BS)
    k.k, k.v, k.src, k.n_src = r.d["k"].cpu()[None], r.d["v"].cpu()[None], src, r.n_slots // BS
    k.gpu().call(kvc)
    assert status(kvc, k.d["status"]) == 0
    k.check()
    # the next token: its key and value behind the rows that stayed in bf16
    a = Q8(98, [n * BS for n in full], [t - n * BS for t, n in zip(T, full)], [1, 1], H, G, D, BS)
    a.t8 = np.zeros((2, a.max_blocks8), np.int64)
    a.t8[0, :full[0]], a.t8[1, :full[1]] = k.dst[:full[0]], k.dst[full[0]:]
    a.k8, a.v8 = k.d["k8"][0].cpu().view(F8), k.d["v8"][0].cpu().view(F8)
    a.ks, a.vs, a.n_blocks8 = k.d["ks"][0].cpu(), k.d["vs"][0].cpu(), k.n_dst
    a.bt = np.stack([r.bt[i, n:n + 1] for i, n in enumerate(full)])
    a.k, a.v, a.n_slots, a.max_blocks = r.d["k"].cpu(), r.d["v"].cpu(), r.n_slots, 1
    for i in range(2):
        at = tree_ref.slots(a.bt[i], BS, a.ctx[i] + 1)[-1]
        a.k[at], a.v[at] = rows(i, H, D), rows(i + 5, H, D)
    go(kvc, a)
