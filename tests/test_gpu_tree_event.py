"""Decoding steps with drafted trees through TreeDecodeEvent, against the 64-bit forms of each
operator (tests/tree_ref.py): the cache, weights and positions carried from step to step, a cache that
starts above its budget and one that starts empty, plain decoding, a captured step."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import tree_ref as ref  # noqa: E402

DEV = "cuda"


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def rows(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16).numpy()


def same(got, want, what):
    bad = int((got != want).sum())
    assert bad == 0, f"{what}: {bad} of {want.size} differ"


def inside(got, want, bound, what):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    over = ((got - want).abs() / bound.clamp(min=1e-300))[~inf]
    assert over.numel() == 0 or float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g}"


class Serving:
    """A few requests on one pool, host copies beside the device's."""

    def __init__(self, seed, ctx, nodes, L=2, H=2, G=2, D=64, BS=8, budget=40, n_sink=2, n_recent=4,
                 observe=0, decay=1.0):
        from query_conditioned_kv_gb300.event import TreeDecodeEvent
        self.rng, self.g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.ctx0, self.T, self.n_req = np.array(ctx), nodes, len(ctx)
        self.L, self.H, self.Hq, self.D, self.BS = L, H, H * G, D, BS
        self.n_q = self.n_req * nodes
        self.max_blocks = -(-(max(max(ctx), budget) + nodes) // BS)
        n_blocks = self.n_req * self.max_blocks + 2
        self.bt = self.rng.permutation(n_blocks)[:-2].reshape(self.n_req, self.max_blocks)
        self.n_slots = n_blocks * BS
        self.k, self.v = rows(self.g, L, self.n_slots, H, D), rows(self.g, L, self.n_slots, H, D)
        self.kd, self.vd, self.btd = self.k.to(DEV), self.v.to(DEV), i32(self.bt)
        self.ev = TreeDecodeEvent(self.n_req, self.max_blocks, BS, L, H, self.Hq, D, self.n_slots,
                                  self.n_q, nodes, budget, n_sink, n_recent,
                                  max_path=min(nodes, 4), max_observe=observe, decay=decay)
        self.ev.start(i32(ctx))
        self.words = (nodes + 31) // 32
        self.q_off = i32(np.arange(self.n_req + 1) * nodes)

    def draw(self):
        """A step's inputs: queries, the nodes' rows, the trees, the accepted paths."""
        s = {"q": rows(self.g, self.L, self.n_q, self.Hq, self.D),
             "nk": rows(self.g, self.L, self.n_req, self.T, self.H, self.D),
             "nv": rows(self.g, self.L, self.n_req, self.T, self.H, self.D),
             "mask": np.concatenate([ref.tree_masks(self.rng, self.T, self.words, "tree")
                                     for _ in range(self.n_req)])}
        m = self.rng.integers(0, self.ev.max_path + 1, self.n_req)
        m[0] = self.ev.max_path
        s["path"] = np.zeros((self.n_req, self.ev.max_path), np.int64)
        for r in range(self.n_req):
            s["path"][r, :m[r]] = np.sort(self.rng.permutation(self.T)[:m[r]])
        s["m"] = m
        return s

    def write_nodes(self, s):
        """What the model does before attention: the nodes' rows, behind the cache."""
        ctx = self.ev.ctx.cpu().numpy()
        for r in range(self.n_req):
            p = ctx[r] + np.arange(self.T)
            at = torch.from_numpy(self.bt[r][p // self.BS] * self.BS + p % self.BS)
            self.k[:, at], self.v[:, at] = s["nk"][:, r], s["nv"][:, r]
            self.kd[:, at.to(DEV)], self.vd[:, at.to(DEV)] = s["nk"][:, r].to(DEV), s["nv"][:, r].to(DEV)
        return ctx

    def step(self, s, stream=None):
        q = s["q"].to(DEV) if isinstance(s["q"], torch.Tensor) and not s["q"].is_cuda else s["q"]
        mask = s["mask_d"] if "mask_d" in s else i32(s["mask"].view(np.int32))
        path = s["path_d"] if "path_d" in s else i32(s["path"])
        m = s["m_d"] if "m_d" in s else i32(s["m"])
        for layer in range(self.L):
            self.ev.attend(layer, q[layer], self.kd[layer], self.vd[layer], self.btd, self.q_off,
                           None if self.T == 1 else mask, stream)
        self.ev.finish(q, self.kd, self.vd, self.btd, self.q_off, path, m, stream)

    def checked_step(self):
        import query_conditioned_kv_gb300 as kvc
        s, ev = self.draw(), self.ev
        ctx = self.write_nodes(s)
        old_mass, old_pos = ev.mass.cpu().clone(), ev.pos.cpu().clone()
        old_end = ev.t_end.cpu().numpy().copy()
        n_mass, n_pos = ev.n_mass.cpu().numpy().copy(), ev.n_pos.cpu().numpy().copy()
        # the same calls one by one, to see the state between them
        q, mask, path, m = s["q"].to(DEV), i32(s["mask"].view(np.int32)), i32(s["path"]), i32(s["m"])
        for layer in range(self.L):
            ev.attend(layer, q[layer], self.kd[layer], self.vd[layer], self.btd, self.q_off,
                      None if self.T == 1 else mask)
            o, ls, ob, lb = ref.attn(s["q"][layer], self.k[layer], self.v[layer], self.bt, self.BS, ctx,
                                     np.arange(self.n_req + 1) * self.T,
                                     None if self.T == 1 else s["mask"], self.H, ev.scale)
            inside(ev.out[layer], o, ob, "out")
            inside(ev.lse[layer], ls, lb, "lse")
        ev.commit(self.kd, self.vd, self.btd, self.q_off, path, m)
        for r in range(self.n_req):
            for i in range(s["m"][r]):
                a, b = ctx[r] + s["path"][r, i], ctx[r] + i
                sa = self.bt[r][a // self.BS] * self.BS + a % self.BS
                sb = self.bt[r][b // self.BS] * self.BS + b % self.BS
                self.k[:, sb], self.v[:, sb] = self.k[:, sa].clone(), self.v[:, sa].clone()
        seq = ctx + s["m"]
        same(ev.seq.cpu().numpy(), seq, "lengths")
        same(bits(self.kd.cpu()), bits(self.k), "K after the commit")
        same(bits(self.vd.cpu()), bits(self.v), "V after the commit")
        ev.accumulate(q, self.kd, self.btd)
        on = np.arange(ev.max_path)[None] < s["m"][:, None]
        idx = np.where(on, np.arange(self.n_req)[:, None] * self.T + s["path"], 0)
        vis = np.where(on, ctx[:, None] + np.arange(ev.max_path)[None] + 1, 0)
        want, bound = ref.mass(s["q"], ev.lse.cpu(), idx.reshape(-1), vis.reshape(-1),
                               np.arange(self.n_req + 1) * ev.max_path, self.k, self.bt, self.BS, seq,
                               n_mass, old_mass, self.H, ev.scale, ev.decay)
        inside(ev.mass, want, bound, "mass")
        mass = ev.mass.cpu().numpy()
        ev.t_end.add_(ev.seq).sub_(ev.ctx)
        ev.evict(self.kd, self.vd, self.btd)
        kn, vn, mo, po, n_out = ref.evict(bits(self.k), bits(self.v), self.bt, self.BS, seq, n_pos,
                                          old_end + s["m"], mass, old_pos.numpy(), self.H, ev.budget,
                                          ev.n_sink, ev.n_recent)
        same(bits(self.kd.cpu()), kn, "K after the eviction")
        same(bits(self.vd.cpu()), vn, "V after the eviction")
        self.k = torch.from_numpy(kn).view(torch.bfloat16).reshape(self.k.shape)
        self.v = torch.from_numpy(vn).view(torch.bfloat16).reshape(self.v.shape)
        same(ev.n_out.cpu().numpy(), n_out, "rows left")
        for r in range(self.n_req):
            n = n_out[r]
            same(ev.mass.cpu().numpy()[:, r, :, :n], mo[:, r, :, :n], "weights")
            same(ev.pos.cpu().numpy()[:, r, :, :n], po[:, r, :, :n], "positions")
        for x in (ev.ctx, ev.n_mass, ev.n_pos):
            x.copy_(ev.n_out)
        assert kvc.kvc_device_status(ev.dev_status) == 0

    def state(self):
        ev = self.ev
        return [t.clone() for t in (self.kd, self.vd, ev.out, ev.lse, ev.mass, ev.pos, ev.ctx,
                                    ev.t_end, ev.n_mass, ev.n_pos)]


@pytest.mark.parametrize("nodes,kw", [
    (13, dict()),                                       # one request over its budget, one empty
    (40, dict(G=4, D=128, BS=16, decay=0.9)),           # wide row sets, decayed weights
    (1, dict(H=3, G=1, n_recent=0)),                    # plain decoding
])
def test_steps_carry_the_cache(nodes, kw):
    sv = Serving(11 + nodes, [61, 0, 38], nodes, **kw)
    for _ in range(4):
        sv.checked_step()
    assert int(sv.ev.ctx.max()) <= sv.ev.budget


def test_finish_is_its_parts():
    a, b = Serving(5, [50, 7], 9), Serving(5, [50, 7], 9)
    for _ in range(3):
        a.checked_step()
        s = b.draw()
        b.write_nodes(s)
        b.step(s)
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


def test_observed_window_decides_the_first_eviction():
    """The prompt's last queries put all their weight on the first rows: those stay."""
    sv = Serving(3, [64, 64], 5, observe=8, n_sink=0, n_recent=8)
    ev, L, H, Hq, D = sv.ev, sv.L, sv.H, sv.Hq, sv.D
    q = torch.zeros(L, 16, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = 8.0
    for r in range(2):
        p = np.arange(64)
        at = torch.from_numpy(sv.bt[r][p // sv.BS] * sv.BS + p % sv.BS)
        sv.k[:, at, :, 0] = torch.where(torch.arange(64) < 30, 4.0, -4.0).to(torch.bfloat16)[None, :, None]
    sv.kd.copy_(sv.k)
    vis = np.concatenate([57 + np.arange(8)] * 2)
    lse = torch.full((L, 16, Hq), 7.5, device=DEV)
    ev.observe(q.to(DEV), lse, i32(vis), i32([0, 8, 16]), sv.kd, sv.btd)
    want, bound = ref.mass(q, lse.cpu(), None, vis, [0, 8, 16], sv.k, sv.bt, sv.BS, [64, 64], [0, 0],
                           torch.zeros(ev.mass.shape), H, ev.scale, 1.0)
    inside(ev.mass[..., :64], want[..., :64], bound[..., :64], "mass")
    sv.checked_step()
    kept = ev.pos.cpu().numpy()[:, :, :, :ev.budget]
    assert all(set(range(30)) <= set(kept[i, r, h]) for i in range(L) for r in range(2) for h in range(H))


def test_a_captured_step_replays():
    eager, graph = Serving(21, [45, 33], 17), Serving(21, [45, 33], 17)
    side = torch.cuda.Stream()
    s0 = graph.draw()
    fixed = {"q": s0["q"].to(DEV), "mask_d": i32(s0["mask"].view(np.int32)), "path_d": i32(s0["path"]),
             "m_d": i32(s0["m"])}
    before = graph.state()
    with torch.cuda.stream(side):
        graph.step(fixed)                 # (loads the kernels)
    side.synchronize()
    ev = graph.ev
    for x, y in zip((graph.kd, graph.vd, ev.out, ev.lse, ev.mass, ev.pos, ev.ctx, ev.t_end, ev.n_mass,
                     ev.n_pos), before):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        graph.step(fixed)
    s = eager.draw()
    for i in range(3):
        s = s if i == 0 else eager.draw()
        eager.write_nodes(s)
        eager.step(s)
        graph.write_nodes(s)
        fixed["q"].copy_(s["q"])
        for name, src in (("mask_d", s["mask"].view(np.int32)), ("path_d", s["path"]), ("m_d", s["m"])):
            fixed[name].copy_(i32(src))
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager.state(), graph.state()):
            assert torch.equal(x, y)
