"""Prompts and decoding through HistoryEvent, whose older blocks move to 8 bits, against the 64-bit
forms of each operator (tests/prefill_ref.py): what every token's rows are wherever they lie, lengths
and tables carried from step to step, a captured step, another stream."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import prefill_ref as ref  # noqa: E402
import tree_ref  # noqa: E402

DEV = "cuda"
F8 = torch.float8_e4m3fn
EPS = 1e-6


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def inside(got, want, bound, what):
    over = (got.double().cpu() - want).abs() / bound.clamp(min=1e-300)
    assert over.numel() == 0 or float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the bound"


class Serving:
    def __init__(self, seed, n_req=3, L=2, H=2, G=3, D=64, BS=8, recent=11, n_q=70, max_rows=40,
                 max_blocks=9, max_move=None):
        from query_conditioned_kv_gb300.event import HistoryEvent
        rng, self.g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.n_req, self.L, self.H, self.G, self.D, self.BS, self.recent = n_req, L, H, G, D, BS, recent
        self.Hq, self.n_q, self.max_blocks, self.mb8 = H * G, n_q, max_blocks, 12
        nb, nb8 = n_req * max_blocks + 1, n_req * self.mb8 + 2
        self.bt0 = rng.permutation(nb)[:n_req * max_blocks].reshape(n_req, max_blocks)
        self.t8 = rng.permutation(nb8)[:n_req * self.mb8].reshape(n_req, self.mb8)
        self.n_slots, self.nb8 = nb * BS, nb8
        self.bt, self.t8d = i32(self.bt0), i32(self.t8)
        self.k, self.v = (torch.zeros(L, self.n_slots, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.k8, self.v8 = (torch.zeros(L, nb8, H, BS, D, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.ks, self.vs = (torch.ones(L, nb8, H, device=DEV) for _ in range(2))
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=self.g)).bfloat16().to(DEV) for _ in range(2))
        self.ev = HistoryEvent(n_req, max_blocks, self.mb8, BS, L, H, self.Hq, D, self.n_slots, nb8, n_q,
                               max_rows, n_pos=200, recent=recent, max_move=max_move, eps=EPS)
        self.rows = [[[], []] for _ in range(n_req)]      # per request: every token's K and V [L][H][D]
        self.ctx, self.len8 = np.zeros(n_req, int), np.zeros(n_req, int)

    def inputs(self, T):
        q_off = np.concatenate([[0], np.cumsum(T)])
        x = torch.randn(self.L, self.n_q, (self.Hq + 2 * self.H) * self.D, generator=self.g).bfloat16()
        return q_off, x

    def parts(self, x):
        a, b = self.Hq * self.D, (self.Hq + self.H) * self.D
        return x[:, :a], x[:, a:b], x[:, b:]

    def launch(self, q_off_d, xd, prompt, stream=None):
        self.ev.begin(q_off_d, stream=stream)
        for l in range(self.L):
            self.ev.write(l, *self.parts(xd[l]), self.k[l], self.v[l], self.bt, self.wq, self.wk, stream=stream)
            if prompt:
                self.ev.prompt(l, self.k[l], self.v[l], self.bt, stream=stream)
            else:
                self.ev.attend(l, self.k[l], self.v[l], self.bt, self.k8[l], self.v8[l], self.ks[l],
                               self.vs[l], self.t8d, stream=stream)

    def finish(self, stream=None):
        self.ev.finish(self.k, self.v, self.bt, self.k8, self.v8, self.ks, self.vs, self.t8d, stream=stream)

    def step(self, T, prompt=False, stream=None):
        q_off, x = self.inputs(T)
        qd, xd = i32(q_off), x.to(DEV)
        torch.cuda.synchronize()
        self.launch(qd, xd, prompt, stream)
        torch.cuda.synchronize()
        self.check_rows(T, q_off, x)
        self.check_attention(T, q_off)
        self.finish(stream)
        torch.cuda.synchronize()
        import query_conditioned_kv_gb300 as kvc
        assert kvc.kvc_device_status(self.ev.dev_status) == 0
        for r in range(self.n_req):
            self.ctx[r] += T[r]
            move = min(max(0, self.ctx[r] - self.recent) // self.BS, self.ev.max_move, self.mb8 - self.len8[r] // self.BS)
            self.ctx[r] -= move * self.BS
            self.len8[r] += move * self.BS
        assert self.ev.ctx.tolist() == list(self.ctx) and self.ev.len8.tolist() == list(self.len8)
        assert self.ev.t_end.tolist() == [len(r[0]) for r in self.rows]
        self.check_residence()

    def check_rows(self, T, q_off, x):
        """What the step stored, and each new token's rows into the record."""
        tab, bt = ref.rope_table(200, self.D), self.bt.cpu().numpy()
        for l in range(self.L):
            q, k, v = (p.reshape(self.n_q, -1, self.D) for p in self.parts(x[l]))
            for r in range(self.n_req):
                a, b, seen = q_off[r], q_off[r + 1], len(self.rows[r][0]) if l == 0 else self.seen[r]
                if l == 0:
                    self.seen = getattr(self, "seen", {})
                    self.seen[r] = seen
                pos = seen + np.arange(b - a)
                y, rel = ref.normed(q[a:b], self.wq.cpu(), EPS)
                want, bound = ref.rotated(y, rel, tab[pos])
                inside(self.ev.q[l, a:b], want, bound, "queries")
                at = tree_ref.slots(bt[r], self.BS, self.ctx[r] + b - a)[self.ctx[r]:]
                y, rel = ref.normed(k[a:b], self.wk.cpu(), EPS)
                want, bound = ref.rotated(y, rel, tab[pos])
                got = self.k[l].cpu()[at]
                inside(got, want, bound, "keys")
                assert torch.equal(self.v[l].cpu()[at], v[a:b])
                for i in range(b - a):
                    if l == 0:
                        for kind in (0, 1):
                            self.rows[r][kind].append(torch.zeros(self.L, self.H, self.D, dtype=torch.bfloat16))
                    self.rows[r][0][seen + i][l], self.rows[r][1][seen + i][l] = got[i], v[a + i]

    def check_attention(self, T, q_off):
        bt = self.bt.cpu().numpy()
        for l in range(self.L):
            o, ls, ob, lb = ref.q8(self.ev.q[l].cpu(), self.k8[l].cpu().view(F8).float(),
                                   self.v8[l].cpu().view(F8).float(), self.ks[l].cpu(), self.vs[l].cpu(),
                                   self.t8, self.len8, self.k[l].cpu(), self.v[l].cpu(), bt, self.BS, self.ctx,
                                   q_off, None, self.H, self.ev.scale)
            n = int(q_off[-1])
            inside(self.ev.out[l, :n], o[:n], ob[:n], "out")
            inside(self.ev.lse[l, :n], ls[:n], lb[:n], "lse")

    def check_residence(self):
        """Every token's rows, wherever they lie now: exact in bf16, within half a step in 8 bits."""
        bt = self.bt.cpu().numpy()
        pools = [[(self.k8, self.ks, self.k), (self.v8, self.vs, self.v)][i] for i in (0, 1)]
        for r in range(self.n_req):
            assert sorted(bt[r]) == sorted(self.bt0[r])
            assert len(self.rows[r][0]) == self.len8[r] + self.ctx[r]
            for kind, (x8, sc, x16) in enumerate(pools):
                x8, sc, x16 = x8.cpu().view(F8).double(), sc.cpu().double(), x16.cpu()
                for t, want in enumerate(self.rows[r][kind]):
                    if t < self.len8[r]:
                        b, o = self.t8[r][t // self.BS], t % self.BS
                        got = x8[:, b, :, o] * sc[:, b, :, None]
                        bound = 2.0 ** -4 * want.double().abs() + 2.0 ** -10 * sc[:, b, :, None]
                        assert bool(((got - want.double()).abs() <= bound).all())
                    else:
                        p = t - self.len8[r]
                        assert torch.equal(x16[:, bt[r][p // self.BS] * self.BS + p % self.BS], want)


@pytest.mark.parametrize("D,BS,recent", [(64, 8, 11), (128, 16, 0), (128, 5, 3)])
def test_prompt_then_decoding(D, BS, recent):
    s = Serving(D + BS, D=D, BS=BS, recent=recent, max_blocks=-(-64 // BS))
    s.step([37, 0, 19], prompt=True)
    for T in ([1, 1, 1], [1, 3, 0], [2, 1, 1], [1, 9, 4], [1, 1, 1], [0, 0, 1], [4, 4, 4], [1, 1, 1]):
        s.step(T)


def test_moves_are_spread_over_steps():
    """At most max_move blocks of a request a step; the others follow."""
    s = Serving(3, recent=0, max_move=1)
    s.step([40, 17, 8], prompt=True)
    for _ in range(5):
        s.step([1, 1, 0])


def test_history_full():
    """With table8 full the rows stay in bf16."""
    s = Serving(4, recent=0)
    s.mb8 = s.ev.max_blocks8 = 2
    s.t8, s.t8d = s.t8[:, :2].copy(), s.t8d[:, :2].contiguous()
    s.step([30, 25, 8], prompt=True)
    for _ in range(3):
        s.step([3, 1, 1])


@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(raw):
    side = torch.cuda.Stream()
    s = Serving(5)
    s.step([20, 33, 1], prompt=True, stream=side.cuda_stream if raw else side)
    for _ in range(3):
        s.step([1, 2, 1], stream=side.cuda_stream if raw else side)


def test_captured_step_repeats():
    """A decoding step captured once and replayed gives the eager steps' bits, as lengths grow and
    blocks move."""
    T = [1, 1, 1]
    a, b = Serving(6), Serving(6)
    for s in (a, b):
        s.step([23, 16, 9], prompt=True)
    steps = [a.inputs(T) for _ in range(12)]
    qd = i32(steps[0][0])
    xd = torch.empty_like(steps[0][1], device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.launch(qd, xd, False)
        b.finish()
    for _, x in steps:
        a.launch(qd, x.to(DEV), False)
        a.finish()
        xd.copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.ev.out[:, :3], b.ev.out[:, :3]) and torch.equal(a.ev.lse[:, :3], b.ev.lse[:, :3])
        for n in ("ctx", "len8", "t_end"):
            assert torch.equal(getattr(a.ev, n), getattr(b.ev, n))
    assert torch.equal(a.k8, b.k8) and torch.equal(a.ks, b.ks) and torch.equal(a.bt, b.bt)
    assert int(a.ev.len8.sum()) > 0


def test_pools_with_spare_rows():
    """A step on pools with a few rows behind the last whole block: every layer's blocks move."""
    s = Serving(8, recent=0)
    s.n_slots += 3
    s.ev.n_slots = s.n_slots
    s.k, s.v = (torch.zeros(s.L, s.n_slots, s.H, s.D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    s.step([30, 25, 8], prompt=True)
    for _ in range(2):
        s.step([3, 1, 1])


def drafted(rng, T):
    """A tree of T nodes (parents before children, -1: a root) and one accepted path of it."""
    parent = [int(rng.integers(-1 if i % 3 == 0 else max(0, i - 3), i)) if i else -1 for i in range(T)]
    chain = lambda i: [] if i < 0 else chain(parent[i]) + [i]  # noqa: E731
    lines = [chain(i) for i in range(T)]
    return lines, (lines[int(rng.integers(0, T))] if T else [])


def draft_step(s, rng, T, tree=True):
    """Drafted nodes through begin(pos), attend(tree_mask), kvc_tree_commit and finish(n_rows): rotations,
    rows and attention of the step, the accepted rows' places after it.  Not a tree: a chain of which the
    first few are accepted."""
    import query_conditioned_kv_gb300 as kvc
    q_off, x = s.inputs(T)
    trees = [drafted(rng, t) for t in T]
    if not tree:
        trees = [([list(range(i + 1)) for i in range(t)], list(range(int(rng.integers(0, t + 1))))) for t in T]
    words = (s.ev.max_rows + 31) // 32
    mask = np.zeros((s.n_q, words), np.uint32)
    depth = np.zeros(s.n_q, int)
    for r, (lines, _) in enumerate(trees):
        for i, line in enumerate(lines):
            depth[q_off[r] + i] = len(line) - 1
            for j in line:
                mask[q_off[r] + i, j // 32] |= np.uint32(1 << (j % 32))
    qd, xd, path = i32(q_off), x.to(DEV), np.zeros((s.n_req, 8), int)
    n_path = [min(len(p), 8) for _, p in trees]
    for r, (_, p) in enumerate(trees):
        path[r, :n_path[r]] = p[:n_path[r]]
    s.ev.begin(qd, pos=i32(depth))
    for l in range(s.L):
        s.ev.write(l, *s.parts(xd[l]), s.k[l], s.v[l], s.bt, s.wq, s.wk)
        s.ev.attend(l, s.k[l], s.v[l], s.bt, s.k8[l], s.v8[l], s.ks[l], s.vs[l], s.t8d,
                    tree_mask=i32(mask.view(np.int32)) if tree else None)
    torch.cuda.synchronize()
    tab, bt = ref.rope_table(200, s.D), s.bt.cpu().numpy()
    seen = [len(s.rows[r][0]) for r in range(s.n_req)]
    took = [[[torch.zeros(s.L, s.H, s.D, dtype=torch.bfloat16) for _ in range(n)] for n in n_path] for _ in (0, 1)]
    for l in range(s.L):
        q, k, v = (p.reshape(s.n_q, -1, s.D) for p in s.parts(x[l]))
        for r in range(s.n_req):
            a, b = q_off[r], q_off[r + 1]
            at = tree_ref.slots(bt[r], s.BS, s.ctx[r] + b - a)[s.ctx[r]:]
            for y, w, got in ((q, s.wq, s.ev.q[l, a:b]), (k, s.wk, s.k[l].cpu()[at])):
                y, rel = ref.normed(y[a:b], w.cpu(), EPS)
                inside(got, *ref.rotated(y, rel, tab[seen[r] + depth[a:b]]), "rotated rows")
            assert torch.equal(s.v[l].cpu()[at], v[a:b])
            for i, j in enumerate(path[r, :n_path[r]]):
                took[0][r][i][l], took[1][r][i][l] = s.k[l].cpu()[at[j]], v[a + j]
        o, ls, ob, lb = ref.q8(s.ev.q[l].cpu(), s.k8[l].cpu().view(F8).float(), s.v8[l].cpu().view(F8).float(),
                               s.ks[l].cpu(), s.vs[l].cpu(), s.t8, s.len8, s.k[l].cpu(), s.v[l].cpu(), bt, s.BS,
                               s.ctx, q_off, mask, s.H, s.ev.scale)
        n = int(q_off[-1])
        inside(s.ev.out[l, :n], o[:n], ob[:n], "out")
        inside(s.ev.lse[l, :n], ls[:n], lb[:n], "lse")
    if tree:
        kvc.kvc_tree_commit(s.k, s.v, s.n_slots, s.bt, s.max_blocks, s.ev.ctx, qd, i32(path), i32(n_path), 8,
                            s.n_req, s.L, s.H, s.D, s.BS, torch.zeros(s.n_req, dtype=torch.int32, device=DEV),
                            None, None, s.ev.dev_status)
    s.ev.finish(s.k, s.v, s.bt, s.k8, s.v8, s.ks, s.vs, s.t8d, n_rows=i32(n_path))
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 0
    for r in range(s.n_req):
        for kind in (0, 1):
            s.rows[r][kind] += took[kind][r]
        s.ctx[r] += n_path[r]
        move = min(max(0, s.ctx[r] - s.recent) // s.BS, s.ev.max_move, s.mb8 - s.len8[r] // s.BS)
        s.ctx[r] -= move * s.BS
        s.len8[r] += move * s.BS
    assert s.ev.ctx.tolist() == list(s.ctx) and s.ev.len8.tolist() == list(s.len8)
    assert s.ev.t_end.tolist() == [len(r[0]) for r in s.rows]
    s.check_residence()


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("D,BS", [(64, 8), (128, 16)])
def test_drafted_steps(tree, D, BS):
    """Drafted trees, or chains of which a part is accepted, over history and cache, and plain steps
    after them: every node's rotation is that of its depth behind the tokens seen."""
    s, rng = Serving(9 + D, D=D, BS=BS, recent=3, max_blocks=-(-88 // BS)), np.random.default_rng(D + tree)
    s.step([37, 0, 19], prompt=True)
    for T in ([7, 3, 12], [1, 9, 0], [20, 5, 4]):
        draft_step(s, rng, T, tree)
        s.step([1, 2, 1])
    assert int(s.ev.len8.max()) > 0


def test_steps_of_their_own_sizes():
    """One event for prompts and for single tokens: a step's buffers and launches go by the sizes that
    begin is given, and give what the largest ones give."""
    a, b = (Serving(10, n_q=70, max_rows=40) for _ in range(2))
    for s in (a, b):
        s.step([37, 0, 19], prompt=True)
    for T in ([1, 1, 1], [2, 0, 1], [1, 1, 1], [4, 4, 4], [1, 1, 1], [0, 1, 0]):
        n, most = sum(T), max(T)
        q_off, x = a.inputs(T)
        qd, xd = i32(q_off), x[:, :n].contiguous().to(DEV)
        a.ev.begin(qd, n_q=n, max_rows=most)
        for l in range(a.L):
            a.ev.write(l, *a.parts(xd[l]), a.k[l], a.v[l], a.bt, a.wq, a.wk)
            got = a.ev.attend(l, a.k[l], a.v[l], a.bt, a.k8[l], a.v8[l], a.ks[l], a.vs[l], a.t8d)
            assert got.shape == (n, a.Hq, a.D) and got.data_ptr() == a.ev.out[l].data_ptr()
        torch.cuda.synchronize()
        a.check_rows(T, q_off, x)
        a.check_attention(T, q_off)
        a.finish()
        b.launch(qd, x.to(DEV), False)
        b.finish()
        torch.cuda.synchronize()
        import query_conditioned_kv_gb300 as kvc
        for s in (a, b):
            assert kvc.kvc_device_status(s.ev.dev_status) == 0
        a.ctx, a.len8 = a.ev.ctx.cpu().numpy(), a.ev.len8.cpu().numpy()
        a.check_residence()
        for name in ("ctx", "len8", "t_end"):
            assert torch.equal(getattr(a.ev, name), getattr(b.ev, name))
    # a prompt of a few rows again, in an event that has taken steps of other sizes
    s = Serving(11)
    s.step([20, 33, 1], prompt=True)
    q_off, x = s.inputs([0, 0, 5])
    s.ev.begin(i32(q_off), n_q=5, max_rows=5)
    for l in range(s.L):
        s.ev.write(l, *s.parts(x[l, :5].to(DEV)), s.k[l], s.v[l], s.bt, s.wq, s.wk)
        s.ev.prompt(l, s.k[l], s.v[l], s.bt)
    torch.cuda.synchronize()
    s.check_rows([0, 0, 5], q_off, x)
    s.check_attention([0, 0, 5], q_off)
    s.finish()
    assert s.ev.t_end.tolist() == [20, 33, 6]


def test_steps_past_the_largest_are_refused():
    import query_conditioned_kv_gb300 as kvc
    s = Serving(12)
    q_off = i32([0, 2, 3, 4])
    for n, most in ((71, 3), (0, 3), (4, 41), (4, 0)):
        with pytest.raises(ValueError, match="event made"):
            s.ev.begin(q_off, n_q=n, max_rows=most)
    # a request that brings more rows than the step's is left out and recorded
    x = s.inputs([2, 1, 1])[1].to(DEV)
    s.ev.out.fill_(7.0)
    s.ev.begin(q_off, n_q=4, max_rows=1)
    s.ev.write(0, *s.parts(x[0, :4]), s.k[0], s.v[0], s.bt)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 0
    s.ev.attend(0, s.k[0], s.v[0], s.bt, s.k8[0], s.v8[0], s.ks[0], s.vs[0], s.t8d)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 7
    assert bool((s.ev.out[0, :2] == 7.0).all()) and not bool((s.ev.out[0, 2:4] == 7.0).any(-1).all())


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_behind_a_history_is_recorded(captured):
    """prompt does not see what lies in 8 bits: a request with new rows behind a history is recorded and
    left alone, the others get their attention; a history without new rows is nothing to record."""
    import query_conditioned_kv_gb300 as kvc
    s = Serving(13, recent=0)
    s.step([37, 0, 5], prompt=True)          # 32, 0 and 0 positions in 8 bits
    assert s.len8.tolist() == [32, 0, 0]
    T = [0, 9, 3]
    q_off, x = s.inputs(T)
    s.ev.out.fill_(7.0)
    qd, xd, graph = i32(q_off), x.to(DEV), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.graph(graph):
            s.launch(qd, xd, True)
        graph.replay()
    else:
        s.launch(qd, xd, True)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 0
    s.check_rows(T, q_off, x)
    s.check_attention(T, q_off)
    qd.copy_(i32([0, 4, 4, 7]))
    s.ev.out.fill_(7.0)
    if captured:
        graph.replay()
    else:
        s.launch(qd, xd, True)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 7
    assert bool((s.ev.out[:, :4] == 7.0).all()) and bool((s.ev.out[:, 4:7] != 7.0).any(-1).all())


def test_write_keeps_the_raw_keys():
    """write(k_raw): the step's keys before the rotation, head by head, in a buffer with room behind them."""
    import query_conditioned_kv_gb300 as kvc
    s = Serving(14)
    q_off, x = s.inputs([9, 0, 4])
    s.ev.begin(i32(q_off), n_q=13, max_rows=9)
    raw = torch.full((s.H, 16, s.D), 7.0, dtype=torch.bfloat16, device=DEV)
    s.ev.write(0, *s.parts(x[0, :13].to(DEV)), s.k[0], s.v[0], s.bt, s.wq, s.wk, k_raw=raw)
    torch.cuda.synchronize()
    assert kvc.kvc_device_status(s.ev.dev_status) == 0
    y, rel = ref.normed(s.parts(x[0])[1].reshape(s.n_q, s.H, s.D)[:13], s.wk.cpu(), EPS)
    inside(raw[:, :13], y.transpose(0, 1), (rel + ref.UBF * (1 + rel)) * y.transpose(0, 1).abs() + 1e-38, "raw keys")
    assert bool((raw[:, 13:] == 7.0).all())
