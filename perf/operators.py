"""Cases of the tree-decoding operators: attention of drafted token trees over a paged KV cache, the
commit of the accepted path, accumulated attention weight per cached row, and eviction by it.

`run` computes one pass in elementary torch operations, or, with `own`, through the library's calls
(kvc_tree_attn, kvc_tree_commit, kvc_attn_mass, kvc_mass_evict).  Layouts are the library's: K and V
pools [L][n_slots][H][D] bf16, position p of request r in slot bt[r][p // BS]·BS + p % BS."""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases
# Head shapes: 8B class (8 KV heads, 32 query heads, D 128), 27B class (48 query heads); page size 16
# unless a case says otherwise.  `ctx` is the longest request's cached length; ragged cases draw the
# others between half of it and all of it, and one request holds nothing yet when `empty` is set.

def _attn(name, n_req, ctx, nodes, H=8, G=4, D=128, BS=16, ragged=True, chain=False, empty=False):
    return {"name": name, "op": "attn", "n_req": n_req, "ctx": ctx, "nodes": nodes, "H": H, "G": G,
            "D": D, "BS": BS, "ragged": ragged, "chain": chain, "empty": empty}


def _mass(name, n_req, ctx, rows, L, H=8, G=4, D=128, BS=16, kind="path", decay=1.0):
    return {"name": name, "op": "mass", "n_req": n_req, "ctx": ctx, "rows": rows, "L": L, "H": H,
            "G": G, "D": D, "BS": BS, "kind": kind, "decay": decay}


def _evict(name, n_req, n, budget, L, H=8, D=128, BS=16, fresh=64):
    return {"name": name, "op": "evict", "n_req": n_req, "n": n, "budget": budget, "L": L, "H": H,
            "D": D, "BS": BS, "fresh": fresh}


def _commit(name, n_req, ctx, nodes, path, L, H=8, D=128, BS=16):
    return {"name": name, "op": "commit", "n_req": n_req, "ctx": ctx, "nodes": nodes, "path": path,
            "L": L, "H": H, "D": D, "BS": BS}


def listed():
    return [
        # plain decoding of one agent over a 4K-token cache: the smallest call, latency counts
        _attn("attn_1tok_1req_4k", 1, 4096, 1, ragged=False, chain=True),
        # plain decoding of 64 agents over their 8192-token views
        _attn("attn_1tok_64req_8k", 64, 8192, 1, chain=True),
        # 16 agents verifying 64-node trees over half-million tokens of cache in all
        _attn("attn_64node_16req_32k", 16, 32768, 64),
        # one agent, odd 27-node tree over the full 128K history, 27B-class heads, pages of 32
        _attn("attn_27node_1req_128k", 1, 131049, 27, G=6, BS=32, ragged=False),
        # small-head model: D 64, one query head per KV head, 13-node trees, pages of 8, one request empty
        _attn("attn_13node_24req_d64", 24, 6144, 13, H=16, G=1, D=64, BS=8, empty=True),
        # weights of the accepted paths of eight agents over their views, 12 layers in one call
        _mass("mass_path_8req_8k", 8, 8192, 6, 12, decay=0.95),
        # a 32-query window over a 128K history, four layers
        _mass("mass_window_1req_128k", 1, 131072, 32, 4, kind="window"),
        # a whole 8192-token prompt, causal
        _mass("mass_prompt_1req_8k", 1, 8192, 8192, 1, kind="window"),
        # steady state: 64 new rows per head evicted from a 4096-row cache, 36 layers
        _evict("evict_step_1req_4k", 1, 4160, 4096, 36),
        # 6K -> 4K tokens (pages of 16), 4 requests, 36 layers
        _evict("evict_6k_4k_4req", 4, 6144, 4096, 36, fresh=2048),
        # accepted path of 5 of 27 nodes, one request, 36 layers: latency counts
        _commit("commit_1req_36l", 1, 1000, 27, 5, 36),
        # accepted paths of up to 8 of 64 nodes, 64 requests, 36 layers
        _commit("commit_64req_36l", 64, 250, 64, 8, 36),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "mass", "mass", "mass", "evict", "evict", "commit"])
    D = rng.choice([64, 128, 128])
    BS = rng.choice([5, 8, 16, 16, 16, 32, 64])
    H = rng.choice([1, 2, 4, 8, 8, 8, 16])
    G = rng.choice([1, 2, 3, 4, 4, 4, 6, 8])
    if op == "attn":
        n_req, nodes = _log(rng, 1, 64), _log(rng, 1, 64)
        ctx = _log(rng, 1, 131072)
        while n_req * (ctx + nodes) * H * D > 16 * 24576 * 8 * 128:
            ctx = max(1, ctx // 2)
        while n_req * (ctx + nodes) * H * D * G * nodes > 16 * 24576 * 8 * 128 * 256:
            nodes = max(1, nodes // 2)
        return {k: v for k, v in _attn("", n_req, ctx, nodes, H, G, D, BS, rng.random() < 0.7,
                                       rng.random() < 0.2, n_req > 1 and rng.random() < 0.3).items()
                if k != "name"}
    if op == "mass":
        if rng.random() < 0.3:  # a prompt: every row causal
            n_req, L, kind = rng.choice([1, 1, 2, 3]), 1, "window"
            ctx = rows = _log(rng, 200, 4096)
        else:
            n_req, L = _log(rng, 1, 64), _log(rng, 1, 36)
            kind = rng.choice(["path", "path", "window"])
            rows = _log(rng, 1, 8) if kind == "path" else _log(rng, 8, 64)
            ctx = max(rows, _log(rng, 1, 131072))
            while L > 1 and n_req * ctx * L * H * D > 4 * 131072 * 8 * 128:
                L = (L + 1) // 2
            while n_req * ctx * L * H * D * max(1.0, G * rows / 128) > 4 * 131072 * 8 * 128:
                ctx, rows = (ctx // 2, rows) if ctx // 2 > rows else (ctx, rows // 2)
        return {k: v for k, v in _mass("", n_req, ctx, rows, L, H, G, D, BS, kind,
                                       rng.choice([1.0, 1.0, 0.9])).items() if k != "name"}
    if op == "evict":
        n_req, L, budget = _log(rng, 1, 8), _log(rng, 1, 36), _log(rng, 48, 8192)
        fresh = _log(rng, 1, budget)
        while L > 1 and n_req * (budget + fresh) * L * H * D > 4 * 6144 * 36 * 8 * 128:
            L = (L + 1) // 2
        while n_req * (budget + fresh) * L * H * D > 4 * 6144 * 36 * 8 * 128:
            budget, fresh = budget // 2, max(1, fresh // 2)
        return {k: v for k, v in _evict("", n_req, budget + fresh, budget, L, H, D, BS,
                                        fresh).items() if k != "name"}
    nodes = _log(rng, 2, 64)
    return {k: v for k, v in _commit("", _log(rng, 1, 64), _log(rng, 1, 250), nodes,
                                     min(nodes, _log(rng, 1, 8)), _log(rng, 1, 36), H, D,
                                     BS).items() if k != "name"}


# ----------------------------------------------------------------- inputs

def _tables(rs, n_req, max_blocks):
    """A block table over a pool with a few spare pages, pages in random order."""
    n_blocks = n_req * max_blocks + 3
    return rs.permutation(n_blocks)[:n_req * max_blocks].reshape(n_req, max_blocks), n_blocks


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def _lens(rs, c):
    n = c["n_req"]
    ctx = np.full(n, c["ctx"], np.int64)
    if c.get("ragged", True) and n > 1:
        ctx[1:] = rs.randint((c["ctx"] + 1) // 2, c["ctx"] + 1, n - 1)
    if c.get("empty"):
        ctx[n // 2] = 0
    return ctx


def _rows(gen, shape):
    """bf16 rows: N(0,1) with a common direction added to about one row in 32 (the rows a model
    attends to), the way the benchmark's histories are planted."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    pick = torch.rand(shape[:-1], generator=gen, device=DEV) < 1 / 32
    x[..., 0].add_(pick.to(x.dtype) * 6.0)
    return x


def _tree(rs, T, words, chain):
    """Ancestor-or-self bit masks of a random tree of T nodes in parent-first order."""
    anc = np.eye(T, dtype=bool)
    for j in range(1, T):
        p = j - 1 if chain else int(rs.randint(max(0, j - 12), j))
        anc[j] |= anc[p]
    bits = np.zeros((T, words * 32), bool)
    bits[:, :T] = anc
    return np.packbits(bits.reshape(T, words, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]


def _queries(gen, shape):
    q = torch.randn(shape, generator=gen, device=DEV)
    q[..., 0].add_(3.0)
    return q.to(torch.bfloat16)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return {"attn": _prep_attn, "mass": _prep_mass, "evict": _prep_evict,
            "commit": _prep_commit}[case["op"]](case, rs, gen)


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=DEV)


def _prep_attn(c, rs, gen):
    n_req, H, G, D, BS = c["n_req"], c["H"], c["G"], c["D"], c["BS"]
    ctx = _lens(rs, c)
    # ragged trees: sizes spread over nodes/2 .. nodes (the same for every seed, as are the outputs' shapes)
    T = c["nodes"] - (np.arange(n_req) * 7) % (c["nodes"] // 2 + 1) * int(c["ragged"])
    max_blocks = int(-(-(ctx + T).max() // BS))
    bt, n_blocks = _tables(rs, n_req, max_blocks)
    words = (c["nodes"] + 31) // 32
    q_off = np.concatenate([[0], np.cumsum(T)])
    mask = np.concatenate([_tree(rs, int(t), words, c["chain"]) for t in T])
    n_q = int(q_off[-1])
    s = dict(c, ctx_max=int(ctx.max()), max_blocks=max_blocks, n_slots=n_blocks * BS, n_q=n_q,
             words=words, Hq=H * G, scale=1.0 / math.sqrt(D), bt=_i32(bt), ctx_len=_i32(ctx),
             q_off=_i32(q_off), mask=_i32(mask.view(np.int32)))
    s["kpool"], s["vpool"] = _rows(gen, (n_blocks * BS, H, D)), _rows(gen, (n_blocks * BS, H, D))
    s["q"] = _queries(gen, (n_q, H * G, D))
    s["out"] = torch.empty(n_q, H * G, D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(n_q, H * G, dtype=torch.float32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        import query_conditioned_kv_gb300 as kvc
        s["ws"] = _ws(kvc.kvc_tree_attn_workspace_size(n_req, max_blocks, c["nodes"], H, H * G, D, BS))
    return s


def _prep_mass(c, rs, gen):
    n_req, L, H, G, D, BS = c["n_req"], c["L"], c["H"], c["G"], c["D"], c["BS"]
    seq = _lens(rs, c)
    if c["kind"] == "path":  # 1 .. rows accepted nodes of a larger tree, at the end of the cache
        m = np.minimum(rs.randint(1, c["rows"] + 1, n_req), seq)
        m[0] = min(c["rows"], seq[0])
        per = 2 * c["rows"] + 3
        n_q = n_req * per
        row_off = np.arange(n_req + 1) * c["rows"]
        idx, vis = np.zeros((n_req, c["rows"]), np.int64), np.zeros((n_req, c["rows"]), np.int64)
        for r in range(n_req):
            idx[r, :m[r]] = r * per + np.sort(rs.permutation(per)[:m[r]])
            vis[r, :m[r]] = seq[r] - m[r] + 1 + np.arange(m[r])
        idx, vis = idx.reshape(-1), vis.reshape(-1)
    else:  # the last `rows` positions of the cache, causal
        m = np.minimum(c["rows"], seq)
        row_off = np.concatenate([[0], np.cumsum(m)])
        n_q = int(row_off[-1])
        idx = None
        vis = np.concatenate([seq[r] - m[r] + 1 + np.arange(m[r]) for r in range(n_req)])
    old = np.maximum(seq - m, 0)
    max_blocks = int(-(-seq.max() // BS))
    cap = max_blocks * BS
    bt, n_blocks = _tables(rs, n_req, max_blocks)
    s = dict(c, max_blocks=max_blocks, n_slots=n_blocks * BS, n_q=n_q, n_rows=len(vis), Hq=H * G,
             seq_max=int(seq.max()), scale=1.0 / math.sqrt(D), bt=_i32(bt), seqused=_i32(seq),
             n_mass=_i32(old), row_off=_i32(row_off), row_vis=_i32(vis),
             row_idx=None if idx is None else _i32(idx))
    s["kpool"] = _rows(gen, (L, n_blocks * BS, H, D))
    s["q"] = _queries(gen, (L, n_q, H * G, D))
    # what attention reported for these rows: an LSE near ln(visible) + the planted rows' share
    live = torch.ones(n_q, device=DEV)
    rows = torch.arange(len(vis), device=DEV) if idx is None else s["row_idx"].long()
    live[rows] = s["row_vis"].clamp(min=1).float()
    s["lse"] = live.log()[None, :, None] + 0.5 + \
        0.3 * torch.rand(L, n_q, H * G, generator=gen, device=DEV)
    s["mass"] = torch.rand(L, n_req, H, cap, generator=gen, device=DEV).pow_(4)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        import query_conditioned_kv_gb300 as kvc
        s["ws"] = _ws(kvc.kvc_attn_mass_workspace_size(n_req, max_blocks, c["rows"], L, H, H * G, D,
                                                       BS))
    return s


def _prep_evict(c, rs, gen):
    n_req, L, H, D, BS, n, B = c["n_req"], c["L"], c["H"], c["D"], c["BS"], c["n"], c["budget"]
    seq = np.full(n_req, n, np.int64)
    if n_req > 1:  # others hold a little less; the last has not filled its budget
        seq[1:] = rs.randint(B, n + 1, n_req - 1)
        seq[-1] = max(1, B - c["fresh"] // 2)
    n_pos = np.maximum(seq - c["fresh"], 0)
    t_end = seq + rs.randint(0, 4 * B, n_req)
    max_blocks = int(-(-n // BS))
    cap = max_blocks * BS
    bt, n_blocks = _tables(rs, n_req, max_blocks)
    s = dict(c, max_blocks=max_blocks, cap=cap, n_slots=n_blocks * BS, bt=_i32(bt), seqused=_i32(seq),
             n_pos=_i32(n_pos), t_end=_i32(t_end), n_sink=min(4, B // 8), n_recent=B // 8)
    s["kpool"], s["vpool"] = _rows(gen, (L, n_blocks * BS, H, D)), _rows(gen, (L, n_blocks * BS, H, D))
    # weights of very different size, one row in ten never attended to (equal zeros)
    u = torch.rand(L, n_req, H, cap, generator=gen, device=DEV)
    s["mass"] = torch.where(u < 0.1, torch.zeros_like(u), torch.exp(6 * u - 4 + 2 * torch.rand(
        L, n_req, H, cap, generator=gen, device=DEV)))
    # original positions of the carried rows: distinct, below the first fresh row's
    old = t_end - (seq - n_pos)
    pos = np.stack([rs.permutation(int(o))[:cap] if o >= cap else
                    np.concatenate([rs.permutation(int(o)), np.zeros(cap - o, np.int64)]) for o in old])
    s["pos"] = _i32(pos)[None, :, None, :].expand(L, n_req, H, cap).contiguous()
    s["mass_out"] = torch.zeros_like(s["mass"])
    s["pos_out"] = torch.zeros_like(s["pos"])
    s["n_out"] = torch.zeros(n_req, dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        import query_conditioned_kv_gb300 as kvc
        s["ws"] = _ws(kvc.kvc_mass_evict_workspace_size(n_req, max_blocks, L, H, BS, B))
    return s


def _prep_commit(c, rs, gen):
    n_req, L, H, D, BS = c["n_req"], c["L"], c["H"], c["D"], c["BS"]
    ctx = _lens(rs, c)
    T = np.full(n_req, c["nodes"])
    m = rs.randint(1, c["path"] + 1, n_req)
    m[0] = c["path"]
    path = np.full((n_req, c["path"]), -1, np.int64)
    for r in range(n_req):
        path[r, 1:m[r]] = 1 + np.sort(rs.permutation(c["nodes"] - 1)[:m[r] - 1])
        path[r, 0] = 0
    max_blocks = int(-(-(ctx + T).max() // BS))
    bt, n_blocks = _tables(rs, n_req, max_blocks)
    s = dict(c, max_blocks=max_blocks, n_slots=n_blocks * BS, bt=_i32(bt), ctx_len=_i32(ctx),
             q_off=_i32(np.concatenate([[0], np.cumsum(T)])), path_nodes=_i32(path), n_path=_i32(m))
    s["kpool"], s["vpool"] = _rows(gen, (L, n_blocks * BS, H, D)), _rows(gen, (L, n_blocks * BS, H, D))
    s["seq_out"] = torch.zeros(n_req, dtype=torch.int32, device=DEV)
    s["row_idx"] = torch.zeros(n_req, c["path"], dtype=torch.int32, device=DEV)
    s["row_vis"] = torch.zeros(n_req, c["path"], dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# -------------------------------------------------------------------- run

def run(s):
    return {"attn": _run_attn, "mass": _run_mass, "evict": _run_evict,
            "commit": _run_commit}[s["op"]](s)


def _slots(s, n):
    """Slot of every position 0 .. n-1 of every request: [n_req][n]."""
    p = torch.arange(n, device=DEV)
    return s["bt"].long()[:, p // s["BS"]] * s["BS"] + p % s["BS"]


def _run_attn(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_tree_attn(s["q"], s["kpool"], s["vpool"], s["n_slots"], s["bt"], s["max_blocks"],
                          s["ctx_len"], s["q_off"], None if s["chain"] else s["mask"], s["words"],
                          s["n_req"], s["n_q"], s["nodes"], s["H"], s["Hq"], s["D"], s["BS"],
                          s["scale"], s["out"], s["lse"], s["ws"], s["status"])
        return s["out"], s["lse"]
    T, P, H, G, D = s["nodes"], s["max_blocks"] * s["BS"], s["H"], s["G"], s["D"]
    q_off, ctx = s["q_off"].long(), s["ctx_len"].long()
    j = torch.arange(T, device=DEV)
    row = q_off[:-1, None] + j                                   # [n_req][T]
    live = row < q_off[1:, None]
    row = row.clamp(max=s["n_q"] - 1)
    # which positions node i of request r sees: the cached ones, and the nodes of its mask
    node = torch.arange(P, device=DEV) - ctx[:, None]            # [n_req][P]
    n_nodes = (q_off[1:] - q_off[:-1])[:, None]
    at = node.clamp(0, T - 1)
    word = s["mask"].view(-1, s["words"])[row].gather(
        2, (at // 32)[:, None, :].expand(-1, T, -1))             # [n_req][T][P]
    bit = ((word >> (at % 32)[:, None, :].int()) & 1) == 1
    sees = (node < 0)[:, None, :] | (bit & ((node >= 0) & (node < n_nodes))[:, None, :])
    slot = _slots(s, P)
    k, v = s["kpool"][slot].float(), s["vpool"][slot].float()    # [n_req][P][H][D]
    q = s["q"][row].float().view(-1, T, H, G, D)
    z = torch.einsum("rthgd,rphd->rhgtp", q, k) * s["scale"]
    z = z.masked_fill(~sees[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("rhgtp,rphd->rthgd", e / total.clamp(min=1e-30), v)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    return (o.reshape(-1, T, H * G, D)[live].to(torch.bfloat16),
            lse.reshape(-1, T, H * G)[live])


def _run_mass(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_attn_mass(s["q"], s["lse"], s["n_q"], s["row_idx"], s["row_vis"], s["row_off"],
                          s["n_rows"], s["rows"], s["kpool"], s["n_slots"], s["bt"],
                          s["max_blocks"], s["seqused"], s["n_mass"], s["n_req"], s["L"], s["H"],
                          s["Hq"], s["D"], s["BS"], s["scale"], s["decay"], s["mass"], s["ws"],
                          s["status"])
        return s["mass"]
    R, P, L, H, G, D = s["rows"], s["seq_max"], s["L"], s["H"], s["G"], s["D"]
    off = s["row_off"].long()
    row = off[:-1, None] + torch.arange(R, device=DEV)           # [n_req][R]
    live = row < off[1:, None]
    row = row.clamp(max=s["n_rows"] - 1)
    vis = torch.where(live, s["row_vis"].long()[row], torch.zeros_like(row))
    qrow = row if s["row_idx"] is None else s["row_idx"].long()[row]
    k = s["kpool"][:, _slots(s, P)].float()                      # [L][n_req][P][H][D]
    q = s["q"][:, qrow].float().view(L, -1, R, H, G, D)
    lse = s["lse"][:, qrow].view(L, -1, R, H, G)
    w = torch.einsum("lrthgd,lrphd->lrhgtp", q, k).mul_(s["scale"])
    w = w.sub_(lse.permute(0, 1, 3, 4, 2)[..., None]).exp_()
    p = torch.arange(P, device=DEV)
    w = w.masked_fill_((p >= vis[..., None])[None, :, None, None], 0.0)
    add = w.sum((3, 4))                                          # [L][n_req][H][P]
    old = s["mass"][..., :P]
    kept = torch.where(p < s["n_mass"].long()[:, None, None], old * s["decay"], torch.zeros_like(old))
    s["mass"][..., :P] = torch.where(p < s["seqused"].long()[:, None, None], kept + add, old)
    return s["mass"]


def _run_evict(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_mass_evict(s["kpool"], s["vpool"], s["n_slots"], s["bt"], s["max_blocks"],
                           s["seqused"], s["n_pos"], s["t_end"], s["mass"], s["pos"], s["mass_out"],
                           s["pos_out"], s["n_out"], s["n_req"], s["L"], s["H"], s["D"], s["BS"],
                           s["budget"], s["n_sink"], s["n_recent"], s["ws"], s["status"])
        return s["kpool"], s["vpool"], s["mass_out"], s["pos_out"], s["n_out"]
    n_req, L, H, cap, B = s["n_req"], s["L"], s["H"], s["cap"], s["budget"]
    p = torch.arange(cap, device=DEV)
    n = s["seqused"].long()[:, None, None]                       # [n_req][1][1]
    t_end = s["t_end"].long()[:, None, None]
    pos = torch.where(p < s["n_pos"].long()[:, None, None], s["pos"].long(), t_end - (n - p))
    pinned = (pos < s["n_sink"]) | (pos >= t_end - s["n_recent"])
    key = torch.where(pinned, torch.full_like(s["mass"], math.inf), s["mass"])
    key = torch.where(p < n, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, p.expand_as(order))
    n_out = n.clamp(max=B)
    keep = (rank < n_out) & (p < n)
    # the k-th kept row past the budget goes to the k-th hole below it
    M = cap - B if cap > B else 1
    hole = (~keep) & (p < n_out)
    tail = keep & (p >= B)
    dst = torch.sort(hole.int(), dim=-1, descending=True, stable=True).indices[..., :M]
    src = torch.sort(tail.int(), dim=-1, descending=True, stable=True).indices[..., :M]
    k = torch.arange(M, device=DEV)
    some = k < tail.sum(-1, keepdim=True)
    stay = (B + k).clamp(max=cap - 1).expand_as(src)             # a row past the budget, onto itself
    src, dst = torch.where(some, src, stay), torch.where(some, dst, stay)
    li = torch.arange(L, device=DEV)[:, None, None, None]
    ri = torch.arange(n_req, device=DEV)[:, None, None]
    hi = torch.arange(H, device=DEV)[:, None]
    slot = _slots(s, cap)
    s_src, s_dst = slot[ri, src], slot[ri, dst]
    for pool in (s["kpool"], s["vpool"]):
        pool[li, s_dst, hi] = pool[li, s_src, hi]
    own_row = keep & (p < n_out)
    for new, old in ((s["mass_out"], s["mass"]), (s["pos_out"], pos.to(torch.int32))):
        new.copy_(torch.where(own_row, old, new))
        moved = old.gather(-1, src)
        new.scatter_(-1, dst, torch.where(some, moved, new.gather(-1, dst)))
    s["n_out"].copy_(n_out[:, 0, 0])
    return s["kpool"], s["vpool"], s["mass_out"], s["pos_out"], s["n_out"]


def _run_commit(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_tree_commit(s["kpool"], s["vpool"], s["n_slots"], s["bt"], s["max_blocks"],
                            s["ctx_len"], s["q_off"], s["path_nodes"], s["n_path"], s["path"],
                            s["n_req"], s["L"], s["H"], s["D"], s["BS"], s["seq_out"],
                            s["row_idx"], s["row_vis"], s["status"])
        return s["kpool"], s["vpool"], s["seq_out"], s["row_idx"], s["row_vis"]
    i = torch.arange(s["path"], device=DEV)
    ctx, n = s["ctx_len"].long()[:, None], s["n_path"].long()[:, None]
    some = i < n
    node = torch.where(some, s["path_nodes"].long(), i.expand_as(some))  # past the path: onto itself
    slot = _slots(s, s["max_blocks"] * s["BS"])
    last = slot.shape[1] - 1
    src = slot.gather(1, (ctx + node).clamp(max=last))
    dst = slot.gather(1, (ctx + i).clamp(max=last))
    src = torch.where(some, src, dst)
    for pool in (s["kpool"], s["vpool"]):
        pool[:, dst] = pool[:, src]
    s["seq_out"].copy_((ctx + n)[:, 0])
    s["row_idx"].copy_(torch.where(some, s["q_off"].long()[:-1, None] + node, torch.zeros_like(node)))
    s["row_vis"].copy_(torch.where(some, ctx + i + 1, torch.zeros_like(node)))
    return s["kpool"], s["vpool"], s["seq_out"], s["row_idx"], s["row_vis"]


# ------------------------------------------------------------------- work

def work(case):
    c, H, D = case, case["H"], case["D"]
    n_req = c["n_req"]
    if c["op"] == "evict":
        seqs = [c["n"]] + [(c["budget"] + c["n"]) / 2] * (n_req - 2) + [c["budget"]] * (n_req > 1)
        B, bts = c["budget"], 0.0
        for n in seqs:
            pin = B // 8 + min(4, B // 8)
            extra = max(0, n - B)
            held = min(B // 8, extra)  # recent rows past the budget, all of them kept
            moved = held + (extra - held) * (B - pin) / max(1, n - pin)
            bts += c["L"] * H * (8 * n + 8 * min(n, B) + moved * D * 2 * 2 * 2)
        return {"bytes": bts, "flops": 0}
    if c["op"] == "commit":
        moved = n_req * max(0.5, (c["path"] - 1) / 2)
        return {"bytes": moved * H * D * 2 * 2 * 2 * c["L"] + n_req * 40, "flops": 0}
    mean = c["ctx"] * (1.0 if n_req == 1 or not c.get("ragged", True) else 0.75)
    Hq = H * c["G"]
    if c["op"] == "attn":
        T = c["nodes"] * (0.75 if c["ragged"] and n_req > 1 else 1.0)
        return {"bytes": n_req * ((mean + T) * H * D * 4 + T * Hq * (D * 4 + 4)),
                "flops": 4 * D * Hq * n_req * T * (mean + T / 4)}
    rows = c["rows"] * (0.55 if c["kind"] == "path" and n_req > 1 else 1.0)
    seen = mean - rows / 2
    return {"bytes": c["L"] * n_req * (mean * H * (D * 2 + 8) + rows * Hq * (D * 2 + 4)),
            "flops": c["L"] * n_req * 2 * D * Hq * rows * seen}


# ------------------------------------------------------------------ exact
# The definitions in 64 bits, request by request, from the same inputs.

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "mass": _exact_mass, "evict": _exact_evict,
            "commit": _exact_commit}[case["op"]](s)


def _where(s, r, n):
    table = s["bt"][r].tolist()
    return torch.tensor([table[i // s["BS"]] * s["BS"] + i % s["BS"] for i in range(n)],
                        dtype=torch.long, device=DEV)


def _exact_attn(s):
    G, words = s["G"], s["words"]
    q_off, ctx = s["q_off"].tolist(), s["ctx_len"].tolist()
    out = torch.zeros(s["n_q"], s["Hq"], s["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((s["n_q"], s["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    masks = s["mask"].cpu().numpy().view(np.uint32).reshape(-1, words)
    for r in range(s["n_req"]):
        a, b = q_off[r], q_off[r + 1]
        n, T = ctx[r], q_off[r + 1] - q_off[r]
        where = _where(s, r, n + T)
        allow = torch.zeros(T, n + T, dtype=torch.bool)
        allow[:, :n] = True
        for i in range(T):
            for j in range(T):
                allow[i, n + j] = bool((int(masks[a + i, j // 32]) >> (j % 32)) & 1)
        allow = allow.to(DEV)
        for h in range(s["H"]):
            k, v = s["kpool"][where, h].double(), s["vpool"][where, h].double()
            for g in range(h * G, h * G + G):
                logit = s["q"][a:b, g].double() @ k.T / math.sqrt(s["D"])
                logit[~allow] = -math.inf
                total = torch.logsumexp(logit, 1)
                lse[a:b, g] = total
                out[a:b, g] = torch.exp(logit - total[:, None]) @ v
    return out, lse


def _exact_mass(s):
    if s["n_req"] * s["L"] * s["H"] * s["G"] > 16384:
        return None
    G = s["G"]
    off, seq, old = s["row_off"].tolist(), s["seqused"].tolist(), s["n_mass"].tolist()
    got = s["mass"].double()
    for r in range(s["n_req"]):
        n = seq[r]
        where = _where(s, r, n)
        vis = s["row_vis"][off[r]:off[r + 1]].long()
        rows = torch.arange(off[r], off[r + 1], device=DEV) if s["row_idx"] is None else \
            s["row_idx"][off[r]:off[r + 1]].long()
        hidden = torch.arange(n, device=DEV)[None] >= vis[:, None]
        for layer in range(s["L"]):
            for h in range(s["H"]):
                k = s["kpool"][layer, where, h].double()
                total = torch.zeros(n, dtype=torch.float64, device=DEV)
                for g in range(h * G, h * G + G):
                    w = torch.exp(s["q"][layer, rows, g].double() @ k.T / math.sqrt(s["D"])
                                  - s["lse"][layer, rows, g].double()[:, None])
                    w[hidden] = 0
                    total += w.sum(0)
                total[:old[r]] += s["decay"] * got[layer, r, h, :old[r]]
                got[layer, r, h, :n] = total
    return got


def _exact_evict(s):
    """Eviction copies rows and computes nothing: the weights that stay, row by row on the host;
    the other outputs are compared as they are."""
    seq, n_pos, t_end = s["seqused"].tolist(), s["n_pos"].tolist(), s["t_end"].tolist()
    mass, pos = s["mass"].cpu().numpy(), s["pos"].cpu().numpy()
    out, B = np.zeros(mass.shape), s["budget"]
    for r in range(s["n_req"]):
        n = seq[r]
        for layer in range(s["L"]):
            for h in range(s["H"]):
                w = mass[layer, r, h, :n]
                at = pos[layer, r, h, :n].astype(np.int64)
                at[n_pos[r]:] = t_end[r] - n + np.arange(n_pos[r], n)
                if n > B:
                    pin = (at < s["n_sink"]) | (at >= t_end[r] - s["n_recent"])
                    free = np.flatnonzero(~pin)
                    best = free[np.lexsort((free, -w[free].astype(np.float64)))][:B - int(pin.sum())]
                    stay = np.zeros(n, bool)
                    stay[pin] = True
                    stay[best] = True
                    new = w[:B].astype(np.float64)
                    new[np.flatnonzero(~stay[:B])] = w[B + np.flatnonzero(stay[B:])]
                else:
                    new = w.astype(np.float64)
                out[layer, r, h, :len(new)] = new
    return None, None, torch.from_numpy(out), None, None


def _exact_commit(s):
    """A commit copies rows: each request's, one after the other."""
    ctx, n = s["ctx_len"].tolist(), s["n_path"].tolist()
    path = s["path_nodes"].tolist()
    k, v = s["kpool"].clone(), s["vpool"].clone()
    for r in range(s["n_req"]):
        where = _where(s, r, ctx[r] + s["nodes"])
        for i in range(n[r]):
            if path[r][i] != i:
                k[:, where[ctx[r] + i]] = s["kpool"][:, where[ctx[r] + path[r][i]]]
                v[:, where[ctx[r] + i]] = s["vpool"][:, where[ctx[r] + path[r][i]]]
    return k, v, None, None, None
