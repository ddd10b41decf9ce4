"""Cases of the operators that fill a paged cache and read what it holds in 8 bits: the norms and the
position rotation of queries and keys with their way into the cache, attention over whole prompts,
packing cached blocks to 8 bits, and attention over an 8-bit history with the recent rows behind it.

`run` computes one pass in elementary torch operations, or, with `own`, through the library's calls
(kvc_qkv_rope, kvc_prompt_attn, kvc_q8_pack, kvc_q8_attn).  Layouts are the library's: K and V pools
[L][n_slots][H][D] bf16, position p of request r in slot bt[r][p // BS]·BS + p % BS; 8-bit pools
[L][n_blocks][H][BS][D] e4m3 with an fp32 scale (a power of two) per block and head."""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
# Head shapes: 8B class (8 KV heads, 32 query heads, D 128), 27B class (48 query heads); page size 16
# unless a case says otherwise.  `ctx` is the longest request's cached length before the call, `rows`
# its new tokens; in ragged cases the other requests bring between half of them and all of them, and
# one brings none when `empty` is set.

def _rope(name, n_req, ctx, rows, H=8, G=4, D=128, BS=16, ragged=False, norm=True, raw=False):
    return {"name": name, "op": "rope", "n_req": n_req, "ctx": ctx, "rows": rows, "H": H, "G": G,
            "D": D, "BS": BS, "ragged": ragged, "empty": False, "norm": norm, "raw": raw}


def _prompt(name, n_req, ctx, rows, H=8, G=4, D=128, BS=16, ragged=False, empty=False):
    return {"name": name, "op": "prompt", "n_req": n_req, "ctx": ctx, "rows": rows, "H": H, "G": G,
            "D": D, "BS": BS, "ragged": ragged, "empty": empty}


def _pack(name, n, L, H=8, D=128, BS=16):
    return {"name": name, "op": "pack", "n": n, "L": L, "H": H, "D": D, "BS": BS}


def _q8(name, n_req, hist, ctx, rows, H=8, G=4, D=128, BS=16, ragged=False, empty=False):
    return {"name": name, "op": "q8", "n_req": n_req, "hist": hist, "ctx": ctx, "rows": rows, "H": H,
            "G": G, "D": D, "BS": BS, "ragged": ragged, "empty": empty}


def listed():
    return [
        # one agent's next token on its way into a 4K cache: the smallest call, latency counts
        _rope("rope_1tok_1req", 1, 4096, 1),
        # a whole 8192-token prompt, its raw keys kept for the block index too
        _rope("rope_prompt_8k", 1, 0, 8192, raw=True),
        # the next pieces of five packed prompts, 27B-class heads, no norms, pages of 32
        _rope("rope_chunks_5req_27b", 5, 4001, 6007, G=6, BS=32, ragged=True, norm=False),
        # short prompts of a small-head model: D 64, one query head per KV head, pages of 8, one empty
        _prompt("prompt_7req_190_d64", 7, 0, 190, H=16, G=1, D=64, BS=8, ragged=True, empty=True),
        # a whole 8192-token prompt
        _prompt("prompt_1req_8k", 1, 0, 8192),
        # four packed prompts of odd lengths, 27B-class heads
        _prompt("prompt_4req_6k_27b", 4, 0, 6001, G=6, ragged=True),
        # the next 2048 tokens behind a 128K history
        _prompt("prompt_2k_after_128k", 1, 129001, 2048),
        # the block that eight agents have just filled, 36 layers: latency counts
        _pack("pack_8blocks_36l", 8, 36),
        # a 32K prompt's blocks, 12 layers
        _pack("pack_32k_12l", 2048, 12),
        # plain decoding of one agent: a 4K history in 8 bits, 100 recent rows
        _q8("q8_1tok_1req_4k", 1, 4096, 100, 1),
        # plain decoding of 64 agents over 8K histories and up to 256 recent rows
        _q8("q8_1tok_64req_8k", 64, 8192, 256, 1, ragged=True),
        # three drafted tokens of two agents over the full 128K history, 27B-class heads, pages of 32
        _q8("q8_3tok_2req_128k", 2, 131072, 41, 3, G=6, BS=32),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "prompt", "pack", "q8", "q8", "q8"])
    D = rng.choice([64, 128, 128])
    BS = rng.choice([5, 8, 16, 16, 16, 32, 64])
    H = rng.choice([1, 2, 4, 8, 8, 8, 16])
    G = rng.choice([1, 2, 3, 4, 4, 4, 6, 8])
    ragged, empty = rng.random() < 0.6, rng.random() < 0.3
    if op == "rope":
        n_req, rows, ctx = _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 1, 8192)
        while n_req * rows * H * (G + 2) * D > 24576 * 64 * 128:
            rows = (rows + 1) // 2
        while n_req * (ctx + rows) * H * D > 4 * 131072 * 8 * 128:
            ctx = ctx // 2
        c = _rope("", n_req, ctx, rows, H, G, D, BS, ragged, rng.random() < 0.7, rng.random() < 0.4)
    elif op == "prompt":
        n_req, rows = _log(rng, 1, 16), _log(rng, 1, 8192)
        ctx = rng.choice([0, 0, _log(rng, 1, 131072)])
        while n_req * G * rows * (ctx + rows) > 2048 * 4 * 131072 or \
                n_req * H * G * D * rows * (ctx + rows) > 2048 * 32 * 128 * 131072:
            ctx, rows = (ctx // 2, rows) if ctx > 2 * rows else (ctx, (rows + 1) // 2)
        c = _prompt("", n_req, ctx, rows, H, G, D, BS, ragged, empty and n_req > 1)
    elif op == "pack":
        L, n = _log(rng, 1, 36), _log(rng, 1, 4096)
        while n * BS * L * H * D > 2048 * 16 * 12 * 8 * 128:
            n = (n + 1) // 2
        c = _pack("", n, L, H, D, BS)
    else:
        n_req, hist, ctx, rows = _log(rng, 1, 64), _log(rng, 1, 131072), rng.randint(0, 512), _log(rng, 1, 8)
        while n_req * hist * H * D > 64 * 8192 * 8 * 128:
            hist = hist // 2
        while n_req * hist * H * D * G * rows > 2 * 131072 * 8 * 128 * 24:
            rows = (rows + 1) // 2 if rows > 1 else rows
            hist = hist // 2 if rows == 1 else hist
        c = _q8("", n_req, hist, ctx, rows, H, G, D, BS, ragged, empty and n_req > 1)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs

def _lens(c, most):
    """The longest request's length first, then ragged ones (the others between half of it and all)."""
    n = c["n_req"]
    x = np.full(n, most, np.int64)
    if c["ragged"] and n > 1:
        x[1:] = most - (np.arange(1, n) * 7919 + 13) % (most // 2 + 1)
    return x


def _shape(c):
    """Cached lengths and new rows of every request: by the case alone, as are the outputs' shapes."""
    ctx, rows = _lens(c, c["ctx"]), np.maximum(_lens(c, c["rows"]), 1)
    if c["empty"]:
        rows[c["n_req"] // 2] = 0
    return ctx, rows


def _tables(rs, n_req, max_blocks, spare=3):
    """A block table over a pool with a few spare pages, pages in random order."""
    n_blocks = n_req * max_blocks + spare
    return rs.permutation(n_blocks)[:n_req * max_blocks].reshape(n_req, max_blocks), n_blocks


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def _rows(gen, shape):
    """bf16 rows: N(0,1) with a common direction added to about one row in 32 (the rows a model
    attends to), the way the benchmark's histories are planted."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    pick = torch.rand(shape[:-1], generator=gen, device=DEV) < 1 / 32
    x[..., 0].add_(pick.to(x.dtype) * 6.0)
    return x


def _queries(gen, shape):
    q = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    q[..., 0].add_(3.0)
    return q


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return {"rope": _prep_rope, "prompt": _prep_prompt, "pack": _prep_pack,
            "q8": _prep_q8}[case["op"]](case, rs, gen)


def _paged(c, rs):
    ctx, rows = _shape(c)
    max_blocks = int(max(1, -(-(ctx + rows).max() // c["BS"])))
    bt, n_blocks = _tables(rs, c["n_req"], max_blocks)
    q_off = np.concatenate([[0], np.cumsum(rows)])
    return dict(c, Hq=c["H"] * c["G"], max_blocks=max_blocks, n_slots=n_blocks * c["BS"],
                n_q=int(q_off[-1]), bt=_i32(bt), ctx_len=_i32(ctx), q_off=_i32(q_off),
                scale=1.0 / math.sqrt(c["D"]),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prep_rope(c, rs, gen):
    s = _paged(c, rs)
    H, Hq, D, n = c["H"], s["Hq"], c["D"], s["n_q"]
    # the fused projection's output, queries, keys and values side by side
    qkv = torch.randn(n, (Hq + 2 * H) * D, generator=gen, device=DEV).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:]
    s["wq"] = s["wk"] = None
    if c["norm"]:
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16)
                            for _ in range(2))
    # positions of the rotation: where the tokens stand in their requests, which is past their place
    # in a cache that has evicted rows
    ctx, rows = s["ctx_len"].tolist(), (s["q_off"][1:] - s["q_off"][:-1]).tolist()
    at = np.concatenate([a + np.arange(b) for a, b in zip(ctx, rows)]) + 1000
    s["pos"], s["n_pos"] = _i32(at), int(at.max()) + 1
    angle = torch.arange(s["n_pos"], device=DEV, dtype=torch.float64)[:, None] * \
        torch.pow(torch.tensor(1e6, dtype=torch.float64, device=DEV),
                  torch.arange(D // 2, device=DEV, dtype=torch.float64) * (-2.0 / D))
    s["tab"] = torch.stack([angle.cos(), angle.sin()], -1).float()      # [n_pos][D/2][2]
    s["kpool"], s["vpool"] = _rows(gen, (s["n_slots"], H, D)), _rows(gen, (s["n_slots"], H, D))
    s["q_out"] = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["k_raw"] = torch.empty(H, n, D, dtype=torch.bfloat16, device=DEV) if c["raw"] else None
    return s


def _prep_prompt(c, rs, gen):
    s = _paged(c, rs)
    H, D = c["H"], c["D"]
    s["max_rows"] = int((s["q_off"][1:] - s["q_off"][:-1]).max())
    s["kpool"], s["vpool"] = _rows(gen, (s["n_slots"], H, D)), _rows(gen, (s["n_slots"], H, D))
    s["q"] = _queries(gen, (s["n_q"], s["Hq"], D))
    s["out"] = torch.empty(s["n_q"], s["Hq"], D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(s["n_q"], s["Hq"], dtype=torch.float32, device=DEV)
    return s


def _prep_pack(c, rs, gen):
    L, H, D, BS, n = c["L"], c["H"], c["D"], c["BS"], c["n"]
    n_src, n_dst = n + 3, n + 5
    s = dict(c, n_slots=n_src * BS, n_blocks8=n_dst, src=_i32(rs.permutation(n_src)[:n]),
             dst=_i32(rs.permutation(n_dst)[:n]),
             status=torch.zeros(1, dtype=torch.int32, device=DEV))
    s["kpool"], s["vpool"] = _rows(gen, (L, n_src * BS, H, D)), _rows(gen, (L, n_src * BS, H, D))
    s["k8"], s["v8"] = (torch.zeros(L, n_dst, H, BS, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    s["kscale"], s["vscale"] = (torch.ones(L, n_dst, H, device=DEV) for _ in range(2))
    return s


def _prep_q8(c, rs, gen):
    s = _paged(c, rs)
    H, D, BS, n_req = c["H"], c["D"], c["BS"], c["n_req"]
    hist = _lens(c, c["hist"])
    s["max_blocks8"] = int(max(1, -(-hist.max() // BS)))
    bt8, s["n_blocks8"] = _tables(rs, n_req, s["max_blocks8"])
    s["bt8"], s["len8"] = _i32(bt8), _i32(hist)
    s["max_rows"] = c["rows"]
    s["kpool"], s["vpool"] = _rows(gen, (s["n_slots"], H, D)), _rows(gen, (s["n_slots"], H, D))
    s["q"] = _queries(gen, (s["n_q"], s["Hq"], D))
    # a history packed earlier: bf16 rows, each block and head under its own scale
    s["k8"], s["kscale"] = _e4m3(_rows(gen, (s["n_blocks8"], H, BS, D)))
    s["v8"], s["vscale"] = _e4m3(_rows(gen, (s["n_blocks8"], H, BS, D)))
    s["out"] = torch.empty(s["n_q"], s["Hq"], D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(s["n_q"], s["Hq"], dtype=torch.float32, device=DEV)
    if own:
        import query_conditioned_kv_gb300 as kvc
        n = kvc.kvc_q8_attn_workspace_size(n_req, s["max_blocks8"], s["max_blocks"], s["max_rows"], H,
                                           s["Hq"], D, BS)
        s["ws"] = torch.empty(max(int(n), 16), dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------------- run

def run(s):
    return {"rope": _run_rope, "prompt": _run_prompt, "pack": _run_pack, "q8": _run_q8}[s["op"]](s)


def _slots(s, n):
    """Slot of every position 0 .. n-1 of every request: [n_req][n]."""
    p = torch.arange(n, device=DEV)
    return s["bt"].long()[:, p // s["BS"]] * s["BS"] + p % s["BS"]


def _run_rope(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_qkv_rope(s["q"], s["k"], s["v"], s["n_q"], s["wq"], s["wk"], EPS, s["tab"], s["n_pos"],
                         s["pos"], s["q_off"], s["ctx_len"], s["n_req"], s["bt"], s["max_blocks"],
                         s["kpool"], s["vpool"], s["n_slots"], s["H"], s["Hq"], s["D"], s["BS"],
                         s["q_out"], s["k_raw"], s["status"])
        return s["q_out"], s["kpool"], s["vpool"], s["k_raw"]
    n, H, D, half = s["n_q"], s["H"], s["D"], s["D"] // 2
    cos, sin = s["tab"][s["pos"].long()].unbind(-1)                      # [n][D/2]
    cos, sin = cos[:, None], sin[:, None]

    def normed(x, w):
        x = x.reshape(n, -1, D).float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        return x

    def rotated(x):
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    x = torch.arange(n, device=DEV)
    r = torch.searchsorted(s["q_off"].long(), x, right=True) - 1         # each token's request
    p = s["ctx_len"].long()[r] + x - s["q_off"].long()[r]
    slot = s["bt"].long()[r, p // s["BS"]] * s["BS"] + p % s["BS"]
    k = normed(s["k"], s["wk"])
    s["q_out"].copy_(rotated(normed(s["q"], s["wq"])))
    s["kpool"][slot] = rotated(k)
    s["vpool"][slot] = s["v"].reshape(n, H, D)
    if s["k_raw"] is not None:
        s["k_raw"].copy_(k.permute(1, 0, 2))
    return s["q_out"], s["kpool"], s["vpool"], s["k_raw"]


def _run_prompt(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_prompt_attn(s["q"], s["kpool"], s["vpool"], s["n_slots"], s["bt"], s["max_blocks"],
                            s["ctx_len"], s["q_off"], s["n_req"], s["n_q"], s["max_rows"], s["H"],
                            s["Hq"], s["D"], s["BS"], s["scale"], s["out"], s["lse"], s["status"])
        return s["out"], s["lse"]
    T, P, G = s["max_rows"], s["max_blocks"] * s["BS"], s["G"]
    q_off, ctx = s["q_off"].long(), s["ctx_len"].long()
    row = q_off[:-1, None] + torch.arange(T, device=DEV)                 # [n_req][T]
    live = row < q_off[1:, None]
    at = row.clamp(max=s["n_q"] - 1)
    last = ctx[:, None] + torch.arange(T, device=DEV)
    hidden = (torch.arange(P, device=DEV) > last[..., None])[:, None]    # [n_req][1][T][P]
    slot = _slots(s, P)
    out, lse = [], []
    for h in range(s["H"]):  # (the logits of one group's heads at a time)
        k, v = s["kpool"][slot, h].float(), s["vpool"][slot, h].float()
        q = s["q"][at][:, :, h * G:h * G + G].float()
        z = torch.einsum("rtgd,rpd->rgtp", q, k).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        top = z.amax(-1, keepdim=True)
        e = z.sub_(top).exp_()
        total = e.sum(-1, keepdim=True)
        out.append(torch.einsum("rgtp,rpd->rtgd", e, v) / total.permute(0, 2, 1, 3))
        lse.append((top + total.log()).squeeze(-1).permute(0, 2, 1))
        del z, e
    s["out"].copy_(torch.cat(out, 2)[live])
    s["lse"].copy_(torch.cat(lse, 2)[live])
    return s["out"], s["lse"]


def _power(e):
    """2^e in fp32, exactly (e of -126 .. 127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _e4m3(x):
    """Blocks [..][BS][D] in 8 bits (bytes), and their scales [..]: the least power of two, from 2^-126
    on, whose 448-fold holds the block's largest value; 1 for a block of zeros."""
    x = x.float()
    top = x.abs().amax((-2, -1))
    m, e = torch.frexp(top)                                              # top = m·2^e, m in [1/2, 1)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    e = torch.where(top > 0, e, torch.zeros_like(e))
    y = x * _power(-e)[..., None, None]
    return y.to(torch.float8_e4m3fn).view(torch.uint8), _power(e)


def _run_pack(s):
    f8 = torch.float8_e4m3fn
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_q8_pack(s["kpool"], s["vpool"], s["n_slots"], s["k8"], s["v8"], s["kscale"], s["vscale"],
                        s["n_blocks8"], s["src"], s["dst"], s["n"], s["L"], s["H"], s["D"], s["BS"],
                        s["status"])
        return s["k8"].view(f8), s["v8"].view(f8), s["kscale"], s["vscale"]
    src, dst = s["src"].long(), s["dst"].long()
    pages = s["kpool"].view(s["L"], -1, s["BS"], s["H"], s["D"])[:, src].transpose(2, 3)
    s["k8"][:, dst], s["kscale"][:, dst] = _e4m3(pages)
    pages = s["vpool"].view(s["L"], -1, s["BS"], s["H"], s["D"])[:, src].transpose(2, 3)
    s["v8"][:, dst], s["vscale"][:, dst] = _e4m3(pages)
    return s["k8"].view(f8), s["v8"].view(f8), s["kscale"], s["vscale"]


def _run_q8(s):
    if own:
        import query_conditioned_kv_gb300 as kvc
        kvc.kvc_q8_attn(s["q"], s["k8"], s["v8"], s["kscale"], s["vscale"], s["n_blocks8"], s["bt8"],
                        s["max_blocks8"], s["len8"], s["kpool"], s["vpool"], s["n_slots"], s["bt"],
                        s["max_blocks"], s["ctx_len"], s["q_off"], None, 0, s["n_req"], s["n_q"],
                        s["max_rows"], s["H"], s["Hq"], s["D"], s["BS"], s["scale"], s["out"], s["lse"],
                        s["ws"], s["status"])
        return s["out"], s["lse"]
    T, P, P8 = s["max_rows"], s["max_blocks"] * s["BS"], s["max_blocks8"] * s["BS"]
    H, G, D, n_req = s["H"], s["G"], s["D"], s["n_req"]
    q_off, ctx = s["q_off"].long(), s["ctx_len"].long()
    row = q_off[:-1, None] + torch.arange(T, device=DEV)                 # [n_req][T]
    live = row < q_off[1:, None]
    at = row.clamp(max=s["n_q"] - 1)
    last = ctx[:, None] + torch.arange(T, device=DEV)
    see8 = torch.arange(P8, device=DEV) < s["len8"].long()[:, None]      # [n_req][P8]
    see = torch.arange(P, device=DEV) <= last[..., None]                 # [n_req][T][P]
    sees = torch.cat([see8[:, None].expand(-1, T, -1), see], -1)[:, None, None]
    slot, blocks = _slots(s, P), s["bt8"].long()

    def held(x8, scale, pool):                                           # [n_req][H][P8 + P][D]
        x = x8[blocks].view(torch.float8_e4m3fn).float() * scale[blocks][..., None, None]
        x = x.transpose(1, 2).reshape(n_req, H, P8, D)
        return torch.cat([x, pool[slot].float().transpose(1, 2)], 2)

    k, v = held(s["k8"], s["kscale"], s["kpool"]), held(s["v8"], s["vscale"], s["vpool"])
    q = s["q"][at].float().view(n_req, T, H, G, D)
    z = torch.einsum("rthgd,rhpd->rhgtp", q, k).mul_(s["scale"]).masked_fill_(~sees, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("rhgtp,rhpd->rthgd", e / total, v)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    s["out"].copy_(o.reshape(n_req, T, H * G, D)[live])
    s["lse"].copy_(lse.reshape(n_req, T, H * G)[live])
    return s["out"], s["lse"]


# ------------------------------------------------------------------- work

def work(case):
    c, H, D = case, case["H"], case["D"]
    if c["op"] == "pack":
        values = 2 * c["n"] * c["BS"] * c["L"] * H * D
        return {"bytes": values * 3 + 8 * c["n"] * c["L"] * H + 8 * c["n"], "flops": 0}
    ctx, rows = _shape(c)
    n, Hq = int(rows.sum()), H * c["G"]
    if c["op"] == "rope":
        head = 2 * D  # bytes of one head's row
        b = n * head * 2 * (Hq + 2 * H) + n * H * head * int(c["raw"]) + 4 * n * D + 4 * n
        return {"bytes": b, "flops": 0}
    seen = float((rows * ctx + rows * (rows + 1) / 2).sum())             # (row, key) pairs, one head
    b = n * Hq * (4 * D + 4) + float((ctx + rows)[rows > 0].sum()) * H * D * 4
    if c["op"] == "q8":
        hist = _lens(c, c["hist"])
        seen += float((rows * hist).sum())
        b += float(hist[rows > 0].sum()) * H * D * 2
    return {"bytes": b, "flops": 4 * D * Hq * seen}


# ------------------------------------------------------------------ exact
# The definitions in 64 bits, request by request and head by head, from the same inputs.

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prompt", "q8") and work(case)["flops"] > 8e12:
        return None
    return {"rope": _exact_rope, "prompt": _exact_attn, "pack": _exact_pack, "q8": _exact_attn}[s["op"]](s)


def _where(s, r, n):
    table, BS = s["bt"][r].cpu().numpy().astype(np.int64), s["BS"]
    i = np.arange(n)
    return torch.from_numpy(table[i // BS] * BS + i % BS).to(DEV)


def _exact_rope(s):
    D, Hq, H = s["D"], s["Hq"], s["H"]
    q_off, ctx = s["q_off"].tolist(), s["ctx_len"].tolist()
    angle = torch.view_as_complex(s["tab"].double())[s["pos"].long()]    # cos + i·sin, [n][D/2]

    def unit(x, w):
        x = x.double().unflatten(1, (-1, D))
        return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()

    def turn(x):
        z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * angle[:, None]
        return torch.cat((z.real, z.imag), -1)

    raw = unit(s["k"], s["wk"])
    k, v, new_k = s["kpool"].double(), s["vpool"].double(), turn(raw)
    for r in range(s["n_req"]):
        a, b = q_off[r], q_off[r + 1]
        to = _where(s, r, ctx[r] + b - a)[ctx[r]:]
        k[to], v[to] = new_k[a:b], s["v"][a:b].double().unflatten(1, (H, D))
    return turn(unit(s["q"], s["wq"])), k, v, None if s["k_raw"] is None else raw.transpose(0, 1).contiguous()


def _exact_attn(s):
    G, q_off, ctx = s["G"], s["q_off"].tolist(), s["ctx_len"].tolist()
    out = torch.zeros(s["n_q"], s["Hq"], s["D"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["n_q"], s["Hq"], dtype=torch.float64, device=DEV)
    for r in range(s["n_req"]):
        a, T, n = q_off[r], q_off[r + 1] - q_off[r], ctx[r]
        if T == 0:
            continue
        where = _where(s, r, n + T)
        old = s["len8"].tolist()[r] if "len8" in s else 0
        later = torch.ones(T, T, dtype=torch.bool, device=DEV).triu(1)
        for h in range(s["H"]):
            k, v = s["kpool"][where, h].double(), s["vpool"][where, h].double()
            if old:
                pages = s["bt8"][r, :-(-old // s["BS"])].long()
                k, v = (torch.cat([(x[pages, h].view(torch.float8_e4m3fn).double() *
                                    e[pages, h].double()[:, None, None]).flatten(0, 1)[:old], y])
                        for x, e, y in ((s["k8"], s["kscale"], k), (s["v8"], s["vscale"], v)))
            for g in range(h * G, h * G + G):
                logit = s["q"][a:a + T, g].double() @ k.T / math.sqrt(s["D"])
                logit[:, old + n:][later] = -math.inf
                lse[a:a + T, g] = torch.logsumexp(logit, 1)
                out[a:a + T, g] = torch.softmax(logit, 1) @ v
    return out, lse


def _exact_pack(s):
    two = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=DEV)

    def block(pool):  # [L][n][H][BS][D]
        x = pool.view(s["L"], -1, s["BS"], s["H"], s["D"])[:, s["src"].long()].double().transpose(2, 3)
        top = x.abs().flatten(-2).amax(-1)
        # how many of the powers from 2^-126 on are too small for the block
        n = (448.0 * two[34:] < top[..., None]).sum(-1)
        scale = torch.where(top > 0, two[34 + n], torch.ones_like(top))
        y = x / scale[..., None, None]
        step = two[torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent.long() - 4 + 160]
        return torch.round(y / step) * step, scale

    got = []
    for pool, new in (("kpool", "k8"), ("vpool", "v8")):
        y, e = block(s[pool])
        x = s[new].double()
        x[:, s["dst"].long()] = y
        es = s[new[0] + "scale"].double()
        es[:, s["dst"].long()] = e
        got += [x, es]
    return got[0], got[2], got[1], got[3]
