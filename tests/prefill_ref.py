"""Filling the paged cache and reading its 8-bit part, in 64 bits, for the tests: norms and rotation
with the way into the cache, causal attention of packed prompts, blocks in e4m3 and attention over
them, each with the bound its stated arithmetic allows."""
from __future__ import annotations

import math

import numpy as np
import torch

from tree_ref import U32, UBF, sees, slots

UH = 2.0 ** -11   # half a step of fp16, relative


def rope_table(n_pos, D, theta=1e6):
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * \
        theta ** (-2.0 / D * torch.arange(D // 2, dtype=torch.float64))
    return torch.stack([a.cos(), a.sin()], -1).float()


def normed(x, w, eps):
    """x [..][D] under the norm (w None: as it is), and what fp32 may make of it, relative."""
    x = x.double()
    if w is None:
        return x, 0.0
    D = x.shape[-1]
    # a sum of D squares, mean + eps, a root, a quotient, two products
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double(), (D / 2 + 8) * U32


def rotated(y, rel, tab):
    """(want, bound) of the rotation by table rows tab [n][D/2][2], y [n][heads][D], one bf16 rounding."""
    h = y.shape[-1] // 2
    c, s = tab[..., 0].double()[:, None], tab[..., 1].double()[:, None]
    a, b = y[..., :h], y[..., h:]
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    size = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    e = (rel + 2 * U32) * size
    return want, e + UBF * (want.abs() + e) + 1e-38


def prompt(q, kpool, vpool, bt, BS, ctx, q_off, H, scale, bad_blocks=()):
    """(out, lse, out_bound, lse_bound): kvc_tree_attn's bounds (tree_ref.attn), rows taken together."""
    n_q, Hq, D = q.shape
    G = Hq // H
    out = torch.zeros(n_q, Hq, D, dtype=torch.float64)
    ob = torch.zeros_like(out)
    lse = torch.full((n_q, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for r in range(len(ctx)):
        c, a, b = int(ctx[r]), int(q_off[r]), int(q_off[r + 1])
        T = b - a
        if T == 0:
            continue
        s = slots(bt[r], BS, c + T)
        ok = torch.tensor([int(bt[r][p // BS]) not in bad_blocks for p in range(c + T)])
        s = torch.where(ok, s, torch.zeros_like(s))
        see = (torch.arange(c + T) <= c + torch.arange(T)[:, None]) & ok
        for h in range(H):
            k, v = kpool[s, h].double(), vpool[s, h].double()
            k, v = (torch.where(ok[:, None], x, torch.zeros_like(x)) for x in (k, v))
            for g in range(h * G, h * G + G):
                qq = q[a:b, g].double()
                out[a:b, g], lse[a:b, g], ob[a:b, g], lb[a:b, g] = _rows(qq, k, v, see, scale, UBF)
    return out, lse, ob, lb


def _rows(qq, k, v, see, scale, weight):
    D = qq.shape[1]
    z = torch.where(see, qq @ k.T * scale, torch.full(see.shape, -math.inf, dtype=torch.float64))
    zabs = torch.where(see, qq.abs() @ k.abs().T * abs(scale), torch.zeros_like(z)).amax(1)
    ls = torch.logsumexp(z, 1)
    none = ls == -math.inf
    w = torch.where(see, torch.exp(z - torch.where(none, torch.zeros_like(ls), ls)[:, None]), torch.zeros_like(z))
    n = see.sum(1)
    ez = (D + 8) * U32 * zabs + 2 * U32 * torch.where(see, z.abs(), torch.zeros_like(z)).amax(1)
    o = w @ v
    ob = (weight + 2 * ez + 2 ** -21 + n * U32)[:, None] * (w @ v.abs()) + UBF * o.abs() * 1.01 + 1e-30
    lb = ez + 2 ** -21 + n * U32 + 4 * U32 * torch.where(none, torch.zeros_like(ls), ls).abs()
    return o, ls, ob, lb


def e4m3(y):
    """Nearest e4m3 value of |y| ≤ 448, even on ties."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.round(y / step) * step


def pack(pool, src, BS):
    """Blocks [n][L][H][BS][D] in 64 bits as they are to be stored, and their scales [n][L][H]."""
    L, n_slots, H, D = pool.shape
    x = pool.double().numpy().reshape(L, n_slots // BS, BS, H, D)[:, src].transpose(1, 0, 3, 2, 4)
    mag = np.where(np.isfinite(x), np.abs(x), 0)
    top = mag.max((-2, -1))
    scale = np.ones(top.shape)
    for at in np.ndindex(top.shape):
        if top[at] > 0:
            e = -126
            while 448.0 * 2.0 ** e < top[at]:
                e += 1
            scale[at] = 2.0 ** e
    y = x / scale[..., None, None]
    with np.errstate(invalid="ignore"):
        y = np.where(np.isinf(x), np.sign(x) * 448.0, e4m3(np.where(np.isfinite(y), y, 0)))
    return np.where(np.isnan(x), np.nan, y), scale


def q8(q, k8, v8, ks, vs, t8, len8, kpool, vpool, bt, BS, ctx, q_off, mask, H, scale, bad_blocks=(),
       bad_blocks8=()):
    """(out, lse, out_bound, lse_bound).  k8, v8 [n_blocks8][H][BS][D] values; ks, vs [n_blocks8][H]."""
    n_q, Hq, D = q.shape
    G = Hq // H
    out = torch.zeros(n_q, Hq, D, dtype=torch.float64)
    ob = torch.zeros_like(out)
    lse = torch.full((n_q, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for r in range(len(ctx)):
        n, c, a, T = int(len8[r]), int(ctx[r]), int(q_off[r]), int(q_off[r + 1] - q_off[r])
        p8 = [p for p in range(n) if int(t8[r][p // BS]) not in bad_blocks8]
        blk = torch.tensor([int(t8[r][p // BS]) for p in p8], dtype=torch.long)
        off = torch.tensor([p % BS for p in p8], dtype=torch.long)
        ok = np.array([int(bt[r][p // BS]) not in bad_blocks for p in range(c + T)], dtype=bool)
        s = slots(bt[r], BS, c + T)
        s = torch.where(torch.from_numpy(ok), s, torch.zeros_like(s)) if len(s) else s
        for i in range(T):
            row = a + i
            vis = np.concatenate([np.ones(c, bool),
                                  sees(None if mask is None else mask[row], i, T, mask is None)]) & ok
            at = s[torch.from_numpy(np.flatnonzero(vis))]
            if len(at) + len(p8) == 0:
                continue
            for h in range(H):
                sv = torch.cat([vs[blk, h].double(), torch.ones(len(at), dtype=torch.float64)])
                k = torch.cat([k8[blk, h, off].double() * ks[blk, h].double()[:, None], kpool[at, h].double()])
                u = torch.cat([v8[blk, h, off].double(), vpool[at, h].double()])
                v = u * sv[:, None]
                sl = slice(h * G, (h + 1) * G)
                qq = q[row, sl].double()
                z = qq @ k.T * scale
                zabs = (qq.abs() @ k.abs().T * abs(scale)).amax(1)
                ls = torch.logsumexp(z, 1)
                w = torch.exp(z - ls[:, None])
                o = w @ v
                out[row, sl], lse[row, sl] = o, ls
                cnt = len(sv)
                # logits: D products and sums, the scales; then the exponent's log2 s_v
                ez = (D + 10) * U32 * zabs + 4 * U32 * z.abs().amax(1)
                lg = float(sv.log2().abs().max()) * 2 * U32 + 2 ** -21
                half = torch.full_like(sv, UBF)
                half[:len(p8)] = UH
                ob[row, sl] = (w * half) @ v.abs() + \
                    (2 * ez + lg + 2 ** -20 + cnt * U32)[:, None] * (w @ v.abs()) + \
                    UBF * o.abs() * 1.01 + 1e-30
                if len(p8):  # weights below fp16's normal range
                    ob[row, sl] += 2 ** -25 * (w * sv).amax(1)[:, None] * u[:len(p8)].abs().sum(0)
                lb[row, sl] = ez + 2 ** -21 + cnt * U32 + 4 * U32 * ls.abs()
    return out, lse, ob, lb
