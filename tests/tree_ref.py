"""The tree-decoding operators in 64 bits, row by row, for the tests: attention of drafted trees,
accumulated attention weight, eviction by it and the commit of an accepted path, each with the bound
its stated arithmetic allows."""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
UBF = 2.0 ** -8    # half a step of bf16, relative


def slots(bt_row, BS, n):
    p = np.arange(n)
    return torch.from_numpy(np.asarray(bt_row)[p // BS].astype(np.int64) * BS + p % BS)


def sees(mask_row, i, T, chain):
    """Which of the T nodes node i sees."""
    if chain:
        return np.arange(T) <= i
    w = np.asarray(mask_row).view(np.uint32)
    return np.array([(int(w[j // 32]) >> (j % 32)) & 1 for j in range(T)], dtype=bool)


def attn(q, kpool, vpool, bt, BS, ctx, q_off, mask, H, scale, bad_blocks=()):
    """(out, lse, out_bound, lse_bound) in fp64.  q [n_q][Hq][D]; pools [n_slots][H][D]."""
    n_q, Hq, D = q.shape
    G = Hq // H
    out = torch.zeros(n_q, Hq, D, dtype=torch.float64)
    ob = torch.zeros_like(out)
    lse = torch.full((n_q, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for r in range(len(ctx)):
        c, T = int(ctx[r]), int(q_off[r + 1] - q_off[r])
        s = slots(bt[r], BS, c + T)
        ok = np.array([int(bt[r][p // BS]) not in bad_blocks for p in range(c + T)], dtype=bool)
        s = torch.where(torch.from_numpy(ok), s, torch.zeros_like(s)) if len(s) else s
        for i in range(T):
            row = int(q_off[r]) + i
            vis = np.concatenate([np.ones(c, bool),
                                  sees(None if mask is None else mask[row], i, T, mask is None)]) & ok
            at = s[torch.from_numpy(np.flatnonzero(vis))]
            if len(at) == 0:
                continue
            for h in range(H):
                k, v = kpool[at, h].double(), vpool[at, h].double()
                qq = q[row, h * G:(h + 1) * G].double()
                z = qq @ k.T * scale
                zabs = (qq.abs() @ k.abs().T * abs(scale)).amax(1)
                ls = torch.logsumexp(z, 1)
                w = torch.exp(z - ls[:, None])
                sl = slice(h * G, (h + 1) * G)
                out[row, sl], lse[row, sl] = w @ v, ls
                # logits: D fp32 products and sums, the scale; weights: ex2 within 2^-22 and
                # the sum of n terms; then one bf16 rounding of each weight and of the result
                ez = (D + 8) * U32 * zabs + 2 * U32 * z.abs().amax(1)
                n = len(at)
                wv = w @ v.abs()
                ob[row, sl] = (UBF + 2 * ez + 2 ** -21 + n * U32)[:, None] * wv + \
                    UBF * out[row, sl].abs() * 1.01 + 1e-30
                lb[row, sl] = ez + 2 ** -21 + n * U32 + 4 * U32 * ls.abs()
    return out, lse, ob, lb


def mass(q, lse, row_idx, row_vis, row_off, kpool, bt, BS, seq, n_mass, old, H, scale, decay,
         bad_blocks=()):
    """(mass, bound).  q [L][n_q][Hq][D], lse [L][n_q][Hq], kpool [L][n_slots][H][D]."""
    L, n_q, Hq, D = q.shape
    G = Hq // H
    got, bound = old.double().clone(), torch.zeros(old.shape, dtype=torch.float64)
    for r in range(len(seq)):
        n = int(seq[r])
        if n == 0:
            continue
        s = slots(bt[r], BS, n)
        ok = torch.tensor([int(bt[r][p // BS]) not in bad_blocks for p in range(n)])
        s = torch.where(ok, s, torch.zeros_like(s))
        rows = range(int(row_off[r]), int(row_off[r + 1]))
        for layer in range(L):
            for h in range(H):
                k = kpool[layer, s, h].double()
                add, err = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
                terms = 0
                for i in rows:
                    x = i if row_idx is None else int(row_idx[i])
                    v = min(int(row_vis[i]), n)
                    if v < 1:
                        continue
                    for g in range(h * G, h * G + G):
                        ls = float(lse[layer, x, g])
                        if ls == -math.inf:
                            continue
                        qq = q[layer, x, g].double()
                        z = k[:v] @ qq * scale
                        w = torch.exp(z - ls) * ok[:v]
                        zabs = k[:v].abs() @ qq.abs() * abs(scale)
                        add[:v] += torch.where(ok[:v], w, torch.zeros_like(w))
                        # the logit, then the exponent z·log2e − lse·log2e in fp32, then ex2
                        e = (D + 8) * U32 * zabs + 4 * U32 * (z.abs() + abs(ls)) + 2 ** -21
                        err[:v] += torch.where(ok[:v], w * e, torch.zeros_like(w))
                        terms += 1
                m = got[layer, r, h, :n]
                m[int(n_mass[r]):] = 0
                m *= decay
                m += add
                bound[layer, r, h, :n] = err + (terms + 4) * U32 * m.abs() + 1e-35
    return got, bound


def evict(kpool, vpool, bt, BS, seq, n_pos, t_end, mass_, pos, H, budget, n_sink, n_recent,
          bad_blocks=()):
    """Everything kvc_mass_evict writes, exactly (numpy arrays in, copies out)."""
    k, v = kpool.copy(), vpool.copy()
    L = k.shape[0]
    mo, po = mass_.copy(), pos.copy()
    n_out = np.minimum(seq, budget)
    for r in range(len(seq)):
        n, np_ = int(seq[r]), min(max(int(n_pos[r]), 0), int(seq[r]))
        for layer in range(L):
            for h in range(H):
                w, o = mass_[layer, r, h, :n], pos[layer, r, h, :n].astype(np.int64)
                o = np.where(np.arange(n) < np_, o, int(t_end[r]) - (n - np.arange(n)))
                po[layer, r, h, :min(n, budget)] = o[:budget]
                mo[layer, r, h, :min(n, budget)] = w[:budget]
                if n <= budget:
                    continue
                pin = (o < n_sink) | (o >= int(t_end[r]) - n_recent)
                # pinned first, then weight descending (NaN last), then the lower row
                rank = sorted(range(n), key=lambda i: (
                    not pin[i], not pin[i] and math.isnan(w[i]),
                    0.0 if pin[i] or math.isnan(w[i]) else -float(w[i]), i))
                stay = np.zeros(n, bool)
                stay[rank[:budget]] = True
                holes = np.flatnonzero(~stay[:budget])
                tails = budget + np.flatnonzero(stay[budget:])
                assert len(holes) == len(tails)
                for d, s in zip(holes, tails):
                    mo[layer, r, h, d], po[layer, r, h, d] = w[s], o[s]
                    bd, bs = int(bt[r][d // BS]), int(bt[r][s // BS])
                    if bd in bad_blocks or bs in bad_blocks:
                        continue
                    sd, ss = bd * BS + d % BS, bs * BS + s % BS
                    k[layer, sd, h], v[layer, sd, h] = kpool[layer, ss, h], vpool[layer, ss, h]
    return k, v, mo, po, n_out


def tree_masks(rng, T, words, kind):
    """uint32 [T][words]: a random tree's ancestors and self, or one of the masks to go wrong on."""
    anc = np.zeros((T, words * 32), bool)
    for j in range(T):
        if kind == "empty":
            continue
        anc[j, j] = kind != "noself"
        if kind == "full":
            anc[j, :T] = True
        elif j and kind != "self":
            p = int(rng.integers(0, j))
            anc[j] |= anc[p]
            anc[j, p] = True
    if kind == "holes":      # padded nodes: nobody sees them and they see nothing
        dead = rng.random(T) < 0.4
        anc[:, :T][:, dead] = False
        anc[dead] = False
    return np.packbits(anc.reshape(T, words, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
