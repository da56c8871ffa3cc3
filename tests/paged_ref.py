"""Plain definitions, in 64 bits on the CPU, of the paged-cache operators, and the error bounds the tests hold the
kernels to. Nothing here is shared with the library.

Error bounds. Let h be half a step of the 16-bit type (finfo.eps / 2) and u = 2^-24 that of fp32. A result y is rounded
once: h |y| (or half the smallest subnormal). A rotation is two fp32 products and one sum: at most 3 u (|a c| + |b s|). A
score is a sum of D fp32 products in an order and with an intermediate rounding that the tensor cores leave open (at most
one unit in the last place, 2 u, per addition): its error is at most ds = (2 D + 8) u scale sum_d |q_d k_d|, the last 8 u
covering the scaling and the exponent's argument. Its weight exp(s) is then off by a factor of at most
1 + 2 ds + 2^-21 (the exponential's own error), may be rounded to the 16-bit type before it multiplies V (h), and the two
sums over n keys add 2 (n + 16) u. So |o - o'| <= h |o| + (h + 2 (2 max ds + 2^-21 + 2 (n + 16) u)) sum_j p_j |v_j| and
|lse - lse'| <= max ds + 2^-21 + 2 (n + 16) u + 8 u (|lse| + max |s|). Weights below the type's smallest normal (a factor of
2^-14 under the row's largest for fp16) are rounded to half its smallest subnormal, tiny / 2, instead of h p: at most
n tiny max|v| more.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dt):
    return torch.finfo(dt).eps / 2


def smallest(dt):
    return torch.finfo(dt).tiny * torch.finfo(dt).eps


def positions(kv_lens, new_lens, T):
    """First position of each sequence's new tokens and their number."""
    n = new_lens if new_lens is not None else [T] * len(kv_lens)
    return [(l - m, m) for l, m in zip(kv_lens, n)]


def rotate(x, cos, sin, rot, interleaved):
    """x [..., D] float64, cos and sin [rot / 2] -> rotated, and the bound of an fp32 evaluation's error."""
    y, err = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    err[..., a] = 3 * U32 * ((x[..., a] * cos).abs() + (x[..., b] * sin).abs())
    err[..., b] = 3 * U32 * ((x[..., b] * cos).abs() + (x[..., a] * sin).abs())
    return y, err


def attend(q, k_pool, v_pool, table, kv_lens, scale, causal, window, new_lens=None, sel=None, sel_lens=None):
    """q [B, Hq, T, D] and the pools in any float type on the CPU, table [B, max_pages], lists of lengths.
    -> o, lse in float64 and the bounds of |o - o'| and |lse - lse'|."""
    B, Hq, T, D = q.shape
    P, Hkv, page, _ = k_pool.shape
    h, tiny = half_step(q.dtype), smallest(q.dtype)
    o = torch.zeros(B, Hq, T, D, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    bo, bl = torch.full_like(o, 0.0), torch.zeros_like(lse)
    rep = Hq // Hkv
    for b, (first, n) in enumerate(positions(kv_lens, new_lens, T)):
        length = kv_lens[b]
        pages = -(-length // page)
        for g in range(Hkv):
            chosen = range(pages) if sel is None else [int(x) for x in sel[b, g, : int(sel_lens[b, g])]]
            where = [(int(table[b, p]), p) for p in chosen if 0 <= p < pages]
            where = [(i, p) for i, p in where if 0 <= i < P]
            if not where:
                continue
            j = torch.cat([torch.arange(p * page, (p + 1) * page) for _, p in where])
            k = torch.cat([k_pool[i, g] for i, _ in where]).double()
            v = torch.cat([v_pool[i, g] for i, _ in where]).double()
            for t in range(min(n, T)):
                at = first + t
                see = j < length
                if causal:
                    see &= j <= at
                if window:
                    see &= ~((at >= j) & (at - j >= window))
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                x = q[b, g * rep:(g + 1) * rep, t].double()
                s = scale * (x @ kk.T)
                ds = ((2 * D + 8) * U32 * scale * (x.abs() @ kk.abs().T)).amax(-1)
                lz = torch.logsumexp(s, -1)
                p = torch.exp(s - lz[:, None])
                rows = slice(g * rep, (g + 1) * rep)
                o[b, rows, t] = p @ vv
                lse[b, rows, t] = lz
                sums = 2 * (kk.shape[0] + 16) * U32
                rel = h + 2 * (2 * ds + 2.0 ** -21 + sums)
                top = p.amax(-1)  # weights are held relative to the row's largest
                bo[b, rows, t] = (h * o[b, rows, t].abs() + rel[:, None] * (p @ vv.abs()) + tiny
                                  + (kk.shape[0] * tiny * top)[:, None] * vv.abs().amax())
                bl[b, rows, t] = ds + 2.0 ** -21 + sums + 8 * U32 * (lz.abs() + s.abs().amax(-1))
    return o, lse, bo, bl


def select(q, bounds, table, kv_lens, page, n_sel, keep_first, keep_last, num_pages=None):
    """q [B, Hq, 1, D], bounds [num_pages, Hkv, 2, D] -> sel, sel_lens as lists."""
    B, Hq, _, D = q.shape
    P, Hkv = bounds.shape[:2]
    rep = Hq // Hkv
    sel = torch.full((B, Hkv, n_sel), -1, dtype=torch.int32)
    count = torch.zeros(B, Hkv, dtype=torch.int32)
    for b in range(B):
        pages = -(-kv_lens[b] // page)
        for g in range(Hkv):
            if pages <= n_sel:
                chosen = list(range(pages))
            else:
                x = q[b, g * rep:(g + 1) * rep, 0].double()
                scored = []
                for p in range(keep_first, pages - keep_last):
                    i = int(table[b, p])
                    if not 0 <= i < P:
                        scored.append((1, 0.0, p))  # below every page that is there
                        continue
                    lo, hi = bounds[i, g, 0].double(), bounds[i, g, 1].double()
                    s = torch.maximum(x * lo, x * hi).sum(-1).amax()  # maximum and amax keep NaN
                    scored.append((0, -math.inf if torch.isnan(s) else -float(s), p) if not torch.isnan(s) else (-1, 0.0, p))
                scored.sort()
                middle = [p for _, _, p in scored[: n_sel - keep_first - keep_last]]
                chosen = sorted(list(range(keep_first)) + middle + list(range(pages - keep_last, pages)))
            sel[b, g, : len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            count[b, g] = len(chosen)
    return sel, count
