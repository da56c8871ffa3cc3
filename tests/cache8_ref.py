"""Plain definitions, in 64 bits on the CPU, of the cache held in 8 bits, of windows with visible first keys and of page
assignment, and the error bounds the tests hold the kernels to. Nothing here is shared with the library.

Error bounds of attention are those of paged_ref.py with what the held values add. K and V are exact (an e4m3 number times a
power of two, in fp16 and fp32). A bf16 query row is brought to fp16 under a power of two that takes its largest magnitude
to [2^14, 2^15): elements below fp16's normal numbers are off by at most 2^-25, 2^-39 of the largest, so a score by at most
2^-39 scale max|q| sum_d |k_d| more. Weights are held in two fp16 words whatever the queries' type, so the smallest
subnormal of fp16, 2^-24, bounds what a weight may lose relative to the row's largest one: at most n 2^-24 max|v| more.
A page's product is scaled and added in fp32: one more rounding per 16 keys, within the 2 (n + 16) u of the sums.

A held value y of x under the scale s: half a step of e4m3, 2^-4 |x|, or below its normal numbers half of 2^-9 s."""
import math

import torch

import paged_ref
from paged_ref import U32, half_step, smallest

E4M3 = torch.float8_e4m3fn


def scale_for(most):
    """Least power of two s >= 2^-126 with most <= 448 s, for a finite Python number."""
    if most == 0:
        return 2.0 ** -126
    e = math.floor(math.log2(most)) - 10
    while most > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def hold(x):
    """x [..., page, D] of any float type -> e4m3 pages and fp32 scales [...], as one append of whole pages gives them."""
    x = x.double()
    most = torch.where(x.isfinite(), x.abs(), 0.0).amax((-2, -1))
    s = torch.tensor([scale_for(float(m)) for m in most.flatten()], dtype=torch.float64).view(most.shape)
    return round8(x / s[..., None, None]), s.float()


def round8(x):
    """To e4m3, to the nearest and ties to even; what is not finite to NaN. (Exact: |x| <= 448 has 24 bits to round from.)"""
    return torch.where(x.isfinite(), x, float("nan")).float().to(E4M3)


def held_value(pool, scales):
    return pool.double() * scales.double()[..., None, None]


def attend(q, k_pool, v_pool, table, kv_lens, scale, causal, window, sinks, new_lens=None, sel=None, sel_lens=None,
           held=False):
    """paged_ref.attend with first keys that a window leaves visible; the pools in float64, `held`: as the bounds above."""
    B, Hq, T, D = q.shape
    P, Hkv, page, _ = k_pool.shape
    h, tiny = half_step(q.dtype), smallest(q.dtype)
    weight = 2.0 ** -24 if held else tiny
    o = torch.zeros(B, Hq, T, D, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    rep = Hq // Hkv
    for b, (first, n) in enumerate(paged_ref.positions(kv_lens, new_lens, T)):
        length = kv_lens[b]
        pages = -(-length // page)
        for g in range(Hkv):
            chosen = range(pages) if sel is None else [int(x) for x in sel[b, g, : int(sel_lens[b, g])]]
            where = [(int(table[b, p]), p) for p in chosen if 0 <= p < pages]
            where = [(i, p) for i, p in where if 0 <= i < P]
            if not where:
                continue
            j = torch.cat([torch.arange(p * page, (p + 1) * page) for _, p in where])
            k = torch.cat([k_pool[i, g] for i, _ in where])
            v = torch.cat([v_pool[i, g] for i, _ in where])
            for t in range(min(n, T)):
                at = first + t
                see = j < length
                if causal:
                    see &= j <= at
                if window:
                    see &= ~((at >= j) & (at - j >= window) & (j >= sinks))
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                rows = slice(g * rep, (g + 1) * rep)
                x = q[b, rows, t].double()
                s = scale * (x @ kk.T)
                ds = ((2 * D + 8) * U32 * scale * (x.abs() @ kk.abs().T)).amax(-1)
                if held and q.dtype == torch.bfloat16:
                    ds = ds + 2.0 ** -39 * scale * x.abs().amax(-1) * kk.abs().sum(-1).amax()
                lz = torch.logsumexp(s, -1)
                p = torch.exp(s - lz[:, None])
                o[b, rows, t] = p @ vv
                lse[b, rows, t] = lz
                sums = 2 * (kk.shape[0] + 16) * U32
                rel = h + 2 * (2 * ds + 2.0 ** -21 + sums)
                top = p.amax(-1)
                bo[b, rows, t] = (h * o[b, rows, t].abs() + rel[:, None] * (p @ vv.abs()) + tiny
                                  + (kk.shape[0] * weight * top)[:, None] * vv.abs().amax())
                bl[b, rows, t] = ds + 2.0 ** -21 + sums + 8 * U32 * (lz.abs() + s.abs().amax(-1))
    return o, lse, bo, bl


def assign(table, lens, held, free, count, page, T, num_pages, new=None, window=0, sinks=0):
    """Page assignment one page after another, on lists. -> table, held, the stack, pages missing, slots."""
    table, stack = [list(r) for r in table], list(free[:count])
    B, mp = len(table), len(table[0])
    new = new if new is not None else [T] * B
    want = []
    for b in range(B):
        h0, f0, _ = held[b]
        end = -(-lens[b] // page)
        if window:
            head, first = min(end, -(-sinks // page)), max(0, lens[b] - new[b] - window + 1) // page
            if f0 > h0:
                head, first = min(head, h0), max(first, f0)
        else:
            head, first = (min(end, h0), f0) if f0 > h0 else (0, 0)
        want.append((head, max(min(first, end), head), end))

    def pages(h, f, e):
        return [p for p in range(mp) if p < h or f <= p < e]

    for b in range(B):
        for p in pages(*held[b]):
            if p not in pages(*want[b]):
                stack.append(table[b][p])
                table[b][p] = -1
    missing, now = 0, []
    for b in range(B):
        got = []
        for p in pages(*want[b]):
            if p not in pages(*held[b]):
                if not stack:
                    table[b][p] = -1
                    missing += 1
                    continue
                table[b][p] = stack.pop()
            got.append(p)
        head, first, end = want[b]
        if len(got) < len(pages(*want[b])):
            head = min(head, len(got))
            end = first + len(got) - head if len(got) > head else head
            first = min(first, end)
        assert got == pages(head, first, end)
        now.append((head, first, end))
    slots = [[-1] * T for _ in range(B)]
    for b in range(B):
        for t in range(min(new[b], T)):
            pos = lens[b] - new[b] + t
            if pos >= 0 and 0 <= table[b][pos // page] < num_pages:
                slots[b][t] = table[b][pos // page] * page + pos % page
    return table, now, stack, missing, slots


def dense(q, k, v, do, scale, causal, window, sinks):
    """Attention with a window and visible first keys, and its gradients, in float64 on the CPU, with bounds of the errors of
    kernels that hold P and dS in one word of the inputs' type: -> dicts of values and bounds for o, lse, dq, dk, dv.

    With the notation of paged_ref.py: a score is off by ds, the exponential by 2^-21, a sum of n terms by 2 (n + 16) u. P, from
    the stored LSE, is off by a factor e = 2 ds + 2^-21 + |lse error|, and by h and the type's smallest step t / 2 where it is
    rounded; dP by d = 2 (D + 8) u sum |do v|; the D-vector, from the stored O, by sum |do| |o error| + 2 (D + 8) u sum |do o|.
    Hence dS = P (dP - D) by |dS| (e + h) + P (d + that) + t, twice over where P is rounded on the way, and each gradient by
    its operands' errors, its own sums and its rounding."""
    B, Hq, T, D = q.shape
    Hkv, N = k.shape[1:3]
    rep = Hq // Hkv
    h, tiny = half_step(q.dtype), smallest(q.dtype)
    i, j = torch.arange(T)[:, None], torch.arange(N)
    hidden = ((i - j >= window) & (j >= sinks)) if window else torch.zeros(T, N, dtype=torch.bool)
    if causal:
        hidden = hidden | (j > i)
    qd, dd = q.double(), do.double()
    kd, vd = (x.double().repeat_interleave(rep, 1) for x in (k, v))
    s = (scale * (qd @ kd.transpose(-1, -2))).masked_fill(hidden, -math.inf)
    ds = ((2 * D + 8) * U32 * scale * (qd.abs() @ kd.abs().transpose(-1, -2))).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None]).nan_to_num(0.0)
    sums = 2 * (N + 16) * U32
    o = p @ vd
    bo = h * o.abs() + (h + 2 * (2 * ds + 2.0 ** -21 + sums)) * (p @ vd.abs()) + tiny + N * tiny * p.amax(-1, keepdim=True) * vd.abs().amax()
    top = s.masked_fill(hidden, 0.0).abs().amax(-1)
    bl = ds[..., 0] + 2.0 ** -21 + sums + 8 * U32 * (lse.nan_to_num(0.0, 0.0, 0.0).abs() + top)
    dp = dd @ vd.transpose(-1, -2)
    dvec = (dd * o).sum(-1, keepdim=True)
    dsm = p * (dp - dvec)
    e = 2 * ds + 2.0 ** -21 + bl[..., None] + 2 * h
    near = 2 * (D + 8) * U32
    off = near * (dd.abs() @ vd.abs().transpose(-1, -2)) + (dd.abs() * bo).sum(-1, keepdim=True) + near * (dd * o).abs().sum(-1, keepdim=True)
    ep = p * e + tiny * ~hidden
    es = dsm.abs() * (e + h) + p * off * (1 + e) + tiny * (1 + (dp - dvec).abs()) * ~hidden
    sumq = 2 * (T * rep + 16) * U32

    def group(x):
        return x.view(B, Hkv, rep, N, D).sum(2)

    dq, bdq = scale * (dsm @ kd), scale * ((es + sums * dsm.abs()) @ kd.abs())
    dk, bdk = group(scale * (dsm.transpose(-1, -2) @ qd)), group(scale * ((es + sumq * dsm.abs()).transpose(-1, -2) @ qd.abs()))
    dv, bdv = group(p.transpose(-1, -2) @ dd), group((ep + sumq * p).transpose(-1, -2) @ dd.abs())
    values = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    bounds = {"o": bo, "lse": bl, **{n: b + h * (values[n].abs() + b) + tiny for n, b in (("dq", bdq), ("dk", bdk), ("dv", bdv))}}
    return values, bounds
