"""Cases of further operators of the attention library: a paged cache held in 8 bits (``append8``, ``attend8``), a sliding
window with first tokens that stay visible (``sink_attend`` over a cache, ``sink_train`` with its gradients), and page tables
and slot maps built from the requests' lengths (``assign``).

The cache is a pool of pages, k and v [num_pages, Hkv, page, D]; sequence b keeps key j in slot j % page of pool page
page_table[b, j // page], and kv_lens[b] counts its keys, the call's new tokens among them. Held in 8 bits (e4m3) a page of a
KV head has one scale, a power of two, for its keys and one for its values: a held value stands for itself times the scale.
``own`` chooses between the plain torch form of each operator and the library's kernels; both take the same state.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    base = {"op": "", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "T": 1, "L": 1024,
            "ragged": False, "window": 0, "sinks": 0, "causal": True, "rot": 128, "interleaved": False, "with_q": True}
    cases = [
        # one user's next token into a cache held in 8 bits: pure latency
        {"name": "append8_b1_t1", "op": "append8", "L": 1000},
        # a padded batch of short prompts: partial interleaved rotation, small pages, odd sizes
        {"name": "append8_b7_t333_d96", "op": "append8", "B": 7, "Hq": 9, "Hkv": 3, "D": 96, "dtype": "fp16", "page": 16,
         "T": 333, "L": 1000, "ragged": True, "rot": 48, "interleaved": True},
        # four long prompts at once
        {"name": "append8_b4_t4096", "op": "append8", "B": 4, "T": 4096, "L": 4096},
        # a short context
        {"name": "attend8_b2_l1024", "op": "attend8", "B": 2, "Hq": 8, "Hkv": 2, "dtype": "fp16", "L": 1024},
        # one user at a long context: few rows, all SMs have to share one sequence
        {"name": "attend8_b1_l131072", "op": "attend8", "L": 131072},
        # a serving batch of ragged lengths over small pages
        {"name": "attend8_b64_l8000_ragged", "op": "attend8", "B": 64, "L": 8000, "ragged": True, "page": 16},
        # five drafted tokens of each sequence checked at once, odd group size, a window with first tokens beside it
        {"name": "attend8_b13_t5_d64_sinks", "op": "attend8", "B": 13, "Hq": 21, "Hkv": 3, "D": 64, "dtype": "fp16", "T": 5,
         "L": 8191, "ragged": True, "page": 32, "window": 2000, "sinks": 5},
        # decoding without end: a window of the last keys and the first page
        {"name": "sink_attend_b16_d256_w4096", "op": "sink_attend", "B": 16, "Hq": 16, "Hkv": 4, "D": 256, "L": 16384,
         "ragged": True, "window": 4096, "sinks": 64},
        # a training step over short, odd sequences
        {"name": "sink_train_b2_t1500_d64", "op": "sink_train", "B": 2, "Hq": 6, "Hkv": 2, "D": 64, "dtype": "fp16",
         "T": 1500, "L": 1500, "window": 300, "sinks": 5},
        # a training step over one long sequence, the windowed benchmark's shape
        {"name": "sink_train_t16384_w4096", "op": "sink_train", "Hq": 16, "Hkv": 2, "T": 16384, "L": 16384, "window": 4096,
         "sinks": 128},
        # a decoding step of a batch: a few sequences begin a page, some pages have left the window
        {"name": "assign_b64_t1", "op": "assign", "B": 64, "L": 8000, "ragged": True, "page": 16, "window": 4096, "sinks": 16},
        # the prompts of a batch, with the slots of all their tokens
        {"name": "assign_b256_t8192", "op": "assign", "B": 256, "T": 8192, "L": 8192, "ragged": True, "page": 16},
    ]
    return [{**base, **c} for c in cases]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm."""

    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append8", "attend8", "attend8", "sink_attend", "sink_train", "assign"])
    D = rng.choice([64, 96, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = Hkv * rep
    B = log_int(1, 96)
    case = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": rng.choice(["fp16", "bf16"]), "page": page,
            "T": 1, "L": 1, "ragged": rng.random() < 0.6, "window": 0, "sinks": 0, "causal": True, "rot": D,
            "interleaved": rng.random() < 0.4, "with_q": True}
    kv_row = B * Hkv * D  # elements of one key of every sequence
    if op == "append8":
        case["T"] = 1 if rng.random() < 0.4 else log_int(2, max(2, min(8192, 16384 * 48 * 128 // (B * (Hq + 2 * Hkv) * D))))
        case["L"] = case["T"] + (0 if rng.random() < 0.3 else log_int(1, max(2, min(8192, 2 ** 27 // kv_row))))
        case["rot"] = rng.choice([D, D, D // 2 // 16 * 16])
        case["with_q"] = rng.random() < 0.8
    elif op in ("attend8", "sink_attend"):
        case["T"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
        most = 64 * 4000 * 1024 * 16 // max(16, rep * case["T"])
        case["L"] = log_int(8, max(16, min(131072, most // kv_row)))
        if op == "sink_attend" or rng.random() < 0.4:
            case["window"] = log_int(1, 8192)
            case["sinks"] = rng.choice([1, 4, log_int(1, 300)])
    elif op == "sink_train":
        case["B"] = log_int(1, 4)
        most = 16 * 16384 * 16384 // (case["B"] * Hq * D // 64)
        case["T"] = log_int(20, min(8192, math.isqrt(most)))
        case["L"] = case["T"] if rng.random() < 0.7 else log_int(20, case["T"])
        case["causal"] = rng.random() < 0.8
        case["window"] = log_int(1, case["T"])
        case["sinks"] = rng.choice([1, 4, log_int(1, 300)])
        case["ragged"] = False
    else:
        case["B"] = log_int(1, 256)
        case["T"] = 1 if rng.random() < 0.5 else log_int(2, 8192)
        case["L"] = case["T"] + (0 if rng.random() < 0.3 else log_int(1, 8192))
        if rng.random() < 0.5:
            case["window"] = log_int(1, 8192)
            case["sinks"] = rng.choice([0, 4, log_int(1, 300)])
    return case


def _lens(c):
    """Lengths of the sequences, new tokens included; which sequence has which depends on the seed, their set does not."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [max(1, min(c["L"], int(c["L"] * (((b + 1) * 0.6180339887498949) % 1.0) + 1))) for b in range(c["B"])]


def _new_lens(c):
    """New tokens of each sequence. In a ragged batch the rest of its T rows are padding: prompts are whole sequences where
    these are shorter than T, drafts have 1 to T tokens."""
    if not c["ragged"] or c["op"] in ("append8", "assign"):
        return [min(c["T"], n) for n in _lens(c)]
    return [min(n, 1 + b % c["T"]) for b, n in enumerate(_lens(c))]


def _max_pages(c):
    return -(-c["L"] // c["page"])


# ------------------------------------------------------------------ inputs
def _power_scale(most):
    """The smallest power of two that brings `most` to 448, the largest e4m3 number, or below; at least 2^-126."""
    m, x = torch.frexp(most)
    return torch.ldexp(torch.ones_like(most), (x - torch.where(m <= 0.875, 9, 8)).clamp(min=-126))


def _held(x):
    """Pages x [..., page, D] in 8 bits with their scales."""
    scale = _power_scale(x.abs().amax((-2, -1)))
    return (x / scale[..., None, None]).to(E4M3), scale


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 2 + 1)
    gc = torch.Generator()
    gc.manual_seed(int(seed) * 2 + 1)
    B, Hq, Hkv, D, page, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["T"]

    def randn(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float32, device=dev)

    if c["op"] == "sink_train":
        s = {"case": dict(c), "q": randn(B, Hq, T, D).to(dt).requires_grad_(), "do": randn(B, Hq, T, D).to(dt)}
        s["k"], s["v"] = (randn(B, Hkv, c["L"], D).to(dt).requires_grad_() for _ in range(2))
        return s
    mp = _max_pages(c)
    order = torch.randperm(B, generator=gc)
    lens = torch.tensor(_lens(c))[order]
    new_lens = torch.tensor(_new_lens(c))[order]
    s = {"case": dict(c), "kv_lens": lens.to(torch.int32).to(dev),
         "new_lens": new_lens.to(torch.int32).to(dev) if c["ragged"] else None}
    if c["op"] == "assign":
        return _prepare_assign(s, lens, new_lens, gc, dev)
    num_pages = B * mp + 1  # the last page of the pool belongs to no sequence
    s["page_table"] = torch.randperm(num_pages - 1, generator=gc).to(torch.int32).view(B, mp).to(dev)
    shape = (num_pages, Hkv, page, D)
    # pages differ in their mean key, as text does, and in their size
    k = randn(*shape)
    k += 0.7 * randn(num_pages, Hkv, 1, D)
    v = randn(*shape) * torch.exp2(randn(num_pages, Hkv, 1, 1).clamp(-2, 2))
    if c["op"] == "sink_attend":
        s["k_cache"], s["v_cache"] = k.to(dt), v.to(dt)
        s["k_scales"] = s["v_scales"] = None
    else:
        (s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"]) = _held(k), _held(v)
    del k, v
    if c["op"] == "append8":
        # the projection's output: one row per token with the heads of q, k and v side by side, seen as [B, H, T, D]; now
        # and then a token is larger than those before it, and the page's scale has to grow
        qkv = randn(B, T, Hq + 2 * Hkv, D) * torch.where(torch.rand((B, T, 1, 1), generator=g, device=dev) < 0.1, 4.0, 1.0)
        s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in qkv.to(dt).split([Hq, Hkv, Hkv], dim=2))
        s["q_out"] = torch.empty((B, Hq, T, D), dtype=dt, device=dev)
        if not c["with_q"]:
            s["q"] = s["q_out"] = None
        half = c["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        ang = torch.arange(c["L"], dtype=torch.float64, device=dev)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        s["q"] = randn(B, Hq, T, D).to(dt)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        s["scale"] = 1.0 / math.sqrt(D)
    if own:  # what a serving program keeps from call to call: the cache's handle and the workspace
        import attention_fa_fwd_03_gb300 as fa
        s["kv"] = fa.PagedKV(s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], k_scales=s["k_scales"],
                             v_scales=s["v_scales"])
        if c["op"] != "append8":
            s["ws"] = torch.empty(fa.fa_paged_workspace_size(Hq, Hkv, T, D), dtype=torch.uint8, device=dev)
    return s


def _prepare_assign(s, lens, new_lens, gc, dev):
    """The state after the step before: every sequence holds the pages of its keys so far, a page more where its first tokens
    or the window would need it no longer, and the rest of the pool is free. `was` keeps it, and each pass starts from it."""
    c = s["case"]
    B, page, mp = c["B"], c["page"], _max_pages(c)
    num_pages = B * mp + 5
    ids = torch.randperm(num_pages, generator=gc)
    old = lens - new_lens
    end = -(-old // page)
    first_key = (lens - new_lens - c["window"] + 1 - page).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    head = torch.minimum(torch.full_like(end, -(-c["sinks"] // page)), end) if c["window"] else torch.zeros_like(end)
    first = torch.maximum(torch.minimum(first_key // page, end), head)
    p = torch.arange(mp)
    held = (p < head[:, None]) | ((p >= first[:, None]) & (p < end[:, None]))
    table = torch.full((B, mp), -1, dtype=torch.int64)
    n = int(held.sum())
    table[held] = ids[:n]
    free = torch.full((num_pages,), -1, dtype=torch.int64)
    free[:num_pages - n] = ids[n:]
    parts = [table.flatten(), torch.stack([head, first, end], 1).flatten(), free, torch.tensor([num_pages - n, 0])]
    s["was"] = torch.cat(parts).to(torch.int32).to(dev)
    s["now"] = s["was"].clone()
    s["page_table"], s["held"], s["free_pages"], s["free_count"] = s["now"].split([t.numel() for t in parts])
    s["page_table"], s["held"] = s["page_table"].view(B, mp), s["held"].view(B, 3)
    s["slots"] = torch.empty((B, c["T"]), dtype=torch.int64, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _append_own, "attend8": _attend_own, "sink_attend": _attend_own, "sink_train": _train_own,
                "assign": _assign_own}[op](state)
    return {"append8": _append, "attend8": _attend, "sink_attend": _attend, "sink_train": _train, "assign": _assign}[op](state)


def _append_own(s):
    import attention_fa_fwd_03_gb300 as fa
    fa.fa_kv_append(s["kv"], s["k"], s["v"], cos=s["cos"], sin=s["sin"], interleaved=s["case"]["interleaved"], q=s["q"],
                    q_out=s["q_out"], new_lens=s["new_lens"])
    return _append_outputs(s)


def _append_outputs(s):
    """The pools in units of their scales, and the scales."""
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales", "q_out") if s[n] is not None}


def _attend_own(s):
    import attention_fa_fwd_03_gb300 as fa
    c = s["case"]
    fa.fa_paged_fwd(s["kv"], s["q"], s["o"], s["lse"], s["scale"], causal=True, window=c["window"], sinks=c["sinks"],
                    new_lens=s["new_lens"], workspace=s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _train_own(s):
    from attention_fa_fwd_03_gb300.autograd import flash_attention
    c = s["case"]
    o = flash_attention(s["q"], s["k"], s["v"], causal=c["causal"], window=c["window"], sinks=c["sinks"])
    dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
    return {"o": o.detach(), "dq": dq, "dk": dk, "dv": dv}


def _assign_own(s):
    import attention_fa_fwd_03_gb300 as fa
    c = s["case"]
    s["now"].copy_(s["was"])
    fa.fa_page_assign(s["page_table"], s["kv_lens"], s["held"], s["free_pages"], s["free_count"], c["page"], c["T"],
                      new_lens=s["new_lens"], window=c["window"], sinks=c["sinks"], slots=s["slots"])
    return _assign_outputs(s)


def _assign_outputs(s):
    """The part of the stack above its count is left out: it holds nothing."""
    n = torch.arange(s["free_pages"].numel(), device=s["slots"].device)
    free = torch.where(n < s["free_count"][0], s["free_pages"], -1)
    return {"page_table": s["page_table"], "held": s["held"], "free_pages": free, "free_count": s["free_count"],
            "slots": s["slots"]}


# ------------------------------------------------------------------ plain forms
def _positions(s, T):
    """Position of each new token and whether it is one (rows behind a sequence's last token are padding), [B, T]."""
    lens = s["kv_lens"].long()[:, None]
    n = s["new_lens"].long()[:, None] if s["new_lens"] is not None else torch.full_like(lens, T)
    t = torch.arange(T, device=lens.device)[None]
    return lens - n + t, t < n


def _rotate(x, cos, sin, rot, interleaved):
    """x [B, H, T, D] in fp32, cos and sin [B, 1, T, rot / 2]."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _append(s):
    c = s["case"]
    T, page, rot = c["T"], c["page"], c["rot"]
    table = s["page_table"].long()
    pos, valid = _positions(s, T)
    at = pos.clamp(min=0, max=s["cos"].shape[0] - 1)
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    # the pages that receive tokens: logical page, pool page, first key among the new ones
    first = (pos[:, :1].clamp(min=0) // page)
    touched = first + torch.arange(-(-T // page) + 1, device=pos.device)[None]
    last = (s["kv_lens"].long()[:, None] - 1) // page
    alive = touched <= last
    spare = s["k_cache"].shape[0] - 1
    ids = torch.where(alive, table.gather(1, touched.clamp(max=table.shape[1] - 1)), spare)  # [B, P]
    j = touched[..., None] * page + torch.arange(page, device=pos.device)  # [B, P, page]
    rel = j - pos[:, :1, None]
    new = (rel >= 0) & (j < s["kv_lens"].long()[:, None, None]) & alive[..., None]
    kept = (rel < 0) & (touched * page < pos[:, :1])[..., None] & alive[..., None]  # keys of the page from before
    rel = rel.clamp(0, T - 1)
    b = torch.arange(c["B"], device=pos.device)[:, None, None]
    for name, x in (("k", _rotate(s["k"].float(), cos, sin, rot, c["interleaved"])), ("v", s["v"].float())):
        cache, scales = s[name + "_cache"], s[name + "_scales"]
        rows = x.transpose(1, 2)[b, rel].transpose(2, 3)  # [B, P, Hkv, page, D]
        most = torch.where(new[:, :, None, :, None], rows.abs(), 0.0).nan_to_num(0.0, 0.0, 0.0).amax((-2, -1))
        was = scales[ids]
        scale = _power_scale(most)
        scale = torch.where(kept.any(-1)[..., None], torch.maximum(scale, was), scale)
        old = cache[ids].float()
        held = torch.where(new[:, :, None, :, None], (rows / scale[..., None, None]),
                           torch.where(kept[:, :, None, :, None], old * (was / scale)[..., None, None], old))
        some = alive[..., None]
        scales[ids] = torch.where(some, scale, was)
        cache.view(torch.uint8)[ids] = torch.where(some[..., None, None], held, old).to(E4M3).view(torch.uint8)
    if s["q"] is not None:
        q = _rotate(s["q"].float(), cos, sin, rot, c["interleaved"])
        s["q_out"] = torch.where(valid[:, None, :, None], q, 0.0).to(s["q_out"].dtype)
    return _append_outputs(s)


def _pages(s, name):
    """Keys or values of every sequence in fp32, [B, Hkv, N, D]."""
    table = s["page_table"].long()
    x = s[name + "_cache"][table] if s[name + "_scales"] is None else s[name + "_cache"].view(torch.uint8)[table].view(E4M3)
    x = x.float()
    if s[name + "_scales"] is not None:
        x = x * s[name + "_scales"][table][..., None, None]
    return x.transpose(1, 2).reshape(table.shape[0], x.shape[2], -1, x.shape[-1])


def _attend(s):
    c = s["case"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    k, v = _pages(s, "k"), _pages(s, "v")
    pos, valid = _positions(s, T)
    j = torch.arange(k.shape[2], device=k.device)
    visible = valid[..., None] & (j <= pos[..., None])
    if c["window"]:
        visible = visible & ((pos[..., None] - j < c["window"]) | (j < c["sinks"]))
    visible = visible[:, None, None].expand(B, Hkv, Hq // Hkv, T, -1).reshape(B, Hkv, Hq // Hkv * T, -1)
    scores = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(-1, -2)) * s["scale"]
    scores = torch.where(visible, scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, 0.0)
    return {"o": o.view(B, Hq, T, D).to(s["q"].dtype), "lse": (m + torch.log(total))[..., 0].reshape(B, Hq, T)}


def _train(s):
    c = s["case"]
    B, Hq, Hkv, D, T, N = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], c["L"]
    rep = Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    q, do = (s[n].detach().float().view(B, Hkv, rep, T, D) for n in ("q", "do"))
    k, v = (s[n].detach().float().view(B, Hkv, 1, N, D) for n in ("k", "v"))
    i, j = torch.arange(T, device=q.device)[:, None], torch.arange(N, device=q.device)
    hidden = (i - j >= c["window"]) & (j >= c["sinks"])
    if c["causal"]:
        hidden = hidden | (j > i)
    p = q @ k.transpose(-1, -2)
    p.mul_(scale).masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    o = p @ v
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = (ds @ k).mul_(scale)
    dk = (ds.transpose(-1, -2) @ q).sum(2).mul_(scale)
    dt = s["q"].dtype
    return {"o": o.view(B, Hq, T, D).to(dt), "dq": dq.view(B, Hq, T, D).to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _assign(s):
    c = s["case"]
    B, T, page, window, sinks = c["B"], c["T"], c["page"], c["window"], c["sinks"]
    s["now"].copy_(s["was"])
    table, free = s["page_table"], s["free_pages"]
    mp = table.shape[1]
    lens = s["kv_lens"].long()
    n = s["new_lens"].long() if s["new_lens"] is not None else torch.full_like(lens, T)
    head0, first0, end0 = s["held"].long().unbind(1)
    # what each sequence has to hold: the pages of its first tokens and those from the first key that the window shows
    end = (lens + page - 1) // page
    if window:
        head = end.clamp(max=-(-sinks // page))
        head = torch.where(first0 > head0, torch.minimum(head, head0), head)  # what was given back does not come again
        first = torch.maximum((lens - n - window + 1).clamp(min=0) // page, torch.where(first0 > head0, first0, 0))
        first = torch.maximum(torch.minimum(first, end), head)
    else:
        head = torch.where(first0 > head0, torch.minimum(end, head0), 0)
        first = torch.where(first0 > head0, torch.maximum(torch.minimum(first0, end), head), 0)
    p = torch.arange(mp, device=lens.device)

    def pages(h, f, e):
        return (p < h[:, None]) | ((p >= f[:, None]) & (p < e[:, None]))

    had, want = pages(head0, first0, end0), pages(head, first, end)
    back, more = had & ~want, want & ~had
    count = s["free_count"][:1].long()
    # given back: on top of the stack, in order of the sequences and their pages; then the new pages from its top
    at = torch.where(back, count + back.flatten().cumsum(0).view(B, mp) - 1, free.numel())
    stack = torch.cat([free, free.new_empty(1)]).scatter_(0, at.flatten(), table.flatten())[:-1]
    total = count + back.sum()
    rank = more.flatten().cumsum(0).view(B, mp) - 1
    there = more & (rank < total)
    table.copy_(torch.where(there, stack[(total - 1 - rank).clamp(0, free.numel() - 1)], torch.where(back | more, -1, table)))
    free.copy_(stack)
    missing = (more & ~there).sum()
    s["free_count"].copy_(torch.stack([(total - more.sum()).clamp(min=0)[0], missing]))
    # (a sequence that got less than it wants holds what it got: the lowest of the pages)
    got = (want & (had | there)).sum(1)
    head = torch.minimum(head, got)
    short = got < want.sum(1)
    end_got = torch.where(got > head, first + got - head, head)
    s["held"].copy_(torch.stack([head, torch.where(short, torch.minimum(first, end_got), first),
                                 torch.where(short, end_got, end)], 1))
    pos, valid = _positions(s, T)
    phys = table.long().gather(1, (pos.clamp(min=0) // page).clamp(max=mp - 1))
    s["slots"].copy_(torch.where(valid & (phys >= 0), phys * page + pos % page, -1))
    return _assign_outputs(s)


# ------------------------------------------------------------------ the floor
def _visible(c, i, n):
    """Keys that a token at position i sees among the first n."""
    upto = min(i + 1, n) if c["causal"] else n
    hidden = max(0, min(i - c["window"] + 1, upto) - c["sinks"]) if c["window"] else 0
    return upto - hidden


def work(case):
    c = case
    D, Hq, Hkv, T, page = c["D"], c["Hq"], c["Hkv"], c["T"], c["page"]
    if c["op"] == "sink_train":
        pairs = sum(_visible(c, i, c["L"]) for i in range(T)) * c["B"] * Hq
        return {"bytes": 2 * D * c["B"] * (4 * Hq * T + 4 * Hkv * c["L"]), "flops": 14 * D * pairs}
    lens, new = _lens(c), _new_lens(c)
    if c["op"] == "assign":
        # lengths, states and stack counts; table entries given and given back, with the stack's; slots
        got = sum(-(-n // page) - -(-(n - m) // page) for n, m in zip(lens, new))
        return {"bytes": c["B"] * (4 + 4 + 24) + 16 * got + 8 * c["B"] * T, "flops": 0}
    if c["op"] == "append8":
        tokens = sum(new)
        angles = min(max(lens), tokens) * c["rot"] * 4
        touched = sum((n - 1) // page - (n - m) // page + 1 for n, m in zip(lens, new))
        q = Hq * 2 * 2 if c["with_q"] else 0
        return {"bytes": tokens * D * (q + 2 * Hkv * 3) + angles + touched * (4 + 2 * 8 * Hkv),
                "flops": tokens * ((Hkv + (Hq if c["with_q"] else 0)) * c["rot"] * 3 + 2 * Hkv * D)}
    held = 2 if c["op"] == "sink_attend" else 1
    rows = Hq * T * c["B"]
    keys = sum(_visible({**c, "causal": True, "window": c["window"] + m - 1 if c["window"] else 0}, n - 1, n)
               for n, m in zip(lens, new))
    pairs = sum(_visible(c, n - m + t, n) for n, m in zip(lens, new) for t in range(m)) * Hq
    return {"bytes": keys * Hkv * 2 * D * held + (8 * Hkv + 4) * (keys // page) + rows * (4 * D + 4), "flops": 4 * D * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Sequence by sequence, from the definition, in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "assign":
        return None
    return {"append8": _exact_append, "attend8": _exact_attend, "sink_attend": _exact_attend,
            "sink_train": _exact_train}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    page, half = c["page"], c["rot"] // 2
    dev = s["kv_lens"].device
    out = {n: s[n].double() for n in ("k_cache", "v_cache", "k_scales", "v_scales")}
    qo = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=dev) if s["q"] is not None else None
    first = torch.arange(half, device=dev) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)

    def turned(x, at):  # [H, n, D] by the angles of positions `at`
        y = x.clone()
        cs, sn = s["cos"][at].double(), s["sin"][at].double()
        y[..., first] = x[..., first] * cs - x[..., second] * sn
        y[..., second] = x[..., first] * sn + x[..., second] * cs
        return y

    for b, (n, m) in enumerate(zip(s["kv_lens"].tolist(),
                                   s["new_lens"].tolist() if s["new_lens"] is not None else [c["T"]] * c["B"])):
        at = torch.arange(n - m, n, device=dev)
        new = {"k": turned(s["k"][b, :, :m].double(), at), "v": s["v"][b, :, :m].double()}
        for pg in range((n - m) // page, (n - 1) // page + 1):
            here = (at // page) == pg
            phys = int(s["page_table"][b, pg])
            old = max(0, min(page, n - m - pg * page))  # keys of the page from before
            for name, x in new.items():
                cache, scales = out[name + "_cache"][phys], out[name + "_scales"][phys]
                # 2^e with amax <= 448 2^e, by counting up from below
                most = x[:, here].abs().amax((1, 2))
                e = torch.floor(torch.log2(most)) - 9
                e = e + (most > 448 * torch.exp2(e)).double()
                e = e + (most > 448 * torch.exp2(e)).double()
                scale = torch.exp2(e.clamp(min=-126))
                if old > 0:
                    scale = torch.maximum(scale, scales)
                    cache[:, :old] *= (scales / scale)[:, None, None]
                cache[:, at[here] % page] = x[:, here] / scale[:, None, None]
                scales.copy_(scale)
        if qo is not None:
            qo[b, :, :m] = turned(s["q"][b, :, :m].double(), at)
    return {n: t for n, t in (*out.items(), ("q_out", qo)) if t is not None}


def _exact_attend(s):
    c = s["case"]
    Hkv, page = c["Hkv"], c["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=o.device)
    new = s["new_lens"].tolist() if s["new_lens"] is not None else [c["T"]] * c["B"]
    for b, (n, m) in enumerate(zip(s["kv_lens"].tolist(), new)):
        pages = s["page_table"][b, : -(-n // page)].long()
        kv = []
        for name in ("k", "v"):
            if s[name + "_scales"] is None:
                x = s[name + "_cache"][pages].double()
            else:
                x = s[name + "_cache"].view(torch.uint8)[pages].view(E4M3).double() * s[name + "_scales"][pages].double()[..., None, None]
            kv.append(x.transpose(0, 1).flatten(1, 2))
        for t in range(m):
            at = n - m + t
            keys = torch.arange(at + 1, device=o.device)
            if c["window"]:
                keys = torch.cat([keys[:c["sinks"]], keys[max(c["sinks"], at + 1 - c["window"]):]])
            q = s["q"][b, :, t].double().view(Hkv, c["Hq"] // Hkv, -1)
            sc = torch.einsum("grd,gnd->grn", q, kv[0][:, keys]) * s["scale"]
            lse[b, :, t] = torch.logsumexp(sc, -1).flatten()
            o[b, :, t] = torch.einsum("grn,gnd->grd", torch.softmax(sc, -1), kv[1][:, keys]).flatten(0, 1)
    return {"o": o, "lse": lse}


def _exact_train(s):
    """Head by head, 1024 queries at a time over the keys that they can see."""
    c = s["case"]
    T, N, W, S, rep = c["T"], c["L"], c["window"], c["sinks"], c["Hq"] // c["Hkv"]
    scale = 1.0 / math.sqrt(c["D"])
    dev = s["q"].device
    out = {n: torch.zeros(s[m].shape, dtype=torch.float64, device=dev) for n, m in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            kk, vv = s["k"][b, h // rep].detach().double(), s["v"][b, h // rep].detach().double()
            for i0 in range(0, T, 1024):
                i1 = min(T, i0 + 1024)
                keys = torch.arange(min(N, i1) if c["causal"] else N, device=dev)
                keys = torch.cat([keys[:S], keys[max(S, i0 - W + 1):]])
                if keys.numel() == 0:
                    continue
                i = torch.arange(i0, i1, device=dev)[:, None]
                seen = ((i - keys < W) | (keys < S)) & ((keys <= i) if c["causal"] else torch.ones_like(keys, dtype=torch.bool))
                q, k, v, do = s["q"][b, h, i0:i1].detach().double(), kk[keys], vv[keys], s["do"][b, h, i0:i1].double()
                sc = ((q @ k.T) * scale).masked_fill(~seen, -math.inf)
                p = torch.nan_to_num(torch.softmax(sc, -1))
                o = p @ v
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True))
                out["o"][b, h, i0:i1] = o
                out["dq"][b, h, i0:i1] = scale * (ds @ k)
                out["dk"][b, h // rep].index_add_(0, keys, scale * (ds.T @ q))
                out["dv"][b, h // rep].index_add_(0, keys, p.T @ do)
    return out
