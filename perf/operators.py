"""Cases of the paged-cache operators: appending keys and values (``append``), attention of new tokens over the cache
(``attend``), and attention over pages that a cheap score selects (``sparse``).

The cache is a pool of pages, k and v [num_pages, Hkv, page, D]; sequence b keeps key j in slot j % page of pool page
page_table[b, j // page], and kv_lens[b] counts its keys, the call's new tokens among them. ``own`` chooses between the
plain torch form of each operator and the library's kernels; both take the same state.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    base = {"op": "", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "T": 1, "L": 1024,
            "ragged": False, "window": 0, "rot": 128, "interleaved": False, "with_q": True, "bounds": False,
            "n_sel": 0, "keep_first": 0, "keep_last": 0}
    cases = [
        # one user's next token: pure latency
        {"name": "append_b1_t1", "op": "append", "L": 1024},
        # a decoding batch of ragged lengths, with the page bounds that the selection reads
        {"name": "append_b96_t1_bounds", "op": "append", "B": 96, "L": 2048, "ragged": True, "bounds": True,
         "dtype": "fp16"},
        # a padded batch of short prompts, partial interleaved rotation, small pages, odd sizes
        {"name": "append_b7_t333_d96", "op": "append", "B": 7, "Hq": 9, "Hkv": 3, "D": 96, "dtype": "fp16", "page": 16,
         "T": 333, "L": 1000, "ragged": True, "rot": 48, "interleaved": True},
        # four long prompts at once
        {"name": "append_b4_t4096_bounds", "op": "append", "B": 4, "T": 4096, "L": 4096, "bounds": True},
        # the short-query shape of the dense path, from a cache
        {"name": "attend_b2_l1024", "op": "attend", "B": 2, "Hq": 8, "Hkv": 2, "dtype": "fp16", "L": 1024},
        # one user at a long context: few rows, all SMs have to share one sequence
        {"name": "attend_b1_l131072", "op": "attend", "L": 131072},
        # a serving batch of ragged lengths over small pages
        {"name": "attend_b64_l8000_ragged", "op": "attend", "B": 64, "L": 8000, "ragged": True, "page": 16},
        # five drafted tokens of each sequence checked at once, odd group size
        {"name": "attend_b13_t5_d64", "op": "attend", "B": 13, "Hq": 21, "Hkv": 3, "D": 64, "dtype": "fp16", "T": 5,
         "L": 4097, "ragged": True, "page": 32},
        # head dim 256 with a sliding window
        {"name": "attend_b16_d256_w4096", "op": "attend", "B": 16, "Hq": 16, "Hkv": 4, "D": 256, "L": 16384,
         "ragged": True, "window": 4096},
        # selection in a short cache of small pages
        {"name": "sparse_b3_l2001_d64", "op": "sparse", "B": 3, "Hq": 12, "Hkv": 4, "D": 64, "dtype": "fp16",
         "page": 16, "L": 2001, "n_sel": 24, "keep_first": 1, "keep_last": 2},
        # one user at a long context
        {"name": "sparse_b1_l131072", "op": "sparse", "L": 131072, "n_sel": 64, "keep_first": 1, "keep_last": 4},
        # a serving batch at long ragged contexts
        {"name": "sparse_b32_l32768_ragged", "op": "sparse", "B": 32, "L": 32768, "ragged": True, "page": 32,
         "n_sel": 128, "keep_first": 1, "keep_last": 2},
    ]
    return [{**base, **c} for c in cases]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm."""

    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "attend", "attend", "sparse"])
    D = rng.choice([64, 96, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    B = log_int(1, 96)
    case = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": rng.choice(["fp16", "bf16"]), "page": page,
            "T": 1, "L": 1, "ragged": rng.random() < 0.6, "window": 0, "rot": D, "interleaved": rng.random() < 0.4,
            "with_q": True, "bounds": False, "n_sel": 0, "keep_first": 0, "keep_last": 0}
    kv_row = B * Hkv * D  # elements of one key of every sequence
    if op == "append":
        case["T"] = 1 if rng.random() < 0.4 else log_int(2, max(2, min(8192, 16384 * 48 * 128 // (B * (Hq + 2 * Hkv) * D))))
        case["L"] = case["T"] + (0 if rng.random() < 0.3 else log_int(1, max(2, min(8192, 2 ** 27 // kv_row))))
        case["rot"] = rng.choice([D, D, D // 2 // 16 * 16])
        case["bounds"] = rng.random() < 0.5
        case["with_q"] = rng.random() < 0.8
    elif op == "attend":
        case["T"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
        most = 64 * 4000 * 1024 * 16 // max(16, Hq // Hkv * case["T"])
        case["L"] = log_int(8, max(16, min(131072, most // kv_row)))
        case["window"] = rng.choice([0, 0, 0, log_int(1, 8192)])
    else:
        case["L"] = log_int(8, max(16, min(131072, 16 * 32768 * 1024 // kv_row * page // 32)))
        case["n_sel"] = log_int(4, max(4, min(256, 32 * 32 * 128 * 1024 // (kv_row * page))))
        case["keep_first"] = rng.choice([0, 1])
        case["keep_last"] = rng.choice([1, 2, 3])
    return case


def _lens(c):
    """Lengths of the sequences, new tokens included; which sequence has which depends on the seed, their set does not."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    return [max(1, min(c["L"], int(c["L"] * (((b + 1) * 0.6180339887498949) % 1.0) + 1))) for b in range(c["B"])]


def _new_lens(c):
    """New tokens of each sequence. In a ragged batch the rest of its T rows are padding: prompts are whole sequences where
    these are shorter than T, drafts have 1 to T tokens."""
    if not c["ragged"] or c["op"] == "append":
        return [min(c["T"], n) for n in _lens(c)]
    return [min(n, 1 + b % c["T"]) for b, n in enumerate(_lens(c))]


def _max_pages(c):
    return -(-c["L"] // c["page"])


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 2 + 1)
    gc = torch.Generator()
    gc.manual_seed(int(seed) * 2 + 1)
    B, Hq, Hkv, D, page, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["T"]
    mp = _max_pages(c)
    order = torch.randperm(B, generator=gc)
    lens = torch.tensor(_lens(c))[order]
    new_lens = torch.tensor(_new_lens(c))[order]
    num_pages = B * mp + 1  # the last page of the pool belongs to no sequence
    table = torch.randperm(num_pages - 1, generator=gc).to(torch.int32).view(B, mp).to(dev)
    s = {"case": dict(c), "page_table": table, "kv_lens": lens.to(torch.int32).to(dev),
         "new_lens": new_lens.to(torch.int32).to(dev) if c["ragged"] else None}

    def randn(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float32, device=dev).to(dt)

    shape = (num_pages, Hkv, page, D)
    if c["op"] == "append":
        s["k_cache"], s["v_cache"] = torch.zeros(shape, dtype=dt, device=dev), torch.zeros(shape, dtype=dt, device=dev)
        # the projection's output: one row per token with the heads of q, k and v side by side, seen as [B, H, T, D]
        qkv = randn(B, T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], dim=2))
        s["q_out"] = torch.empty((B, Hq, T, D), dtype=dt, device=dev)
        if not c["with_q"]:
            s["q"] = s["q_out"] = None
        half = c["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        ang = torch.arange(c["L"], dtype=torch.float64, device=dev)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["k_bounds"] = None
        if c["bounds"]:
            s["k_bounds"] = torch.zeros((num_pages, Hkv, 2, D), dtype=dt, device=dev)
            s["k_bounds"][:, :, 0] = -randn(num_pages, Hkv, D).abs()
            s["k_bounds"][:, :, 1] = randn(num_pages, Hkv, D).abs()
    else:
        # pages differ in their mean key, as text does; slots that no key was written to hold anything, NaN too
        k = torch.randn(shape, generator=g, dtype=torch.float32, device=dev)
        k += 0.7 * torch.randn((num_pages, Hkv, 1, D), generator=g, dtype=torch.float32, device=dev)
        s["k_cache"] = k.to(dt)
        del k
        s["v_cache"] = randn(*shape)
        last = (s["kv_lens"].long() - 1).clamp(min=0)
        phys = table.long().gather(1, (last // page)[:, None])[:, 0]
        unused = torch.arange(page, device=dev)[None] > (last % page)[:, None]
        fill = torch.where(unused, float("nan"), 0.0).to(dt)[:, None, :, None]
        s["k_cache"][phys] += fill
        s["v_cache"][phys] += fill
        s["k_bounds"] = None
        if c["op"] == "sparse":
            kk = s["k_cache"]
            lo = torch.nan_to_num(kk, nan=float("inf")).amin(2)
            hi = torch.nan_to_num(kk, nan=float("-inf")).amax(2)
            s["k_bounds"] = torch.stack([lo, hi], 2).contiguous()
            s["sel"] = torch.empty((B, Hkv, c["n_sel"]), dtype=torch.int32, device=dev)
            s["sel_lens"] = torch.empty((B, Hkv), dtype=torch.int32, device=dev)
        s["q"] = randn(B, Hq, T, D)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        s["scale"] = 1.0 / math.sqrt(D)
    if own:  # what a serving program keeps from call to call: the cache's handle and the workspaces
        import attention_fa_fwd_03_gb300 as fa
        s["kv"] = fa.PagedKV(s["k_cache"], s["v_cache"], table, s["kv_lens"], k_bounds=s["k_bounds"])
        if c["op"] != "append":
            s["ws"] = torch.empty(fa.fa_paged_workspace_size(Hq, Hkv, T, D), dtype=torch.uint8, device=dev)
        if c["op"] == "sparse":
            s["ws_sel"] = torch.empty(fa.fa_page_select_workspace_size(B, Hkv, mp), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"append": _append_own, "attend": _attend_own, "sparse": _sparse_own}[c["op"]](state)
    return {"append": _append, "attend": _attend, "sparse": _sparse}[c["op"]](state)


def _append_own(s):
    import attention_fa_fwd_03_gb300 as fa
    c = s["case"]
    fa.fa_kv_append(s["kv"], s["k"], s["v"], cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"], q=s["q"],
                    q_out=s["q_out"], new_lens=s["new_lens"])
    return _append_outputs(s)


def _append_outputs(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_bounds", "q_out") if s[n] is not None}


def _attend_own(s):
    import attention_fa_fwd_03_gb300 as fa
    fa.fa_paged_fwd(s["kv"], s["q"], s["o"], s["lse"], s["scale"], causal=True, window=s["case"]["window"],
                    new_lens=s["new_lens"], workspace=s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _sparse_own(s):
    import attention_fa_fwd_03_gb300 as fa
    c = s["case"]
    fa.fa_page_select(s["kv"], s["q"], s["sel"], s["sel_lens"], keep_first=c["keep_first"], keep_last=c["keep_last"],
                      workspace=s["ws_sel"])
    fa.fa_paged_fwd(s["kv"], s["q"], s["o"], s["lse"], s["scale"], causal=True, sel=s["sel"], sel_lens=s["sel_lens"],
                    workspace=s["ws"])
    return {"o": s["o"], "lse": s["lse"], "sel": s["sel"], "sel_lens": s["sel_lens"]}


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
    kc, vc, table = s["k_cache"], s["v_cache"], s["page_table"].long()
    dt = kc.dtype
    pos, valid = _positions(s, T)
    at = pos.clamp(min=0)
    cos, sin = s["cos"][at.clamp(max=s["cos"].shape[0] - 1)][:, None], s["sin"][at.clamp(max=s["cos"].shape[0] - 1)][:, None]
    k = _rotate(s["k"].float(), cos, sin, rot, c["interleaved"]).to(dt)
    spare = kc.shape[0] - 1
    logical = (at // page).clamp(max=table.shape[1] - 1)
    phys = torch.where(valid, table.gather(1, logical), spare)
    slot = torch.where(valid, at % page, 0)
    keep = valid[..., None, None]
    kc[phys, :, slot] = torch.where(keep, k.transpose(1, 2), kc[spare, :, 0])
    vc[phys, :, slot] = torch.where(keep, s["v"].transpose(1, 2), vc[spare, :, 0])
    if s["q"] is not None:
        q = _rotate(s["q"].float(), cos, sin, rot, c["interleaved"])
        s["q_out"] = torch.where(valid[:, None, :, None], q, 0.0).to(dt)
    if s["k_bounds"] is not None:
        bounds = s["k_bounds"]
        first = logical[:, :1]
        n_pages = -(-T // page) + 1
        touched = first + torch.arange(n_pages, device=first.device)[None]
        last = (s["kv_lens"].long()[:, None] - 1) // page
        alive = (touched <= last) & (s["kv_lens"].long()[:, None] > 0)
        ids = torch.where(alive, table.gather(1, touched.clamp(max=table.shape[1] - 1)), spare)
        fresh = (touched * page >= pos[:, :1])[..., None, None]  # the page's first slot is among the new tokens
        old = bounds[ids].float()
        rel = (logical - first)[:, :, None, None].expand(-1, -1, *k.shape[1::2])
        kt = k.transpose(1, 2).float()
        lo = torch.where(fresh, math.inf, old[:, :, :, 0]).scatter_reduce(1, rel, torch.where(keep, kt, math.inf), "amin")
        hi = torch.where(fresh, -math.inf, old[:, :, :, 1]).scatter_reduce(1, rel, torch.where(keep, kt, -math.inf), "amax")
        new = torch.stack([lo, hi], 3)
        bounds[ids] = torch.where(alive[..., None, None, None], new, bounds[spare].float()).to(dt)
    return _append_outputs(s)


def _softmax_av(q, k, v, visible, scale):
    """q [..., R, D], k and v [..., N, D] in fp32, visible [..., R, N] -> (o, lse); a row that sees nothing gives 0, -inf."""
    scores = torch.where(visible, (q @ k.transpose(-1, -2)) * scale, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where(visible.any(-2)[..., None], v, 0.0)
    o = torch.where(total > 0, (p @ v) / total, 0.0)
    return o, (m + torch.log(total))[..., 0]


def _attend(s):
    c = s["case"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    table = s["page_table"].long()
    k = s["k_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D).float()
    pos, valid = _positions(s, T)
    j = torch.arange(k.shape[2], device=k.device)
    visible = valid[..., None] & (j <= pos[..., None]) & (j < s["kv_lens"].long()[:, None, None])
    if c["window"]:
        visible = visible & (pos[..., None] - j < c["window"])
    visible = visible[:, None, None].expand(B, Hkv, Hq // Hkv, T, -1).reshape(B, Hkv, Hq // Hkv * T, -1)
    o, lse = _softmax_av(s["q"].float().view(B, Hkv, -1, D), k, v, visible, s["scale"])
    return {"o": o.view(B, Hq, T, D).to(s["q"].dtype), "lse": lse.reshape(B, Hq, T)}


def _sparse(s):
    c = s["case"]
    B, Hq, Hkv, D, page, n_sel = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["n_sel"]
    table, lens = s["page_table"].long(), s["kv_lens"].long()
    mp = table.shape[1]
    q = s["q"].view(B, Hkv, Hq // Hkv, 1, D)
    # scores in 64 bits: which page wins a place is a whole number, and neighbours differ by little
    b = s["k_bounds"][table].transpose(1, 2).double()
    q64 = q.double()
    score = torch.maximum(q64 * b[:, :, None, :, 0], q64 * b[:, :, None, :, 1]).sum(-1).amax(2)
    pages = ((lens + page - 1) // page)[:, None, None]
    p = torch.arange(mp, device=lens.device)
    score = torch.where((p < c["keep_first"]) | (p >= pages - c["keep_last"]), math.inf, score)
    score = torch.where(p < pages, score, -math.inf)
    best = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :n_sel]
    none = torch.iinfo(torch.int32).max
    chosen = torch.sort(torch.where(best < pages, best, none), dim=-1).values
    if mp < n_sel:
        chosen = torch.cat([chosen, torch.full((B, Hkv, n_sel - mp), none, device=p.device)], -1)
    there = chosen < none
    idx = torch.where(there, chosen, 0)
    phys = table[:, None].expand(B, Hkv, mp).gather(2, idx)
    g = torch.arange(Hkv, device=p.device)[None, :, None]
    k = s["k_cache"][phys, g].reshape(B, Hkv, n_sel * page, D).float()
    v = s["v_cache"][phys, g].reshape(B, Hkv, n_sel * page, D).float()
    j = idx[..., None] * page + torch.arange(page, device=p.device)
    visible = (there[..., None] & (j < lens[:, None, None, None])).reshape(B, Hkv, 1, n_sel * page)
    visible = visible.expand(-1, -1, Hq // Hkv, -1)
    o, lse = _softmax_av(q.float()[:, :, :, 0], k, v, visible, s["scale"])
    return {"o": o.view(B, Hq, 1, D).to(s["q"].dtype), "lse": lse.reshape(B, Hq, 1),
            "sel": torch.where(there, chosen, -1).to(torch.int32), "sel_lens": there.sum(-1).to(torch.int32)}


# ------------------------------------------------------------------ the floor
def work(case):
    c = case
    D, Hq, Hkv, T = c["D"], c["Hq"], c["Hkv"], c["T"]
    lens, new = _lens(c), _new_lens(c)
    if c["op"] == "append":
        tokens = sum(new)
        heads = 2 * Hkv + (Hq if c["with_q"] else 0)
        angles = min(max(lens), tokens) * c["rot"] * 4
        touched = sum((n - 1) // c["page"] - (n - m) // c["page"] + 1 for n, m in zip(lens, new))
        bounds = touched * Hkv * 2 * D * 2 if c["bounds"] else 0
        return {"bytes": tokens * heads * D * 2 * 2 + angles + bounds + 4 * touched,
                "flops": tokens * (heads - Hkv) * c["rot"] * 3}
    rows = Hq * T * c["B"]
    small = rows * (4 * D + 4)  # q read, o and lse written
    if c["op"] == "attend":
        keys = sum(min(n, c["window"] + m - 1) if c["window"] else n for n, m in zip(lens, new))
        pairs = sum(min(n, c["window"] or n) * m for n, m in zip(lens, new)) * Hq
        return {"bytes": keys * Hkv * 4 * D + small + 4 * keys // c["page"], "flops": 4 * D * pairs}
    pages = [-(-n // c["page"]) for n in lens]
    keys = sum(min(n, c["n_sel"] * c["page"]) for n in lens)
    return {"bytes": sum(pages) * Hkv * 4 * D + keys * Hkv * 4 * D + small + 4 * sum(pages) + 4 * c["B"] * Hkv * c["n_sel"],
            "flops": 4 * D * Hq * (sum(pages) + keys)}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Sequence by sequence, from the definition, in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "sparse": _exact_sparse}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    page, half = c["page"], c["rot"] // 2
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kb = s["k_bounds"].double() if s["k_bounds"] is not None else None
    qo = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=kc.device) if s["q"] is not None else None
    first = torch.arange(half, device=kc.device) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)

    def turned(x, at):  # [H, n, D] by the angles of positions `at`
        y = x.clone()
        cs, sn = s["cos"][at].double(), s["sin"][at].double()
        y[..., first] = x[..., first] * cs - x[..., second] * sn
        y[..., second] = x[..., first] * sn + x[..., second] * cs
        return y

    for b, (n, m) in enumerate(zip(s["kv_lens"].tolist(),
                                   s["new_lens"].tolist() if s["new_lens"] is not None else [c["T"]] * c["B"])):
        at = torch.arange(n - m, n, device=kc.device)
        k = turned(s["k"][b, :, :m].double(), at)
        stored = k.to(s["k_cache"].dtype).double()
        for p in range((n - m) // page, (n - 1) // page + 1):
            here = (at // page) == p
            phys = int(s["page_table"][b, p])
            kc[phys][:, at[here] % page] = k[:, here]
            vc[phys][:, at[here] % page] = s["v"][b, :, :m].double()[:, here]
            if kb is not None:
                lo, hi = stored[:, here].amin(1), stored[:, here].amax(1)
                if p * page < n - m:
                    lo, hi = torch.minimum(lo, kb[phys, :, 0]), torch.maximum(hi, kb[phys, :, 1])
                kb[phys, :, 0], kb[phys, :, 1] = lo, hi
        if qo is not None:
            qo[b, :, :m] = turned(s["q"][b, :, :m].double(), at)
    return {n: t for n, t in (("k_cache", kc), ("v_cache", vc), ("k_bounds", kb), ("q_out", qo)) if t is not None}


def _exact_rows(q, k, v, scale):
    """q [H, D], k and v [Hkv, N, D] in 64 bits, every key seen."""
    rep = q.shape[0] // k.shape[0]
    sc = torch.einsum("grd,gnd->grn", q.view(k.shape[0], rep, -1), k) * scale
    lse = torch.logsumexp(sc, -1)
    return torch.einsum("grn,gnd->grd", torch.exp(sc - lse[..., None]), v).reshape(q.shape), lse.reshape(-1)


def _exact_attend(s):
    c = s["case"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=o.device)
    new = s["new_lens"].tolist() if s["new_lens"] is not None else [c["T"]] * c["B"]
    for b, (n, m) in enumerate(zip(s["kv_lens"].tolist(), new)):
        pages = s["page_table"][b, : -(-n // c["page"])].long()
        k = s["k_cache"][pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
        v = s["v_cache"][pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
        for t in range(m):
            at = n - m + t
            lo = max(0, at - c["window"] + 1) if c["window"] else 0
            o[b, :, t], lse[b, :, t] = _exact_rows(s["q"][b, :, t].double(), k[:, lo:at + 1], v[:, lo:at + 1], s["scale"])
    return {"o": o, "lse": lse}


def _exact_sparse(s):
    c = s["case"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=o.device)
    rep, page = c["Hq"] // c["Hkv"], c["page"]
    for b, n in enumerate(s["kv_lens"].tolist()):
        count = -(-n // page)
        pages = s["page_table"][b, :count].long()
        for g in range(c["Hkv"]):
            q = s["q"][b, g * rep:(g + 1) * rep, 0].double()
            lo, hi = s["k_bounds"][pages, g, 0].double(), s["k_bounds"][pages, g, 1].double()
            score = (q.clamp(min=0) @ hi.T + q.clamp(max=0) @ lo.T).amax(0)
            if count > c["n_sel"]:
                score[:c["keep_first"]] = math.inf
                score[count - c["keep_last"]:] = math.inf
                chosen = torch.sort(torch.argsort(-score, stable=True)[:c["n_sel"]]).values
            else:
                chosen = torch.arange(count, device=o.device)
            j = (chosen[:, None] * page + torch.arange(page, device=o.device)).flatten()
            k = s["k_cache"][pages[chosen], g].flatten(0, 1)[j < n].double()
            v = s["v_cache"][pages[chosen], g].flatten(0, 1)[j < n].double()
            h = slice(g * rep, (g + 1) * rep)
            o[b, h, 0], lse[b, h, 0] = _exact_rows(q, k[None], v[None], s["scale"])
    return {"o": o, "lse": lse, "sel": None, "sel_lens": None}
