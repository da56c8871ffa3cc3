"""Edges of the paged-cache operators on the GPU: lists of more items than a CTA holds at a time, rankings full of ties,
scores at the ends of the range, weights whose second word decides, calls that meet a full launch queue."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
import paged_ref
from test_paged_gpu import (attend, bounds_for, check_attend, check_select, gen, handle, i32, make_table, paged_inputs, randn, select,
                            status_clear)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- walks past the window
def scattered(heads, D, dtype, seed=31):
    """3000 sequences, five of them with keys and hundreds without between them: shares of several tiles, so that a CTA
    that comes to the end of one sequence has to look for the next behind many windows of items."""
    B, Hkv, page = 3000, 2, 64
    lens = [0] * B
    for i, n in ((5, 9000), (700, 8970), (705, 9001), (1500, 8999), (2999, 64 * 140 + 1)):
        lens[i] = n
    g = gen(seed)
    mp = 141
    table = torch.zeros(B, mp, dtype=torch.int32)
    live = [i for i in range(B) if lens[i]]
    pool = torch.randperm(len(live) * mp + 2, generator=g)[: len(live) * mp].view(len(live), mp)
    table[live] = pool.to(torch.int32)
    P = len(live) * mp + 2
    k, v = randn(g, P, Hkv, page, D, dtype=dtype), randn(g, P, Hkv, page, D, dtype=dtype)
    return k, v, table, randn(g, B, Hkv * heads, 2, D, dtype=dtype), lens


@pytest.mark.parametrize("heads,D", [(2, 64), (4, 128), (10, 128), (20, 64), (40, 96), (9, 256)])
def test_attend_over_sequences_far_apart(heads, D):
    k, v, table, q, lens = scattered(heads, D, torch.bfloat16)
    new = [2 if i % 3 else 1 for i in range(len(lens))]
    kv = handle(k, v, table, i32(lens))
    o, lse = attend(kv, q, 1 / math.sqrt(D), True, 0, i32(new))
    assert status_clear()
    check_attend(o, lse, paged_ref.attend(q, k, v, table, lens, 1 / math.sqrt(D), True, 0, new))


@pytest.mark.parametrize("heads,D", [(2, 64), (20, 128), (9, 256)])
def test_waits_that_give_up_end_cleanly_in_sequences_far_apart(heads, D):
    import time
    k, v, table, q, lens = scattered(heads, D, torch.bfloat16)
    kv = handle(k, v, table, i32(lens))
    want = attend(kv, q, 0.1)
    assert status_clear()
    fa.fa_set_wait_limit_cycles(8)
    try:
        t = time.time()
        attend(kv, q, 0.1)
        torch.cuda.synchronize()
        assert time.time() - t < 2
        assert fa.fa_device_status() & 1
    finally:
        fa.fa_set_wait_limit_cycles(0)
    o, lse = attend(kv, q, 0.1)
    assert status_clear()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("heads", [2, 20])
def test_attend_more_short_sequences_than_a_window_holds(heads):
    """40000 sequences of one to three tiles in a table 17 pages wide: shares of more than a hundred items."""
    B, page, D, mp = 40000, 64, 64, 17
    g = gen(32)
    kinds = [1, 64, 65, 130, 0]
    P = 40
    k, v = randn(g, P, 1, page, D, dtype=torch.float16), randn(g, P, 1, page, D, dtype=torch.float16)
    kind = torch.arange(B) % 5
    lens = torch.tensor(kinds)[kind]
    table = (kind[:, None] * 7 + torch.arange(mp)[None] % 3).to(torch.int32)  # read only: sequences share pages
    q = randn(g, 5, heads, 1, D, dtype=torch.float16)
    kv = handle(k, v, table, lens.to(torch.int32))
    o, lse = attend(kv, q[kind], 0.125)
    assert status_clear()
    few = paged_ref.attend(q, k, v, table[:5], kinds, 0.125, True, 0)
    o, lse = o.view(-1, 5, heads, 1, D), lse.view(-1, 5, heads, 1)
    for part in (0, o.shape[0] - 1):
        check_attend(o[part], lse[part], few)
    check_attend(o.double().mean(0), lse[0], few)
    assert torch.isfinite(o).all() and (o.float() - o[:1].float()).abs().max() <= 2 * few[2].max()


# ------------------------------------------------------------- lengths written between calls
def test_calls_follow_lengths_written_between_them():
    """Selection and attention over the chosen pages, queued behind writes of the lengths that move sequences between no
    pages, fewer pages than places and many more: each call gives what it gives alone."""
    B, Hq, Hkv, D, page, mp, n_sel = 5, 8, 2, 128, 16, 700, 24
    g = gen(61)
    table, P = make_table(g, B, mp)
    a, b = randn(g, P, Hkv, D, dtype=torch.bfloat16), randn(g, P, Hkv, D, dtype=torch.bfloat16)
    bounds = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2).contiguous()
    k, v = randn(g, P, Hkv, page, D, dtype=torch.bfloat16), randn(g, P, Hkv, page, D, dtype=torch.bfloat16)
    q = randn(g, B, Hq, 1, D, dtype=torch.bfloat16).cuda()
    kv = handle(k, v, table, i32([0] * B), bounds)
    steps = [torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32) for hi in (0, 16, 390, 11200, 400, 11200) * 10]
    steps = torch.stack(steps).cuda()
    wf = torch.empty(fa.fa_paged_workspace_size(Hq, Hkv, 1, D), dtype=torch.uint8, device="cuda")
    ws = torch.empty(fa.fa_page_select_workspace_size(B, Hkv, mp), dtype=torch.uint8, device="cuda")
    sel = torch.empty(B, Hkv, n_sel, dtype=torch.int32, device="cuda")
    count = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")

    def run(apart):
        out = []
        for n in steps:
            kv.kv_lens.copy_(n)
            if apart:
                torch.cuda.synchronize()
            fa.fa_page_select(kv, q, sel, count, keep_first=1, keep_last=2, workspace=ws)
            if apart:
                torch.cuda.synchronize()
            fa.fa_paged_fwd(kv, q, o, lse, 0.1, causal=True, sel=sel, sel_lens=count, workspace=wf)
            out.append([t.clone() for t in (sel, count, o, lse)])
        assert status_clear()
        return out

    for x, y in zip(run(True), run(False)):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
    for n, (s, c, _, _) in list(zip(steps.tolist(), run(False)))[:6]:
        want, wc = paged_ref.select(q.cpu(), bounds, table, n, page, n_sel, 1, 2)
        assert torch.equal(s.cpu(), want) and torch.equal(c.cpu(), wc)


# ------------------------------------------------------------- tiles without a load
@pytest.mark.parametrize("heads,D,page", [(4, 128, 16), (4, 128, 64), (16, 64, 16), (40, 128, 16), (24, 256, 32)])
@pytest.mark.parametrize("n", [900, 40000])
def test_attend_tiles_of_bad_pages_alone(heads, D, page, n):
    """Tiles whose pages are all bad bring no bytes, so that their stage is full as soon as the positions of its keys are
    written: no consumer may take the positions of the tile that held the stage before."""
    k, v, table, q = paged_inputs(1, heads, 1, D, page, 1, [n], torch.bfloat16, seed=41)
    r = torch.Generator().manual_seed(42)
    for t in range(-(-n // 64)):  # about every other tile, in runs
        if (t // 3) % 2 and torch.rand(1, generator=r) < 0.9:
            table[0, t * 64 // page:(t + 1) * 64 // page if page < 64 else t * 64 // page + 1] = -5
    kv = handle(k, v, table, i32([n]))
    ref = paged_ref.attend(q, k, v, table, [n], 0.1, True, 0)
    first = None
    for _ in range(5):
        o, lse = attend(kv, q, 0.1)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 4
        check_attend(o, lse, ref)
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


# ------------------------------------------------------------- rankings full of ties
def tied_inputs(kind, B, pages, dtype, D=128, Hq=4, Hkv=2, seed=71):
    g = gen(seed)
    table, P = make_table(g, B, pages)
    bounds, q = bounds_for(g, P, Hkv, D, dtype), randn(g, B, Hq, 1, D, dtype=dtype)
    if kind == "zero_query":
        q.zero_()
    elif kind == "one_zero_query":
        q[:, :-1].zero_()
    elif kind == "zero_query_bad_pages":
        q.zero_()
        table[:, 5::7] = -1
    elif kind == "bad_pages":
        table[:, 40:] = P
    elif kind == "equal":
        bounds[:] = bounds[:1]
    elif kind == "zero_bounds":
        bounds.zero_()
    elif kind == "classes":
        bounds[:] = bounds[torch.randint(0, 5, (P,), generator=g)]
    elif kind == "nan_bound":
        bounds[int(table[0, 77]), :, :, 3] = float("nan")
    elif kind == "infinite_bounds":
        bounds[int(table[0, 77]), :, 1, 3] = math.inf
        bounds[int(table[0, 78]), :, 0, 3] = -math.inf
        bounds[int(table[0, 79])] = -math.inf
        bounds[int(table[0, 80])] = math.inf
    elif kind == "nan_query":
        q[..., 5] = float("nan")
    elif kind == "infinite_query":
        q[..., 5] = math.inf
    elif kind == "cancelling":  # large parts that cancel in every page, in another order each; a small rest decides
        big = randn(g, D // 2 - 4, dtype=dtype) * 256
        for i in range(P):
            perm = torch.randperm(D - 8, generator=g)
            x = torch.cat([torch.cat([big, -big])[perm], (randn(g, 8, dtype=dtype) * 2.0 ** -10).to(dtype)])
            bounds[i, :, 0] = bounds[i, :, 1] = x
        q.fill_(1.0)
    return q, bounds, table


KINDS = ["zero_query", "one_zero_query", "zero_query_bad_pages", "bad_pages", "equal", "zero_bounds", "classes", "nan_bound",
         "infinite_bounds", "nan_query", "infinite_query", "cancelling"]


@pytest.mark.parametrize("B", [1, 11])  # few and many blocks
@pytest.mark.parametrize("kind", KINDS)
def test_select_more_ties_than_are_ranked_directly(kind, B):
    lens = [16 * 700 - 3] + [16 * (90 * i % 640) + 7 for i in range(1, B)]
    for dtype, D in ((torch.bfloat16, 128), (torch.float16, 96)):
        q, bounds, table = tied_inputs(kind, B, 700, dtype, D)
        for n_sel in (3, 333):
            check_select(q, bounds, table, lens, 16, n_sel, 1, 1)
        fa.fa_device_status()


@pytest.mark.parametrize("kind", ["zero_query", "classes", "nan_bound"])
def test_select_ties_beyond_shared_memory(kind):
    """More pages than scores are held of, and more query heads than are held at a time."""
    for Hq in (2, 40):
        q, bounds, table = tied_inputs(kind, 1, 13000, torch.bfloat16, D=64 if Hq == 2 else 256, Hq=Hq, Hkv=1)
        pool = torch.zeros(bounds.shape[0], 1, 16, q.shape[3], dtype=q.dtype)
        kv = handle(pool, pool, table, i32([16 * 13000]), bounds)
        sel, count = select(kv, q, 500, 0, 1)
        assert int(count[0, 0]) == 500
        b = bounds[table[0].long(), 0].double()
        x = q[0, :, 0].double()
        score = torch.maximum(x[:, None] * b[None, :, 0], x[:, None] * b[None, :, 1]).sum(-1).amax(0)[:-1]
        score = torch.where(score.isnan(), math.inf, score)
        want = torch.sort(torch.argsort(score, descending=True, stable=True)[:499]).values.tolist() + [12999]
        assert sel[0, 0].tolist() == want


@pytest.mark.parametrize("kind,most", [("zero_query", 4), ("equal", 40), ("nan_bound", 40)])
def test_select_ties_take_no_milliseconds(kind, most):
    """A padded sequence's query is zeros: its pages all tie, and its choice must not keep the batch waiting. (With a 64-bit
    score for every page the factor was 100 and more.)"""
    def time(kind):
        q, bounds, table = tied_inputs(kind, 2, 2000, torch.bfloat16, Hq=16, Hkv=4)
        pool = torch.zeros(bounds.shape[0], 4, 16, 128, dtype=q.dtype)
        kv = handle(pool, pool, table, i32([32000, 31000]), bounds)
        q = q.cuda()
        sel = torch.empty(2, 4, 64, dtype=torch.int32, device="cuda")
        count = torch.empty(2, 4, dtype=torch.int32, device="cuda")
        ws = torch.empty(fa.fa_page_select_workspace_size(2, 4, 2000), dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(5):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(20):
                fa.fa_page_select(kv, q, sel, count, keep_first=1, keep_last=2, workspace=ws)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times)

    assert time(kind) < most * time("ordinary")


# ------------------------------------------------------------- scores at the ends of the range
@pytest.mark.parametrize("exponent", [-60, -66, -70, -72, -73, -74, -76, -80])
@pytest.mark.parametrize("pages", [200, 600])
def test_select_tiny_scores_as_in_64_bits(exponent, pages):
    """bf16 products below fp32's normal numbers, down to where all of them vanish there: the choice stays the one that
    scores in 64 bits give, with the place cut in the middle of the ranking."""
    for seed in range(4):
        g = gen(seed)
        table, P = make_table(g, 2, pages)
        bounds = (bounds_for(g, P, 1, 128, torch.float32) * 2.0 ** exponent).to(torch.bfloat16)
        q = (randn(g, 2, 2, 1, 128, dtype=torch.float32) * 2.0 ** exponent).to(torch.bfloat16)
        check_select(q, bounds, table, [16 * pages, 8 * pages + 1], 16, pages // 3, 0, 0)
    assert status_clear()


LARGE = [  # value of the query, of the keys, scale; scores from 5e6 to near what fp32 holds, of both signs
    ("fp16", 300.0, 303.0, 1.0), ("fp16", 3000.0, 3030.0, 1.0), ("fp16", 3000.0, -3030.0, 0.125),
    ("fp16", 30000.0, 30310.0, 1.0), ("fp16", 30000.0, -30310.0, 0.3), ("fp16", 65504.0, 65504.0, 1.0),
    ("bf16", 2.0 ** 20, 2.0 ** 24 * 1.25, 0.7), ("bf16", 2.0 ** 40, -2.0 ** 41, 0.7),
    ("bf16", 1.28125 * 2.0 ** 60, 2.0 ** 61, 1.0), ("bf16", 1.28125 * 2.0 ** 60, -2.0 ** 61, 1.0),
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{c[0]}_{c[1]:.3g}_{c[2]:.3g}")
@pytest.mark.parametrize("heads,n,D", [(4, 1, 64), (4, 300, 64), (4, 40000, 64), (12, 30000, 64), (24, 9000, 64), (40, 300, 64), (40, 20000, 64),
                                       (100, 20000, 64), (40, 17003, 64)])
def test_attend_large_scores(case, heads, n, D):
    """Keys that are all alike, with scores whose fp32 steps are 1/2 and much more: whatever the scores are rounded to, all
    weights are equal, so O is the mean of V up to the rounding of its sum and its own (2 (n + 16) u and h), and LSE is
    score + ln n up to what 64 products, the scaling and the logarithm's two roundings leave."""
    dt, x, y, scale = case
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    page = 64
    g = gen(n + heads)
    P = -(-n // page) + 1
    k = torch.full((P, 1, page, D), float("nan"), dtype=dtype)
    v = torch.full((P, 1, page, D), float("nan"), dtype=dtype)
    table = torch.randperm(P, generator=g)[: P - 1].view(1, -1).to(torch.int32)
    for p in range(P - 1):
        m = min(page, n - p * page)
        k[int(table[0, p]), :, :m] = y
        v[int(table[0, p]), :, :m] = randn(g, 1, m, D, dtype=dtype)
    q = torch.full((1, heads, 1, D), x, dtype=dtype)
    o, lse = attend(handle(k, v, table, i32([n])), q, scale)
    assert status_clear()
    vv = torch.cat([v[int(p), 0] for p in table[0]])[:n].double()
    u, h = 2.0 ** -24, torch.finfo(dtype).eps / 2
    want = vv.mean(0)
    bound = h * want.abs() + 2 * (n + 16) * u * vv.abs().mean(0) * (1 + h) + torch.finfo(dtype).tiny
    assert ((o[0, :, 0].double().cpu() - want).abs() <= bound).all()
    s = float(torch.tensor(x, dtype=dtype).double() * torch.tensor(y, dtype=dtype).double()) * D * scale
    assert (lse.double().cpu() - (s + math.log(n))).abs().max() <= (2 * D + 16) * u * abs(s)


@pytest.mark.parametrize("heads,n", [(4, 200), (4, 40000), (40, 20000)])
def test_attend_large_scores_that_differ(heads, n):
    """The one key in a hundred with the largest scores has all the weight, wherever it stands."""
    D, page = 128, 32
    g = gen(heads)
    P = -(-n // page)
    k = torch.full((P, 1, page, D), 20000.0, dtype=torch.float16)
    v = randn(g, P, 1, page, D, dtype=torch.float16)
    top = torch.randperm(n, generator=g)[: max(1, n // 100)]
    k.view(P * page, D)[top] = 20100.0
    q = torch.full((1, heads, 1, D), 20000.0, dtype=torch.float16)
    o, lse = attend(handle(k, v, torch.arange(P, dtype=torch.int32).view(1, P), i32([n])), q, 0.5)
    assert status_clear()
    vv = v.view(P * page, D)[top].double()
    want, u, h = vv.mean(0), 2.0 ** -24, 2.0 ** -11
    assert ((o[0, :, 0].double().cpu() - want).abs() <= h * want.abs() + 2 * (n + 16) * u * vv.abs().mean(0) + 2.0 ** -24).all()


# ------------------------------------------------------------- the host's side
@pytest.mark.parametrize("call", ["append", "attend", "select"])
def test_other_threads_run_while_a_call_waits_for_the_queue(call):
    """With the queue of launches full behind a long kernel a call waits. Another thread goes on meanwhile."""
    import threading
    import time
    g = gen(51)
    table, P = make_table(g, 1, 4)
    bounds = bounds_for(g, P, 1, 64, torch.bfloat16)
    k, v = randn(g, P, 1, 16, 64, dtype=torch.bfloat16), randn(g, P, 1, 16, 64, dtype=torch.bfloat16)
    kv = handle(k, v, table, i32([60]), bounds)
    q = randn(g, 1, 1, 1, 64, dtype=torch.bfloat16).cuda()
    o, lse = torch.empty_like(q), torch.empty(1, 1, 1, device="cuda")
    sel, count = torch.empty(1, 1, 2, dtype=torch.int32, device="cuda"), torch.empty(1, 1, dtype=torch.int32, device="cuda")
    wf = torch.empty(fa.fa_paged_workspace_size(1, 1, 1, 64), dtype=torch.uint8, device="cuda")
    ws = torch.empty(fa.fa_page_select_workspace_size(1, 1, 4), dtype=torch.uint8, device="cuda")
    run = {"append": lambda: fa.fa_kv_append(kv, q, q), "attend": lambda: fa.fa_paged_fwd(kv, q, o, lse, 0.1, workspace=wf),
           "select": lambda: fa.fa_page_select(kv, q, sel, count, workspace=ws)}[call]
    run()
    torch.cuda.synchronize()
    gap, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0] = max(gap[0], now - last)
            last = now

    t = threading.Thread(target=tick)
    t.start()
    try:
        time.sleep(0.05)
        gap[0] = 0.0
        begin = time.perf_counter()
        torch.cuda._sleep(int(0.4e9 * 2))  # cycles: about 0.4 s
        for _ in range(3000):
            run()
        took = time.perf_counter() - begin
    finally:
        stop.set()
        t.join()
    assert status_clear()
    assert took > 0.2, "the queue was never full: nothing was tested"
    assert gap[0] < 0.5 * took


# ------------------------------------------------------------- weights in two words
def weights_that_round_alike(dtype):
    """A key whose weight exp(x) beside weights of 1 is as far from the type's numbers as can be: -> x, exp(x), the weight
    rounded to the type."""
    step = torch.finfo(dtype).eps / 2  # below 1
    xs = torch.linspace(-0.9 * step, -0.1 * step, 400).to(dtype).unique()
    w = xs.double().exp()
    i = (w.to(dtype).double() - w).abs().argmax()
    return float(xs[i]), float(w[i]), float(w[i].to(dtype))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,heads,D,n", [(1, 4, 128, 256), (1, 12, 64, 500), (1, 4, 128, 30000), (1, 16, 256, 20000), (1, 40, 128, 300),  # warps
                                         (80, 20, 128, 1100), (80, 40, 64, 1100), (80, 100, 96, 1100), (40, 40, 256, 2100)])  # tcgen05
def test_attend_weights_keep_their_second_word(dt, B, heads, D, n):
    """Every other key has the weight w < 1 and V = -1, the others 1 and V = 1: O = (1 - w) / (1 + w), next to nothing, and
    all weights w round alike. With the weights' first word alone O would be off by about (1 - w) / 2 or w's rounding.

    Bound. Both words hold w up to 2^-17 (bf16) or 2^-22 (fp16: and half its smallest number); its exponential is off by
    2^-21 w and the score's by (2 D + 8) u |x| w. Partial sums of O are at most 64 of one sign beyond what cancels, n (1 - w) / 2
    in all, so n additions of 2 u each leave 2 u (64 + n (1 - w) / 2) n over a sum of weights of n (1 + w) / 2; joins a few u."""
    dtype = torch.float16 if dt == "fp16" else torch.bfloat16
    x, w, rounded = weights_that_round_alike(dtype)
    page, mp = 64, -(-n // 64)
    k = torch.zeros(mp, 1, page, D, dtype=dtype)
    v = torch.ones(mp, 1, page, D, dtype=dtype)
    k[:, :, 1::2, 0] = x
    v[:, :, 1::2] = -1
    q = torch.zeros(B, heads, 1, D, dtype=dtype)
    q[..., 0] = 1
    o, lse = attend(handle(k, v, torch.arange(mp, dtype=torch.int32).repeat(B, 1), i32([n] * B)), q, 1.0)
    assert status_clear()
    ones, ws = (n + 1) // 2, n // 2
    want = (ones - ws * w) / (ones + ws * w)
    u, h = 2.0 ** -24, torch.finfo(dtype).eps / 2
    second = 2.0 ** -17 if dt == "bf16" else 2.0 ** -22 + 2.0 ** -24
    bound = h * abs(want) + second + 2.0 ** -20 + (2 * D + 8) * u * abs(x) + 4 * u * (64 + n * (1 - w) / 2) + 16 * u
    one_word = (ones - ws * rounded) / (ones + ws * w)
    assert abs(one_word - want) > 5 * bound  # the oracle with one word does not pass
    assert (o.double().cpu() - want).abs().max() <= bound
    assert (lse.double().cpu() - math.log(ones + ws * w)).abs().max() <= 2.0 ** -20 + 2 * (n + 16) * u


# ------------------------------------------------------------- masks over what is not there
@pytest.mark.parametrize("B,heads,D,n", [(1, 4, 128, 700), (1, 4, 64, 30000), (1, 16, 128, 700), (80, 12, 64, 1100), (80, 30, 96, 1100), (40, 10, 256, 2100)])
@pytest.mark.parametrize("window", [1, 100, 900, 2 ** 31 - 1])
def test_attend_bad_pages_under_windows(B, heads, D, n, window):
    """Drafted tokens, windows from one key to more than there are positions, and pages that are not there among those
    that are seen, hidden and partly hidden."""
    Tq, page = 3, 32
    lens = [n] + [max(1, n - 37 * b) for b in range(1, B)]
    k, v, table, q = paged_inputs(B, heads, 1, D, page, Tq, lens, torch.bfloat16, seed=81)
    r = gen(82)
    table[torch.rand(table.shape, generator=r) < 0.2] = -1
    table[0, (n - 1) // page - 1] = k.shape[0]
    kv = handle(k, v, table, i32(lens))
    for causal in (True, False):
        o, lse = attend(kv, q, 0.1, causal, window)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 4
        check_attend(o, lse, paged_ref.attend(q, k, v, table, lens, 0.1, causal, window))


@pytest.mark.parametrize("B,heads,D,n", [(1, 4, 128, 300), (1, 4, 128, 40000), (80, 20, 64, 1100), (80, 100, 128, 1100), (40, 40, 256, 2100)])
@pytest.mark.parametrize("scale", [0.01, 3.0])
def test_attend_nan_with_small_and_large_scales(B, heads, D, n, scale):
    """A NaN query row is NaN whatever the scale; a NaN key makes every row that sees it NaN; no other row changes."""
    k, v, table, q = paged_inputs(B, heads, 1, D, 64, 1, [n] * B, torch.bfloat16, seed=83)
    kv = handle(k, v, table, i32([n] * B))
    clean = attend(kv, q, scale)
    q[0, heads // 2, 0, 7] = float("nan")
    o, lse = attend(kv, q, scale)
    row = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    row[0, heads // 2, 0] = True
    assert torch.isnan(o[row]).all() and torch.isnan(lse[row]).all()
    assert torch.equal(o[~row], clean[0][~row]) and torch.equal(lse[~row], clean[1][~row])
    kv.k[int(table[0, 0]), 0, 5, 3] = float("nan")
    o, lse = attend(kv, q, scale)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(o[1:], clean[0][1:]) and torch.equal(lse[1:], clean[1][1:])
    assert status_clear()
