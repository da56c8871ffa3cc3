"""A sliding window with first keys that stay visible, on the GPU, against the definition in 64 bits: over the paged cache
(bounds of cache8_ref.py), with the pages in between given back."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
import cache8_ref as ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype):
    return torch.randn(shape, generator=g).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def clear():
    torch.cuda.synchronize()
    return fa.fa_device_status() == 0


def paged(kv, q, scale, causal, window, sinks, new_lens=None):
    q = q.cuda()
    o, lse = torch.full_like(q, NAN), torch.full(q.shape[:3], NAN, device="cuda")
    ws = torch.full((fa.fa_paged_workspace_size(q.shape[1], kv.Hkv, q.shape[2], kv.D),), 255, dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(kv, q, o, lse, scale, causal=causal, window=window, sinks=sinks,
                    new_lens=None if new_lens is None else new_lens.cuda(), workspace=ws)
    return o, lse


def check(o, lse, want):
    ro, rl, bo, bl = want
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(lse == -math.inf, rl == -math.inf)
    assert ((o - ro).abs() <= bo).all(), f"O off by {((o - ro).abs() / bo.clamp(min=1e-300)).max():.3g} bounds"
    fin = rl > -math.inf
    assert ((lse - rl).abs()[fin] <= bl[fin]).all()


PAGED = [  # B, Hq, Hkv, D, page, T, lengths, causal, window, sinks, dtype
    (2, 4, 2, 64, 16, 1, [500, 30], True, 100, 1, "fp16"),
    (3, 8, 2, 128, 64, 1, [1000, 0, 65], True, 64, 64, "bf16"),
    (2, 6, 2, 96, 32, 3, [700, 2], True, 33, 5, "bf16"),
    (2, 8, 1, 256, 64, 2, [900, 900], True, 200, 100, "fp16"),
    (1, 32, 1, 128, 16, 1, [5000], True, 1000, 17, "bf16"),         # clusters of many rows
    (1, 4, 4, 128, 64, 1, [40000], True, 30000, 4, "bf16"),         # split list
    (1, 8, 1, 96, 128, 8, [20000], True, 15000, 129, "fp16"),       # split list on tcgen05, a row for each token
    (1, 48, 1, 64, 16, 1, [16000], True, 14000, 30, "bf16"),
    (2, 4, 2, 128, 256, 4, [3000, 257], False, 50, 300, "bf16"),    # later keys visible
    (2, 4, 2, 64, 32, 1, [300, 200], True, 1 << 30, 7, "fp16"),     # a window that hides nothing
    (2, 4, 2, 64, 32, 2, [300, 200], True, 1, 1 << 30, "fp16"),     # first keys beyond the cache: all are
    (2, 4, 2, 64, 32, 8, [8, 9], True, 3, 2, "fp16"),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"B{c[0]}h{c[1]}x{c[2]}d{c[3]}p{c[4]}T{c[5]}w{c[8]}s{c[9]}{c[10]}")
def test_paged_matches_the_definition(case):
    """The table holds no page where neither the window nor the first keys show a key: such pages are not looked at."""
    B, Hq, Hkv, D, page, T, lens, causal, window, sinks, dt = case
    g = gen(D + T + window % 1000)
    mp = -(-max(lens) // page)
    P = B * mp + 2
    table = torch.randperm(P, generator=g)[: B * mp].view(B, mp).to(torch.int32)
    k, v = (randn(g, P, Hkv, page, D, dtype=DT[dt]) for _ in range(2))
    q = randn(g, B, Hq, T, D, dtype=DT[dt])
    given_back = table.clone()
    for b, n in enumerate(lens):
        first = max(0, n - min(T, n) - window + 1) // page
        given_back[b, -(-sinks // page):first] = -1
    kv = fa.PagedKV(k.cuda(), v.cuda(), given_back.cuda(), i32(lens).cuda())
    new = i32([min(T, n) for n in lens])
    o, lse = paged(kv, q, 0.7 / math.sqrt(D), causal, window, sinks, new)
    assert clear()
    check(o, lse, ref.attend(q, k.double(), v.double(), table, lens, 0.7 / math.sqrt(D), causal, window, sinks, new.tolist()))


def test_paged_without_first_keys_is_the_window_alone():
    """sinks = 0, sinks without a window, and the call that knows none give the same bits."""
    g = gen(2)
    B, Hq, Hkv, D, page, L = 2, 8, 2, 128, 64, 3000
    mp = -(-L // page)
    table = torch.randperm(B * mp, generator=g).view(B, mp).to(torch.int32)
    k, v = (randn(g, B * mp, Hkv, page, D, dtype=torch.bfloat16).cuda() for _ in range(2))
    kv = fa.PagedKV(k, v, table.cuda(), i32([L, L - 100]).cuda())
    q = randn(g, B, Hq, 2, D, dtype=torch.bfloat16)
    for window, sinks in ((500, 0), (0, 9), (0, 0)):
        a = paged(kv, q, 0.1, True, window, sinks)
        o, lse = torch.empty_like(q, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        ws = torch.empty(fa.fa_paged_workspace_size(Hq, Hkv, 2, D), dtype=torch.uint8, device="cuda")
        st = fa.library().fa_paged_fwd(kv_struct(kv), q.cuda().data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, 2, 0.1, 1, window,
                                       None, None, None, 0, ws.data_ptr(), ws.numel(), None)
        torch.cuda.synchronize()
        assert st == 0 and clear()
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)


def kv_struct(kv):
    import ctypes
    return ctypes.byref(fa._PagedKVStruct(kv.k.data_ptr(), kv.v.data_ptr(), None, kv.page_table.data_ptr(), kv.kv_lens.data_ptr(),
                                          kv.B, kv.Hkv, kv.D, kv.num_pages, kv.page_size, kv.max_pages,
                                          1 if kv.dtype == torch.bfloat16 else 0))


@pytest.mark.parametrize("rep,T", [(4, 3), (16, 4)])
def test_paged_hidden_keys_hold_anything(rep, T):
    """NaN in keys that the window hides from every row, between first keys and window, in pages that are read for others."""
    g = gen(rep)
    Hkv, D, page, L, window, sinks = 1, 128, 64, 1000, 130, 70
    table = torch.arange(-(-L // page), dtype=torch.int32)[None]
    k, v = (randn(g, table.numel(), Hkv, page, D, dtype=torch.bfloat16) for _ in range(2))
    q = randn(g, 1, rep, T, D, dtype=torch.bfloat16)
    want = ref.attend(q, k.double(), v.double(), table, [L], 0.1, True, window, sinks)
    for x in (k, v):
        x.view(-1, D)[sinks:L - T - window + 1] = NAN
    kv = fa.PagedKV(k.cuda(), v.cuda(), table.cuda(), i32([L]).cuda())
    o, lse = paged(kv, q, 0.1, True, window, sinks)
    assert clear()
    check(o, lse, want)


# ------------------------------------------------------------------ training
DENSE = [  # B, Hq, Hkv, Tq, Tkv, D, causal, window, sinks, dtype
    (1, 2, 1, 300, 300, 64, True, 40, 1, "fp16"),
    (2, 4, 2, 513, 513, 128, True, 100, 64, "bf16"),
    (1, 3, 3, 400, 400, 96, True, 129, 5, "bf16"),
    (1, 4, 1, 640, 640, 256, True, 200, 130, "fp16"),
    (1, 2, 2, 700, 700, 128, True, 64, 300, "fp16"),       # several blocks of first keys
    (1, 4, 2, 1100, 1100, 64, True, 128, 128, "bf16"),     # on tile borders
    (1, 2, 1, 1500, 1500, 256, True, 33, 3, "bf16"),       # parts of the first block
    (1, 2, 1, 2000, 2000, 128, True, 100, 4, "bf16"),
    (1, 2, 2, 600, 200, 64, True, 50, 7, "bf16"),          # queries behind the last key see first keys alone
    (1, 2, 1, 500, 900, 128, False, 60, 9, "fp16"),        # later keys visible
    (1, 2, 1, 700, 300, 96, False, 20, 150, "bf16"),
    (1, 4, 2, 800, 100, 256, False, 10, 60, "fp16"),
    (2, 2, 1, 9, 9, 64, True, 3, 2, "bf16"),
    (1, 2, 1, 5, 5, 128, True, 1, 1, "fp16"),              # no more tokens than a decoding step's
    (1, 4, 4, 257, 257, 64, True, 1, 255, "bf16"),
    (1, 2, 1, 300, 300, 128, True, 200, 100, "bf16"),      # nothing hidden: a causal call
    (1, 4, 2, 100, 80, 64, False, 30, 80, "fp16"),         # nor here: no mask at all
    (70, 4, 2, 260, 260, 64, True, 30, 6, "fp16"),         # more items than the GPU takes at once
]


def dense_inputs(case):
    B, Hq, Hkv, Tq, Tkv, D, causal, window, sinks, dt = case
    g = gen(Tq + D)
    q, do = (randn(g, B, Hq, Tq, D, dtype=DT[dt]) for _ in range(2))
    k, v = (randn(g, B, Hkv, Tkv, D, dtype=DT[dt]) for _ in range(2))
    return q, k, v, do


def dense_call(q, k, v, do, scale, causal, window, sinks):
    B, Hq, Tq, D = q.shape
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    o, lse = torch.full_like(q, NAN), torch.full(q.shape[:3], NAN, device="cuda")
    dq, dk, dv = torch.full_like(q, NAN), torch.full_like(k, NAN), torch.full_like(v, NAN)
    ws = torch.full((fa.fa_bwd_sinks_workspace_size(B, Hq, k.shape[1], Tq, k.shape[2], D, window, sinks),), 255,
                    dtype=torch.uint8, device="cuda")
    fa.fa_fwd(q, k, v, o, lse, scale, causal, window, sinks=sinks)
    fa.fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, causal, window, workspace=ws, sinks=sinks)
    assert clear()
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.parametrize("case", DENSE, ids=lambda c: f"B{c[0]}h{c[1]}x{c[2]}t{c[3]}x{c[4]}d{c[5]}{'c' if c[6] else ''}w{c[7]}s{c[8]}{c[9]}")
def test_dense_matches_the_definition(case):
    B, Hq, Hkv, Tq, Tkv, D, causal, window, sinks, dt = case
    q, k, v, do = dense_inputs(case)
    scale = 1.0 / math.sqrt(D)
    got = dense_call(q, k, v, do, scale, causal, window, sinks)
    part = slice(0, 2) if B > 2 else slice(0, B)
    values, bounds = ref.dense(q[part], k[part], v[part], do[part], scale, causal, window, sinks)
    for n, x in values.items():
        y = got[n][part].double().cpu()
        empty = x == -math.inf
        assert torch.equal(y == -math.inf, empty), n
        bad = ~((y - x).abs()[~empty] <= bounds[n][~empty])
        assert not bad.any(), f"{n} off by {((y - x).abs()[~empty] / bounds[n][~empty]).max():.3g} bounds"
    again = dense_call(q, k, v, do, scale, causal, window, sinks)
    for n in got:
        assert torch.equal(got[n], again[n]), n
    if B > 2:  # the batch's last sequence, which another CTA's later item has
        values, bounds = ref.dense(q[-1:], k[-1:], v[-1:], do[-1:], scale, causal, window, sinks)
        for n, x in values.items():
            assert ((got[n][-1:].double().cpu() - x).abs() <= bounds[n]).all(), n


def test_dense_equals_the_calls_without_first_keys():
    """sinks = 0 through the new entries, and sinks whose window hides nothing, give the bits of the older calls."""
    g = gen(9)
    B, Hq, Hkv, T, D = 1, 4, 2, 500, 128
    q, do = (randn(g, B, Hq, T, D, dtype=torch.bfloat16).cuda() for _ in range(2))
    k, v = (randn(g, B, Hkv, T, D, dtype=torch.bfloat16).cuda() for _ in range(2))
    lib = fa.library()

    def run(window, sinks, entry):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(fa.fa_bwd_sinks_workspace_size(B, Hq, Hkv, T, T, D, window, sinks), dtype=torch.uint8, device="cuda")
        p = [x.data_ptr() for x in (q, k, v, o, do, lse, dq, dk, dv, ws)]
        extra = [sinks] if entry else []
        st = (lib.fa_fwd_sinks if entry else lib.fa_fwd)(p[0], p[1], p[2], p[3], p[5], B, Hq, Hkv, T, T, D, 0.1, 1, window, *extra, 1, None)
        st |= (lib.fa_bwd_sinks if entry else lib.fa_bwd)(*p[:4], p[4], p[5], p[6], p[7], p[8], B, Hq, Hkv, T, T, D, 0.1, 1, window,
                                                          *extra, 1, p[9], ws.numel(), None)
        assert st == 0 and clear()
        return o, lse, dq, dk, dv

    for window, sinks, like in ((100, 0, 100), (0, 0, 0), (0, 33, 0), (400, 100, 0)):
        for a, b in zip(run(window, sinks, True), run(like, 0, False)):
            assert torch.equal(a, b)


def test_dense_through_autograd_and_captured():
    """flash_attention(sinks=) and its gradients: views as inputs, a broadcast cotangent, a shared input, and the same
    step captured into a graph and replayed on other inputs."""
    from attention_fa_fwd_03_gb300.autograd import flash_attention
    g = gen(12)
    B, Hq, Hkv, T, D, window, sinks = 1, 4, 2, 400, 64, 70, 6
    qkv = randn(g, B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    x = qkv.cuda().requires_grad_()
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    o, lse = flash_attention(q, k, v, causal=True, window=window, sinks=sinks, return_lse=True)
    do = randn(g, 1, 1, 1, D, dtype=torch.bfloat16).expand(B, Hq, T, D)
    o.backward(do.cuda())
    want, bounds = ref.dense(*(t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], 2)), do, 1 / math.sqrt(D), True, window, sinks)
    grads = dict(zip(("dq", "dk", "dv"), (t.transpose(1, 2) for t in x.grad.split([Hq, Hkv, Hkv], 2))))
    for n, y in {"o": o.detach(), "lse": lse, **grads}.items():
        assert ((y.double().cpu() - want[n]).abs() <= bounds[n]).all(), n
    # one tensor as keys and as values
    kv = randn(g, B, Hkv, T, D, dtype=torch.bfloat16)
    a = kv.cuda().requires_grad_()
    flash_attention(q.detach(), a, a, causal=True, window=window, sinks=sinks).backward(do.cuda())
    want, bounds = ref.dense(q.detach().cpu(), kv, kv, do, 1 / math.sqrt(D), True, window, sinks)
    both, limit = want["dk"] + want["dv"], bounds["dk"] + bounds["dv"]
    assert ((a.grad.double().cpu() - both).abs() <= limit + 2.0 ** -8 * both.abs()).all()
    # captured
    ins = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dog = do.cuda().contiguous()
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(flash_attention(*ins, causal=True, window=window, sinks=sinks), ins, dog)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        oc = flash_attention(*ins, causal=True, window=window, sinks=sinks)
        gc = torch.autograd.grad(oc, ins, dog)
    for seed in (1, 2):
        new = [randn(gen(seed + n), *t.shape, dtype=torch.bfloat16).cuda() for n, t in enumerate(ins)]
        with torch.no_grad():
            for t, y in zip(ins, new):
                t.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        fresh = [y.clone().requires_grad_() for y in new]
        oe = flash_attention(*fresh, causal=True, window=window, sinks=sinks)
        ge = torch.autograd.grad(oe, fresh, dog)
        assert torch.equal(oc, oe) and all(torch.equal(a, b) for a, b in zip(gc, ge))
    assert clear()


def test_dense_many_times_over():
    """Enough work items that CTAs take several, with the first blocks in parts: the same bits every time."""
    case = (2, 8, 2, 4000, 4000, 128, True, 300, 10, "bf16")
    q, k, v, do = dense_inputs(case)
    first = dense_call(q, k, v, do, 0.1, True, 300, 10)
    assert all(x.isfinite().all() for x in first.values())
    for _ in range(10):
        again = dense_call(q, k, v, do, 0.1, True, 300, 10)
        for n in first:
            assert torch.equal(first[n], again[n]), n


def test_dense_waits_give_up():
    case = (1, 4, 2, 2000, 2000, 128, True, 100, 4, "bf16")
    q, k, v, do = dense_inputs(case)
    want = dense_call(q, k, v, do, 0.1, True, 100, 4)
    for D in (128, 256):
        x = [t if D == 128 else t.repeat(1, 1, 1, 2).contiguous() for t in (q, k, v, do)]
        fa.fa_set_wait_limit_cycles(8)
        try:
            a = [t.cuda() for t in x]
            o, lse = torch.empty_like(a[0]), torch.empty(a[0].shape[:3], device="cuda")
            outs = [torch.empty_like(t) for t in a[:3]]
            ws = torch.empty(fa.fa_bwd_sinks_workspace_size(1, 4, 2, 2000, 2000, D, 100, 4), dtype=torch.uint8, device="cuda")
            fa.fa_fwd(a[0], a[1], a[2], o, lse, 0.1, True, 100, sinks=4)
            fa.fa_bwd(a[0], a[1], a[2], o, a[3], lse, *outs, 0.1, True, 100, workspace=ws, sinks=4)
            torch.cuda.synchronize()
        finally:
            fa.fa_set_wait_limit_cycles(0)
        assert fa.fa_device_status() & 1
    got = dense_call(q, k, v, do, 0.1, True, 100, 4)
    for n in want:
        assert torch.equal(want[n], got[n]), n
