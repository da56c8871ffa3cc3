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
