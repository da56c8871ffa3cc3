"""Host-side tests of the paged-cache calls: every refusal happens before the device is touched (no call here reaches
CUDA), and the binding checks what it marshals."""
import ctypes

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
from attention_fa_fwd_03_gb300 import build_lib

INVALID, HEAD_DIM, DTYPE, MISALIGNED = 1, 2, 3, 4
BASE, GAP = 1 << 40, 1 << 36  # fake, well separated, 16-byte aligned device addresses


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return fa.library()


def addr(i):
    return BASE + i * GAP


CACHE = dict(k=addr(0), v=addr(1), k_bounds=addr(2), page_table=addr(3), kv_lens=addr(4), B=2, Hkv=2, D=128,
             num_pages=40, page_size=32, max_pages=16, dt=1)

BAD_CACHE = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=-1), INVALID),
    (dict(page_size=8), INVALID), (dict(page_size=48), INVALID), (dict(page_size=512), INVALID),
    (dict(D=80), HEAD_DIM), (dict(D=512), HEAD_DIM), (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_table=None), INVALID), (dict(kv_lens=None), INVALID),
    (dict(k=addr(0) + 8), MISALIGNED), (dict(v=addr(1) + 2), MISALIGNED), (dict(k_bounds=addr(2) + 4), MISALIGNED),
    (dict(page_table=addr(3) + 2), MISALIGNED), (dict(kv_lens=addr(4) + 1), MISALIGNED),
    (dict(B=1 << 23, Hkv=4), INVALID),                    # B * Hkv beyond 2^24
    (dict(num_pages=(1 << 30) + 1, Hkv=1), INVALID),      # num_pages * Hkv beyond 2^30
    (dict(max_pages=(1 << 25) + 1), INVALID),             # positions beyond 2^30
]


def cache(**kw):
    return ctypes.byref(fa._PagedKVStruct(**dict(CACHE, **kw)))


def strides(b, h, t):
    return (ctypes.c_int64 * 3)(b, h, t)


def append(lib, cache_kw=None, **kw):
    a = dict(k=addr(5), ks=strides(4096, 128, 256), v=addr(6), vs=strides(4096, 128, 256), q=addr(7),
             qs=strides(8192, 128, 512), q_out=addr(8), Hq=4, T=16, new_lens=addr(9), cos=addr(10), sin=addr(11),
             rope_len=512, rot_dim=128, interleaved=0)
    a.update(kw)
    return lib.fa_kv_append(cache(**(cache_kw or {})), a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["q_out"],
                            a["Hq"], a["T"], a["new_lens"], a["cos"], a["sin"], a["rope_len"], a["rot_dim"],
                            a["interleaved"], None)


def paged_fwd(lib, cache_kw=None, **kw):
    a = dict(q=addr(5), o=addr(6), lse=addr(7), Hq=4, Tq=2, scale=0.1, causal=1, window=0, new_lens=addr(8),
             sel=addr(9), sel_lens=addr(10), n_sel=8, ws=addr(11), ws_bytes=1 << 30)
    a.update(kw)
    return lib.fa_paged_fwd(cache(**(cache_kw or {})), a["q"], a["o"], a["lse"], a["Hq"], a["Tq"], a["scale"],
                            a["causal"], a["window"], a["new_lens"], a["sel"], a["sel_lens"], a["n_sel"], a["ws"],
                            a["ws_bytes"], None)


def select(lib, cache_kw=None, **kw):
    a = dict(q=addr(5), Hq=4, n_sel=8, first=1, last=2, sel=addr(6), sel_lens=addr(7), ws=addr(8), ws_bytes=1 << 30)
    a.update(kw)
    return lib.fa_page_select(cache(**(cache_kw or {})), a["q"], a["Hq"], a["n_sel"], a["first"], a["last"], a["sel"],
                              a["sel_lens"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
@pytest.mark.parametrize("call", [append, paged_fwd, select])
def test_bad_cache_is_refused(lib, call, kw, code):
    assert call(lib, cache_kw=kw) == code


@pytest.mark.parametrize("call", [lambda l: l.fa_kv_append(None, *[None] * 7, 0, 1, None, None, None, 0, 0, 0, None),
                                  lambda l: l.fa_paged_fwd(None, None, None, None, 1, 1, 1.0, 0, 0, None, None, None, 0,
                                                           None, 0, None),
                                  lambda l: l.fa_page_select(None, None, 1, 1, 0, 0, None, None, None, 0, None)])
def test_null_cache_is_refused(lib, call):
    assert call(lib) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INVALID), (dict(T=(1 << 22) + 1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(q_out=None), INVALID), (dict(q=None), INVALID),
    (dict(qs=None), INVALID), (dict(Hq=0), INVALID), (dict(Hq=3), INVALID), (dict(cos=None), INVALID),
    (dict(sin=None), INVALID), (dict(cos=None, sin=None), INVALID),  # rot_dim without angles
    (dict(rot_dim=0), INVALID), (dict(rot_dim=24), INVALID), (dict(rot_dim=144), INVALID), (dict(rope_len=0), INVALID),
    (dict(interleaved=2), INVALID),
    (dict(ks=strides(4096, 128, 100)), INVALID), (dict(vs=strides(-8, 128, 256)), INVALID),
    (dict(qs=strides(8192, 4, 512)), INVALID),
    (dict(k=addr(5) + 8), MISALIGNED), (dict(v=addr(6) + 2), MISALIGNED), (dict(q=addr(7) + 4), MISALIGNED),
    (dict(q_out=addr(8) + 8), MISALIGNED), (dict(cos=addr(10) + 4), MISALIGNED), (dict(sin=addr(11) + 8), MISALIGNED),
    (dict(new_lens=addr(9) + 2), MISALIGNED),
    (dict(q_out=addr(7)), INVALID),                      # rotating in place
    (dict(k=CACHE["k"] + 256), INVALID),                 # new keys inside the pool
    (dict(q_out=CACHE["v"]), INVALID), (dict(cos=CACHE["k"]), INVALID), (dict(new_lens=CACHE["k_bounds"]), INVALID),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_refuses_overlapping_pools(lib):
    assert append(lib, cache_kw=dict(v=CACHE["k"] + 4096)) == INVALID
    assert append(lib, cache_kw=dict(page_table=CACHE["k"])) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(Tq=0), INVALID), (dict(Tq=9), INVALID), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=16), INVALID), (dict(sel=None), INVALID),
    (dict(sel_lens=None), INVALID), (dict(n_sel=0), INVALID), (dict(n_sel=(1 << 20) + 1), INVALID),
    (dict(q=addr(5) + 8), MISALIGNED), (dict(o=addr(6) + 8), MISALIGNED), (dict(lse=addr(7) + 4), MISALIGNED),
    (dict(ws=addr(11) + 8), MISALIGNED), (dict(sel=addr(9) + 1), MISALIGNED), (dict(sel_lens=addr(10) + 2), MISALIGNED),
    (dict(o=addr(5)), INVALID), (dict(lse=addr(6) + 16), INVALID), (dict(ws=CACHE["k"]), INVALID),
    (dict(o=CACHE["v"]), INVALID),
])
def test_paged_fwd_refusals(lib, kw, code):
    assert paged_fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=0), INVALID), (dict(Hq=3), INVALID), (dict(n_sel=0), INVALID), (dict(n_sel=(1 << 20) + 1), INVALID),
    (dict(first=-1), INVALID), (dict(last=-1), INVALID), (dict(first=5, last=4), INVALID), (dict(q=None), INVALID),
    (dict(sel=None), INVALID), (dict(sel_lens=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(q=addr(5) + 2), MISALIGNED), (dict(ws=addr(8) + 4), MISALIGNED), (dict(sel=addr(6) + 2), MISALIGNED),
    (dict(sel_lens=addr(6)), INVALID), (dict(sel=CACHE["k_bounds"]), INVALID),
])
def test_page_select_refusals(lib, kw, code):
    assert select(lib, **kw) == code


def test_paged_fwd_refuses_more_tiles_than_it_counts(lib):
    big = dict(B=1 << 20, Hkv=16, max_pages=1 << 20)
    assert paged_fwd(lib, cache_kw=big, Hq=16, sel=None, sel_lens=None) == INVALID


def test_append_refuses_strides_whose_extent_leaves_64_bits(lib):
    # 2^23 sequences, 2^40 elements apart: the extent in bytes is 2^64
    big = dict(B=1 << 23, Hkv=1, num_pages=1, max_pages=1)
    assert append(lib, cache_kw=big, Hq=1, ks=strides(1 << 40, 0, 0)) == INVALID
    for name in ("ks", "vs", "qs"):
        for i in range(3):
            assert append(lib, **{name: strides(*((1 << 39) if j == i else 256 for j in range(3)))}) == INVALID


def test_outputs_inside_parts_of_the_cache_that_a_call_does_not_read_are_refused(lib):
    assert paged_fwd(lib, o=CACHE["k_bounds"]) == INVALID
    assert paged_fwd(lib, ws=CACHE["k_bounds"]) == INVALID
    assert select(lib, sel=CACHE["k"]) == INVALID
    assert select(lib, ws=CACHE["v"]) == INVALID


def test_workspace_sizes_beyond_the_limits_are_zero(lib):
    assert fa.fa_paged_workspace_size(1 << 30, 1, 8, 64) == 0            # 2^33 rows
    assert fa.fa_page_select_workspace_size(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) == 0
    assert fa.fa_page_select_workspace_size(1 << 20, 16, 1 << 30) == 12 << 54


def test_attributes_of_a_cache_cannot_be_assigned():
    """Calls go to the tensors that the object was made with: an assignment would be silently without effect."""
    kv = fa.PagedKV.__new__(fa.PagedKV)
    for name in ("kv_lens", "page_table", "k", "B"):
        with pytest.raises(AttributeError, match="in place"):
            setattr(kv, name, torch.ones(2, dtype=torch.int32))
        with pytest.raises(AttributeError):
            delattr(kv, name)
    lens = torch.ones(2, dtype=torch.int32)
    object.__setattr__(kv, "kv_lens", lens)
    kv.kv_lens += 1                            # in place
    assert kv.kv_lens is lens and lens.tolist() == [2, 2]
    with pytest.raises(AttributeError):
        kv.kv_lens = lens + 1


def test_page_select_needs_bounds(lib):
    assert select(lib, cache_kw=dict(k_bounds=None)) == INVALID


def test_workspace_sizes(lib):
    assert fa.fa_paged_workspace_size(32, 8, 1, 128) > 0
    for bad in ((0, 1, 1, 64), (5, 2, 1, 64), (4, 2, 9, 64), (4, 2, 0, 64), (4, 2, 1, 80)):
        assert fa.fa_paged_workspace_size(*bad) == 0
    need = fa.fa_paged_workspace_size(4, 2, 2, 128)
    assert paged_fwd(lib, ws_bytes=need - 1) == INVALID
    assert fa.fa_page_select_workspace_size(2, 2, 16) >= 2 * 2 * 16 * 4
    assert fa.fa_page_select_workspace_size(0, 2, 16) == 0
    assert select(lib, ws_bytes=fa.fa_page_select_workspace_size(2, 2, 16) - 1) == INVALID


def test_status_names(lib):
    assert fa.fa_status_string(7) not in ("", "unknown status")
    assert "FA_ERR_BAD_INDEX" in str(fa.FaError(7, "x"))


def test_binding_refuses_cpu_and_mismatched_tensors(lib):
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.PagedKV(pool, pool.clone(), table, lens)          # not on a GPU
    with pytest.raises(ValueError):
        fa.PagedKV(pool[0], pool[0], table, lens)            # no pool
    with pytest.raises(ValueError):
        fa.PagedKV(pool, pool[:2], table, lens)              # v of another shape
    with pytest.raises(ValueError):
        fa.PagedKV(pool, pool.clone(), table.long(), lens)   # 64-bit table
    with pytest.raises(ValueError):
        fa.PagedKV(pool, pool.clone(), table, torch.ones(2, dtype=torch.int32))
    with pytest.raises(fa.FaError):
        fa.PagedKV(pool.float(), pool.float(), table, lens)  # fp32 pools


# ------------------------------------------------------------------ the compiled binding
@pytest.fixture(scope="module")
def calls(lib):
    return fa._paged_calls()


def fake_handle(calls, dt=0):
    """A cache of B 2, Hkv 2, D 64 on device 0 at addresses that nothing is at: every call below is refused before it
    would use them."""
    return calls.handle(addr(0), addr(1), addr(2), addr(3), addr(4), 2, 2, 64, 40, 16, 8, dt, 0)


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_binding_refuses_what_is_no_tensor_or_not_on_the_device(calls):
    h = fake_handle(calls)
    q, lse, ws = half(2, 4, 1, 64), torch.zeros(2, 4, 1), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(TypeError):
        calls.paged_fwd(h, q, q)                                                     # too few arguments
    with pytest.raises(ValueError, match="workspace"):
        calls.paged_fwd(h, q, q.clone(), lse, 0.1, True, 0, None, None, None, None, None)
    with pytest.raises(ValueError):                                                  # CPU tensors
        calls.paged_fwd(h, q, q.clone(), lse, 0.1, True, 0, None, None, None, ws, None)
    with pytest.raises(TypeError):
        calls.kv_append(h, 3, q, None, None, False, None, None, None, None)
    k = half(2, 2, 1, 64)
    with pytest.raises(ValueError, match="k"):
        calls.kv_append(h, k, k.clone(), None, None, False, None, None, None, None)  # CPU tensors
    with pytest.raises(ValueError, match="k"):
        calls.kv_append(h, k.float(), k, None, None, False, None, None, None, None)  # dtype
    with pytest.raises(ValueError, match="k"):
        calls.kv_append(h, half(2, 2, 64), k, None, None, False, None, None, None, None)  # three dimensions
    with pytest.raises(ValueError):
        calls.page_select(h, q, torch.zeros(2, 2, 4, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), 0, 1, ws, None)
    with pytest.raises(ValueError):
        calls.paged_fwd(object(), q, q, lse, 0.1, True, 0, None, None, None, ws, None)  # no handle


def test_missing_binding_fails_loudly(lib, monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "attention_fa_fwd_03_gb300._paged", None)
    monkeypatch.delattr(fa, "_paged", raising=False)
    with pytest.raises(RuntimeError, match="not built"):
        fa._paged_calls()
