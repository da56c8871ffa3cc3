"""Host-side tests of the 8-bit cache, of windows with first keys and of page assignment: every refusal happens before the
device is touched (no call here reaches CUDA), and the list of tiles with a gap in it."""
import ctypes
import os
import subprocess

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


CACHE8 = dict(k=addr(0), v=addr(1), k_scales=addr(2), v_scales=addr(12), page_table=addr(3), kv_lens=addr(4), B=2, Hkv=2, D=128,
              num_pages=40, page_size=32, max_pages=16)
CACHE = dict(k=addr(0), v=addr(1), k_bounds=addr(2), page_table=addr(3), kv_lens=addr(4), B=2, Hkv=2, D=128,
             num_pages=40, page_size=32, max_pages=16, dt=1)
BAD_CACHE8 = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=-1), INVALID),
    (dict(page_size=8), INVALID), (dict(page_size=48), INVALID), (dict(page_size=512), INVALID),
    (dict(D=80), HEAD_DIM), (dict(D=512), HEAD_DIM), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID), (dict(page_table=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(k=addr(0) + 8), MISALIGNED), (dict(v=addr(1) + 2), MISALIGNED),
    (dict(k_scales=addr(2) + 2), MISALIGNED), (dict(v_scales=addr(12) + 1), MISALIGNED),
    (dict(page_table=addr(3) + 2), MISALIGNED), (dict(kv_lens=addr(4) + 1), MISALIGNED), (dict(B=1 << 23, Hkv=4), INVALID),
    (dict(num_pages=(1 << 30) + 1, Hkv=1), INVALID), (dict(max_pages=(1 << 25) + 1), INVALID),
]


def strides(b, h, t):
    return (ctypes.c_int64 * 3)(b, h, t)


def append8(lib, cache_kw=None, **kw):
    a = dict(k=addr(5), ks=strides(4096, 128, 256), v=addr(6), vs=strides(4096, 128, 256), q=addr(7),
             qs=strides(8192, 128, 512), q_out=addr(8), Hq=4, T=16, new_lens=addr(9), cos=addr(10), sin=addr(11),
             rope_len=512, rot_dim=128, interleaved=0, dt=1)
    a.update(kw)
    c = ctypes.byref(fa._PagedKV8Struct(**dict(CACHE8, **(cache_kw or {}))))
    return lib.fa_kv_append8(c, a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["q_out"], a["Hq"], a["T"],
                             a["new_lens"], a["cos"], a["sin"], a["rope_len"], a["rot_dim"], a["interleaved"], a["dt"], None)


def fwd_args(kw):
    a = dict(q=addr(5), o=addr(6), lse=addr(7), Hq=4, Tq=2, scale=0.1, causal=1, window=0, sinks=0, new_lens=addr(8),
             sel=addr(9), sel_lens=addr(10), n_sel=8, dt=1, ws=addr(11), ws_bytes=1 << 30)
    a.update(kw)
    return a


def fwd8(lib, cache_kw=None, **kw):
    a = fwd_args(kw)
    c = ctypes.byref(fa._PagedKV8Struct(**dict(CACHE8, **(cache_kw or {}))))
    return lib.fa_paged_fwd8(c, a["q"], a["o"], a["lse"], a["Hq"], a["Tq"], a["scale"], a["causal"], a["window"], a["sinks"],
                             a["new_lens"], a["sel"], a["sel_lens"], a["n_sel"], a["dt"], a["ws"], a["ws_bytes"], None)


def fwd_sinks(lib, cache_kw=None, **kw):
    a = fwd_args(kw)
    c = ctypes.byref(fa._PagedKVStruct(**dict(CACHE, **(cache_kw or {}))))
    return lib.fa_paged_fwd_sinks(c, a["q"], a["o"], a["lse"], a["Hq"], a["Tq"], a["scale"], a["causal"], a["window"],
                                  a["sinks"], a["new_lens"], a["sel"], a["sel_lens"], a["n_sel"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", BAD_CACHE8)
@pytest.mark.parametrize("call", [append8, fwd8])
def test_bad_cache_is_refused(lib, call, kw, code):
    assert call(lib, cache_kw=kw) == code


def test_null_cache_is_refused(lib):
    assert lib.fa_kv_append8(None, *[None] * 7, 0, 1, None, None, None, 0, 0, 0, 1, None) == INVALID
    assert lib.fa_paged_fwd8(None, None, None, None, 1, 1, 1.0, 0, 0, 0, None, None, None, 0, 1, None, 0, None) == INVALID
    assert lib.fa_paged_fwd_sinks(None, None, None, None, 1, 1, 1.0, 0, 0, 0, None, None, None, 0, None, 0, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INVALID), (dict(T=(1 << 22) + 1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(Hq=3), INVALID), (dict(cos=None), INVALID),
    (dict(rot_dim=24), INVALID), (dict(rot_dim=144), INVALID), (dict(rope_len=0), INVALID), (dict(interleaved=2), INVALID),
    (dict(k=addr(5) + 2), MISALIGNED), (dict(q_out=addr(8) + 8), MISALIGNED), (dict(new_lens=addr(9) + 1), MISALIGNED),
    (dict(ks=strides(4096, 130, 256)), INVALID), (dict(vs=strides(-8, 128, 256)), INVALID), (dict(dt=2), DTYPE),
    (dict(dt=-1), DTYPE), (dict(k=CACHE8["k"]), INVALID), (dict(v=CACHE8["k_scales"]), INVALID),
    (dict(q_out=CACHE8["v_scales"]), INVALID),
])
def test_append_refuses(lib, kw, code):
    assert append8(lib, **kw) == code


def test_append_refuses_scales_that_meet(lib):
    assert append8(lib, cache_kw=dict(v_scales=CACHE8["k_scales"])) == INVALID
    assert append8(lib, cache_kw=dict(v_scales=CACHE8["k"])) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(Tq=0), INVALID), (dict(Tq=9), INVALID), (dict(Hq=3), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(window=5, sinks=-3), INVALID), (dict(q=None), INVALID), (dict(ws=None), INVALID), (dict(sel=None), INVALID),
    (dict(n_sel=0), INVALID), (dict(ws_bytes=8), INVALID), (dict(o=addr(6) + 2), MISALIGNED), (dict(o=CACHE8["k"]), INVALID),
])
@pytest.mark.parametrize("call", [fwd8, fwd_sinks])
def test_attend_refuses(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_attend8_refuses(lib):
    assert fwd8(lib, dt=2) == DTYPE
    assert fwd8(lib, o=CACHE8["v_scales"]) == INVALID
    assert fwd8(lib, lse=CACHE8["k_scales"]) == INVALID


def assign(lib, **kw):
    a = dict(table=addr(0), lens=addr(1), held=addr(2), free=addr(3), count=addr(4), B=4, num_pages=100, page=16, mp=20, T=8,
             new=addr(5), window=0, sinks=0, slots=addr(6))
    a.update(kw)
    return lib.fa_page_assign(a["table"], a["lens"], a["held"], a["free"], a["count"], a["B"], a["num_pages"], a["page"], a["mp"],
                              a["T"], a["new"], a["window"], a["sinks"], a["slots"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(B=65537), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=(1 << 30) + 1), INVALID),
    (dict(page=8), INVALID), (dict(page=48), INVALID), (dict(mp=0), INVALID), (dict(mp=(1 << 26) + 1), INVALID),
    (dict(B=65536, mp=1 << 15), INVALID), (dict(T=0), INVALID), (dict(T=(1 << 22) + 1), INVALID),
    (dict(B=65536, T=1 << 15), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(held=None), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID),
    (dict(table=addr(0) + 2), MISALIGNED), (dict(new=addr(5) + 1), MISALIGNED), (dict(slots=addr(6) + 4), MISALIGNED),
    (dict(held=addr(0) + 4), INVALID), (dict(slots=addr(1)), INVALID), (dict(free=addr(5)), INVALID), (dict(count=addr(2) + 40), INVALID),
])
def test_assign_refuses(lib, kw, code):
    assert assign(lib, **kw) == code


def test_cache_object_refuses(lib):
    e4m3, half = torch.zeros(4, 2, 16, 64).to(torch.float8_e4m3fn), torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    table, lens, sc = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.ones(4, 2)
    for kw in (dict(k=e4m3, v=e4m3), dict(k=e4m3, v=e4m3, k_scales=sc), dict(k=half, v=half, k_scales=sc, v_scales=sc),
               dict(k=half, v=half, v_scales=sc)):
        with pytest.raises(ValueError, match="scales"):
            fa.PagedKV(page_table=table, kv_lens=lens, **kw)
    with pytest.raises(ValueError, match="k_bounds"):
        fa.PagedKV(e4m3, e4m3, table, lens, k_bounds=torch.zeros(4, 2, 2, 64), k_scales=sc, v_scales=sc)
    with pytest.raises(ValueError, match="k_scales"):
        fa.PagedKV(e4m3, e4m3, table, lens, k_scales=sc[:3], v_scales=sc)
    with pytest.raises(ValueError, match="CUDA"):
        fa.PagedKV(e4m3, e4m3, table, lens, k_scales=sc, v_scales=sc)


def test_assign_binding_refuses(lib):
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_page_assign(t, t[:, 0], torch.zeros(2, 3, dtype=torch.int32), torch.zeros(9, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), 16, 1)
    with pytest.raises(ValueError, match="page_table"):
        fa.fa_page_assign(t[0], t[:, 0], t, t[0], t[0], 16, 1)
    with pytest.raises(TypeError):
        fa.fa_page_assign(None, None, None, None, None, 16, 1)


HARNESS = r"""
#include "fa_paged_walk.h"
using namespace fa;
// bit t of seen[]: tile t of the keys is in the item's list; -1 if twice or out of order
extern "C" int tiles(int window, int sinks, int len, int n, int* seen, int most) {
  const ListShape list = {1, 1, 0, window, 4, sinks};
  const Item it = make_item(list, ItemLens::of(len, n, 0));
  int last = -1;
  for (int t = 0; t < it.tiles; ++t) {
    const int x = it.tile(t);
    if (x <= last || x >= most) return -1;
    last = x;
    seen[x] = 1;
  }
  return it.tiles;
}
"""


def test_tiles_of_a_window_with_first_keys(tmp_path):
    """Every tile with a key that some token sees is in the list, in order, and no other tile but those of first keys and
    window."""
    src = tmp_path / "walk.cpp"
    src.write_text(HARNESS)
    so = tmp_path / "walk.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{build_lib.CSRC}", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))
    for length in (1, 63, 64, 65, 700, 1000):
        for n in (1, 3, 8):
            if n > length:
                continue
            for window in (1, 5, 64, 65, 200, 2000):
                for sinks in (0, 1, 64, 65, 300, 5000, 1 << 30):
                    most = -(-length // 64)
                    seen = (ctypes.c_int * most)()
                    count = lib.tiles(window, sinks, length, n, seen, most)
                    need = {j // 64 for t in range(n) for j in range(length - n + t + 1)
                            if length - n + t - j < window or j < sinks}
                    got = {t for t in range(most) if seen[t]}
                    assert count == len(got) and need <= got
                    first = max(0, length - n - window + 1) // 64
                    assert got == set(range(min(-(-sinks // 64), most))) | set(range(first, most))


def test_reference_gradients():
    """The tests' own gradients of a window with first keys, against torch's and against differences."""
    import cache8_ref as ref
    torch.manual_seed(0)
    for T, N, causal, window, sinks in ((9, 9, True, 3, 2), (8, 5, False, 2, 1), (7, 3, True, 2, 1)):
        q, do = (torch.randn(1, 2, T, 4, dtype=torch.float64) for _ in range(2))
        k, v = (torch.randn(1, 1, N, 4, dtype=torch.float64) for _ in range(2))
        i, j = torch.arange(T)[:, None], torch.arange(N)
        hidden = (i - j >= window) & (j >= sinks) | ((j > i) if causal else torch.zeros(T, N, dtype=torch.bool))

        def plain(q, k, v):
            s = (0.3 * q @ k.transpose(-1, -2)).masked_fill(hidden, -1e300)
            return torch.softmax(s, -1) @ v

        ins = [t.clone().requires_grad_() for t in (q, k, v)]
        want = torch.autograd.grad(plain(*ins), ins, do)
        got, _ = ref.dense(q, k, v, do, 0.3, causal, window, sinks)
        assert torch.allclose(got["o"], plain(q, k, v), rtol=0, atol=1e-13)
        for n, x, w in zip(("dq", "dk", "dv"), (q, k, v), want):
            assert torch.allclose(got[n], w, rtol=0, atol=1e-12)
            d = torch.randn_like(x)
            at = {"dq": 0, "dk": 1, "dv": 2}[n]
            ends = []
            for sign in (1, -1):
                y = [q, k, v]
                y[at] = x + sign * 1e-6 * d
                ends.append((plain(*y) * do).sum())
            assert abs((ends[0] - ends[1]) / 2e-6 - (got[n] * d).sum()) < 1e-7


def dense_args(**kw):
    a = dict(q=addr(0), k=addr(1), v=addr(2), o=addr(3), do=addr(4), lse=addr(5), dq=addr(6), dk=addr(7), dv=addr(8), B=1, Hq=4, Hkv=2,
             Tq=500, Tkv=500, D=128, scale=0.1, causal=1, window=50, sinks=5, dt=1, ws=addr(9), bytes=1 << 32)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(sinks=-1), INVALID), (dict(window=-1), INVALID), (dict(causal=2), INVALID), (dict(scale=0.0), INVALID),
    (dict(Hkv=3), INVALID), (dict(Tq=0), INVALID), (dict(D=80), HEAD_DIM), (dict(dt=2), DTYPE), (dict(q=None), INVALID),
    (dict(o=None), INVALID), (dict(lse=addr(5) + 4), MISALIGNED), (dict(o=addr(0)), INVALID), (dict(lse=addr(1)), INVALID),
])
def test_dense_refuses(lib, kw, code):
    a = dense_args(**kw)
    assert lib.fa_fwd_sinks(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["Tq"], a["Tkv"], a["D"],
                            a["scale"], a["causal"], a["window"], a["sinks"], a["dt"], None) == code
    if kw.keys() != {"o"} and kw.keys() != {"lse"} or kw.get("o", 1) is None:
        assert bwd_sinks(lib, a) == code


def bwd_sinks(lib, a):
    return lib.fa_bwd_sinks(a["q"], a["k"], a["v"], a["o"], a["do"], a["lse"], a["dq"], a["dk"], a["dv"], a["B"], a["Hq"], a["Hkv"],
                            a["Tq"], a["Tkv"], a["D"], a["scale"], a["causal"], a["window"], a["sinks"], a["dt"], a["ws"],
                            a["bytes"], None)


def test_dense_backward_refuses(lib):
    size = fa.fa_bwd_sinks_workspace_size(1, 4, 2, 500, 500, 128, 50, 5)
    assert size > fa.fa_bwd_workspace_size(1, 4, 500)       # the first block's sums
    assert bwd_sinks(lib, dense_args(bytes=size - 1)) == INVALID
    assert bwd_sinks(lib, dense_args(bytes=fa.fa_bwd_workspace_size(1, 4, 500))) == INVALID
    assert bwd_sinks(lib, dense_args(ws=addr(8))) == INVALID
    assert bwd_sinks(lib, dense_args(dq=addr(1))) == INVALID
    assert bwd_sinks(lib, dense_args(ws=addr(9) + 8)) == MISALIGNED


def test_dense_workspace_sizes():
    base = fa.fa_bwd_workspace_size
    size = fa.fa_bwd_sinks_workspace_size
    assert size(1, 4, 2, 500, 500, 128, 50, -1) == 0 and size(0, 4, 2, 500, 500, 128, 50, 5) == 0
    assert size(1, 4, 2, 500, 500, 80, 50, 5) == 0 and size(1, 4, 2, 500, 500, 128, -50, 5) == 0
    for kw in ((0, 5), (450, 50), (500, 1), (1 << 30, 1 << 30), (10, 500), (50, 0)):  # nothing hidden, or no first keys
        assert size(1, 4, 2, 500, 500, 128, *kw) == base(1, 4, 500)
    # however many sequences and first keys, the sums stay small beside the card
    for B, T, sinks in ((1, 1 << 20, 4), (64, 1 << 16, 1 << 15), (1, 1 << 22, 1 << 21), (512, 2048, 1000)):
        assert size(B, 64, 8, T, T, 256, 64, sinks) - base(B, 64, T) < 1 << 30
