"""The split list where units count for places beside their tiles (a cache held in 8 bits, up to 16 rows): what the host
accepts can be counted in 32 bits, and the walk of csrc/fa_paged_walk.h, compiled for the host, takes every tile once, in every
warp alike, with parts recorded for the join that are exactly those which hold the unit. No call here reaches CUDA."""
import ctypes
import os
import random
import subprocess

import pytest

import attention_fa_fwd_03_gb300 as fa
from attention_fa_fwd_03_gb300 import build_lib

INVALID = 1
BASE, GAP = 1 << 40, 1 << 36  # fake, well separated, 16-byte aligned device addresses

HARNESS = r"""
#include <climits>
#include <vector>
#include "fa_paged_walk.h"
using namespace fa;

extern "C" int over_of(int e4m3, int rows) { return list_over(e4m3 != 0, rows); }
extern "C" int fits(long long units, long long keys, int over) { return list_fits(units, keys, over); }
// shares of `total` places: in order, without a gap, from 0 to the end, none out of range
extern "C" int divides(int total, int parts) {
  int at = 0;
  for (int part = 0; part < parts; ++part) {
    Share s;
    s.divide(total, part, parts);
    if (s.lo != at || s.hi < s.lo || s.hi > total) return 0;
    if (s.hi > s.lo && (s.part_of(s.lo) != part || s.part_of(s.hi - 1) != part)) return 0;
    at = s.hi;
  }
  return at == total;
}

static const int *g_len, *g_n;
static int g_items, g_change;
static unsigned g_state;
static ItemLens lens_now(int i) {
  int j = i;
  if (g_change) {
    g_state = g_state * 1664525u + 1013904223u;
    j = static_cast<int>((g_state >> 8) % static_cast<unsigned>(g_items));
  }
  return ItemLens::of(g_len[j], g_n[j], 0);
}
struct Cta {  // the windows that a CTA fills, kept so that each of its warps meets the same ones
  std::vector<std::vector<ItemLens>> windows;
  std::vector<int> bases;
  void fill(int from) {
    bases.push_back(from);
    windows.emplace_back(kItemWindow, ItemLens{0, 0});
    for (int i = 0; i < kItemWindow && from + i < g_items; ++i) windows.back()[i] = lens_now(from + i);
  }
};
struct Role {
  Cta& cta;
  int at = 0;
  bool outside = false;
  ItemLens operator()(int item) {
    if (item - cta.bases[at] >= kItemWindow) {
      if (++at == static_cast<int>(cta.windows.size())) cta.fill(item);
      if (cta.bases[at] != item) outside = true;
    }
    const int slot = item - cta.bases[at];
    if (slot < 0 || slot >= kItemWindow) { outside = true; return {0, 0}; }
    return cta.windows[at][slot];
  }
};
struct Seg { int item, sub, t0, t1, tiles; };

// 0: as it has to be; 1: walks of a CTA differ; 2: outside the list; 3: a tile not taken once; 4: the record for the
// join names other parts than those that hold the unit
extern "C" int check(int items, int mult, int window, int sinks, int over, const int* len, const int* n, int parts, int change,
                     unsigned seed) {
  g_len = len; g_n = n; g_items = items; g_change = 0; g_state = seed;
  const ListShape list = {items, mult, 0, window, 4, sinks, over};
  std::vector<long long> before(items + 1, 0);
  std::vector<std::vector<int>> taken, held(static_cast<size_t>(items) * mult);
  std::vector<int> first_of(held.size(), -1), last_of(held.size(), -1);
  for (int i = 0; i < items; ++i) {
    const Item it = make_item(list, lens_now(i));
    before[i + 1] = before[i] + static_cast<long long>(unit_places(list, it)) * mult;
    for (int s = 0; s < mult; ++s) taken.emplace_back(it.tiles, 0);
  }
  for (int part = 0; part < parts; ++part) {
    Share s;
    s.divide(static_cast<int>(before[items]), part, parts);
    s.item = s.rest = 0;
    for (int i = 0; i < items; ++i)
      if (s.lo >= before[i] && s.lo < before[i + 1]) { s.item = i; s.rest = static_cast<int>(s.lo - before[i]); }
    g_change = change;
    Cta cta;
    cta.fill(items <= kItemWindow ? 0 : s.item);
    std::vector<Seg> first;
    for (int role = 0; role < 3; ++role) {
      Role r{cta};
      std::vector<Seg> segs;
      Walk w;
      for (bool more = w.start(list, s, r); more; more = w.next(list, r)) {
        if (w.item < 0 || w.item >= items || w.sub < 0 || w.sub >= mult || w.t0 < 0 || w.t1 < w.t0 || w.used <= 0) return 2;
        segs.push_back({w.item, w.sub, w.t0, w.t1, w.it.tiles});
      }
      if (r.outside) return 2;
      if (role == 0) { first = segs; continue; }
      bool same = segs.size() == first.size();
      for (size_t i = 0; same && i < segs.size(); ++i)
        same = segs[i].item == first[i].item && segs[i].sub == first[i].sub && segs[i].t0 == first[i].t0 &&
               segs[i].t1 == first[i].t1;
      if (!same) return 1;
    }
    g_change = 0;
    if (change) continue;
    for (const Seg& g : first) {
      const size_t u = static_cast<size_t>(g.item) * mult + g.sub;
      if (g.t1 <= g.t0) return 3;
      for (int t = g.t0; t < g.t1; ++t)
        if (taken[u][t]++) return 3;
      held[u].push_back(part);
      if (g.t0 == 0) {  // as the kernels record it
        first_of[u] = part;
        last_of[u] = g.t1 == g.tiles ? part : walk_min(s.part_of(s.hi - g.t1 + g.tiles - 1), s.parts - 1);
      }
    }
  }
  if (change) return 0;
  for (size_t u = 0; u < taken.size(); ++u) {
    for (int x : taken[u])
      if (x != 1) return 3;
    if (taken[u].empty()) {
      if (!held[u].empty()) return 4;
      continue;
    }
    if (held[u].empty() || held[u].front() != first_of[u] || held[u].back() != last_of[u] ||
        static_cast<int>(held[u].size()) != last_of[u] - first_of[u] + 1)
      return 4;
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("places")
    src, so = os.path.join(d, "walk.cpp"), os.path.join(d, "walk.so")
    with open(src, "w") as fh:
        fh.write(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build_lib.CSRC, "-o", so, src], check=True)
    lib = ctypes.CDLL(so)
    lib.fits.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int]
    return lib


@pytest.mark.parametrize("units,heads,tokens", [(1 << 24, 1, 1), (1 << 24, 1, 8), (1 << 22, 3, 3), (1 << 23, 2, 8)])
def test_lists_beyond_32_bits_are_refused(units, heads, tokens):
    """Tiles and two places of every unit are 2^31 in all; their pages may be shared, so memory does not forbid them."""
    build_lib.build()
    pages = (1 << 31) // units - 2
    cache = fa._PagedKV8Struct(k=BASE, v=BASE + GAP, k_scales=BASE + 2 * GAP, v_scales=BASE + 3 * GAP, page_table=BASE + 4 * GAP,
                               kv_lens=BASE + 5 * GAP, B=units >> 4, Hkv=1 << 4, D=64, num_pages=40, page_size=64, max_pages=pages)
    q, o, lse, ws = (BASE + (6 + i) * GAP for i in range(4))
    st = fa.library().fa_paged_fwd8(ctypes.byref(cache), q, o, lse, heads * cache.Hkv, tokens, 0.1, 1, 0, 0, None, None, None, 0, 1,
                                    ws, 1 << 30, None)
    assert st == INVALID


def test_what_fits_is_divided_without_overflow(walk):
    """At the limit of every number of extra places, for all numbers of shares a GPU may have."""
    most = 2 ** 31 - 1
    assert [walk.over_of(1, r) for r in (1, 8, 16, 17, 128)] == [2, 2, 2, 0, 0] and walk.over_of(0, 8) == 0
    for over in (0, 2):
        for tiles in (1, 126, 127, 1 << 24):
            units = most // (tiles + over)
            for keys in (64 * tiles - 63, 64 * tiles):
                assert walk.fits(units, keys, over)
                assert not walk.fits(units + 1, keys, over)
            assert not walk.fits(units, 64 * tiles + 1, over) or (tiles + 1 + over) * units <= most
            for parts in (1, 152, 304, 456, 608):
                assert walk.divides(units * (tiles + over), parts)
    assert not walk.fits(1 << 24, 126 * 64, 2) and walk.fits(1 << 24, 126 * 64, 0)


def batches(seed):
    r = random.Random(seed)
    yield dict(lens=[r.randrange(1, 9000) for _ in range(r.randrange(1, 9))], mult=r.randrange(1, 9))
    yield dict(lens=[r.randrange(0, 200) for _ in range(r.randrange(100, 300))], mult=r.randrange(1, 4))
    yield dict(lens=[r.choice([0, 0, 0, 1, 64, 65]) for _ in range(r.randrange(2000, 3000))])
    yield dict(lens=[9000 if r.random() < 0.002 else 0 for _ in range(3000)] + [7], mult=r.randrange(1, 3))
    yield dict(lens=[r.randrange(1, 9000) for _ in range(20)], window=r.randrange(1, 3000), sinks=r.randrange(1, 400), mult=2)
    yield dict(lens=[r.choice([0, 1, 65]) for _ in range(r.randrange(3, 40))])  # shares shorter than a unit's places


def call(walk, lens, new, mult=1, window=0, sinks=0, over=2, parts=456, change=0, seed=1):
    arr = ctypes.c_int * len(lens)
    return walk.check(len(lens), mult, window, sinks, over, arr(*lens), arr(*new), parts, change, seed)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("over", [0, 1, 2, 5])
def test_every_tile_is_walked_once_and_the_parts_are_recorded(walk, seed, over):
    r = random.Random(seed)
    for b in batches(seed):
        new = [r.choice([1, 1, 8, 0]) for _ in b["lens"]]
        for parts in (1, 2, 152, 304, 456):
            assert call(walk, new=new, over=over, parts=parts, **b) == 0, (seed, over, parts, b)


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("over", [1, 2])
def test_warps_walk_alike_whatever_the_lengths_do(walk, seed, over):
    r = random.Random(seed)
    for b in batches(seed):
        new = [r.choice([1, 1, 8, 0]) for _ in b["lens"]]
        assert call(walk, new=new, over=over, change=1, seed=seed + 1, **b) == 0, (seed, over, b)
