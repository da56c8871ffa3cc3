"""How the split list of fa_paged_fwd is shared and walked (csrc/fa_paged_walk.h), compiled for the host: every tile of
every unit belongs to one CTA's walk, and all warps of a CTA walk the same segments within the list's bounds even when the
lengths in memory change meanwhile. (On the GPU they meet at barriers once per segment, so a disagreement would wait for
ever; it is looked for here, not there.)"""
import ctypes
import os
import random
import subprocess

import pytest

from attention_fa_fwd_03_gb300 import build_lib

HARNESS = r"""
#include <vector>
#include "fa_paged_walk.h"
using namespace fa;

// lengths of the items in memory; with `change` every read of a window is followed by another draw
static const int *g_len, *g_n, *g_listed;
static int g_items, g_change;
static unsigned g_state;
static ItemLens lens_now(int i) {
  int j = i;
  if (g_change) {
    g_state = g_state * 1664525u + 1013904223u;
    j = static_cast<int>((g_state >> 8) % static_cast<unsigned>(g_items));
  }
  return ItemLens::of(g_len[j], g_n[j], g_listed[j]);
}

// the windows that a CTA fills, in turn; kept so that each of its warps meets the same ones
struct Cta {
  std::vector<std::vector<ItemLens>> windows;
  std::vector<int> bases;
};
struct Role {
  Cta& cta;
  int at = 0;
  bool outside = false;
  const ItemLens& operator()(int item) {
    if (item - cta.bases[at] >= kItemWindow) {
      if (++at == static_cast<int>(cta.windows.size())) fill(cta, item);
      if (cta.bases[at] != item) outside = true;
    }
    const int slot = item - cta.bases[at];
    if (slot < 0 || slot >= kItemWindow) { outside = true; static const ItemLens none = {0, 0}; return none; }
    return cta.windows[at][slot];
  }
  static void fill(Cta& c, int from) {
    c.bases.push_back(from);
    c.windows.emplace_back(kItemWindow, ItemLens{0, 0});
    for (int i = 0; i < kItemWindow && from + i < g_items; ++i) c.windows.back()[i] = lens_now(from + i);
  }
};
struct Own {  // as if every warp read memory for itself
  ItemLens operator()(int item) const { return lens_now(item); }
};

struct Seg { int item, sub, t0, t1; };
template <class L>
static std::vector<Seg> walk(const ListShape& list, const Share& s, L& lens) {
  std::vector<Seg> out;
  Walk w;
  for (bool more = w.start(list, s, lens); more; more = w.next(list, lens)) out.push_back({w.item, w.sub, w.t0, w.t1});
  return out;
}

// 0: as it has to be; 1: walks of a CTA differ; 2: outside the list; 3: a tile not taken once
extern "C" int check(int items, int mult, int sel, int window, int shift, const int* len, const int* n, const int* listed,
                     int parts, int change, int own_reads, unsigned seed) {
  g_len = len; g_n = n; g_listed = listed; g_items = items; g_change = 0; g_state = seed;
  const ListShape list = {items, mult, sel, window, shift};
  std::vector<int> tiles(items);
  std::vector<long long> before(items + 1, 0);
  for (int i = 0; i < items; ++i) {
    tiles[i] = make_item(list, lens_now(i)).tiles;
    before[i + 1] = before[i] + static_cast<long long>(tiles[i]) * mult;
  }
  std::vector<std::vector<char>> taken(static_cast<size_t>(items) * mult);
  for (int i = 0; i < items; ++i)
    for (int s = 0; s < mult; ++s) taken[static_cast<size_t>(i) * mult + s].assign(tiles[i], 0);
  int status = 0;
  for (int part = 0; part < parts; ++part) {
    Share s;
    s.divide(static_cast<int>(before[items]), part, parts);
    s.item = s.rest = 0;
    for (int i = 0; i < items; ++i)
      if (s.lo >= before[i] && s.lo < before[i + 1]) { s.item = i; s.rest = static_cast<int>(s.lo - before[i]); }
    g_change = change;
    Cta cta;
    Role::fill(cta, items <= kItemWindow ? 0 : s.item);
    std::vector<Seg> first;
    for (int role = 0; role < 3; ++role) {
      std::vector<Seg> segs;
      if (own_reads) {
        Own own;
        segs = walk(list, s, own);
      } else {
        Role r{cta};
        segs = walk(list, s, r);
        if (r.outside) return 2;
      }
      for (const Seg& g : segs)
        if (g.item < 0 || g.item >= items || g.sub < 0 || g.sub >= mult || g.t0 < 0 || g.t1 < g.t0) return 2;
      if (role == 0) { first = segs; continue; }
      bool same = segs.size() == first.size();
      for (size_t i = 0; same && i < segs.size(); ++i)
        same = segs[i].item == first[i].item && segs[i].sub == first[i].sub && segs[i].t0 == first[i].t0 &&
               segs[i].t1 == first[i].t1;
      if (!same) status = 1;
    }
    g_change = 0;
    if (change) continue;
    for (const Seg& g : first)
      for (int t = g.t0; t < g.t1; ++t) {
        char& x = taken[static_cast<size_t>(g.item) * mult + g.sub][t];
        if (x) return 3;
        x = 1;
      }
    // where a unit goes on: the part that holds its last tile
    if (!first.empty() && s.part_of(s.hi - 1) != part) return 3;
  }
  if (!change)
    for (auto& u : taken)
      for (char x : u)
        if (!x) return 3;
  return status;
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    src, lib = os.path.join(d, "walk.cpp"), os.path.join(d, "walk.so")
    with open(src, "w") as fh:
        fh.write(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build_lib.CSRC, "-o", lib, src],
                   check=True)
    fn = ctypes.CDLL(lib).check

    def call(lens, new, listed=None, mult=1, window=0, shift=4, parts=304, change=False, own_reads=False, seed=1):
        arr = ctypes.c_int * len(lens)
        return fn(len(lens), mult, int(listed is not None), window, shift, arr(*lens), arr(*new),
                  arr(*(listed or [0] * len(lens))), parts, int(change), int(own_reads), seed)
    return call


def batches(seed):
    """Lists of a few long sequences, of many short ones, of long stretches without keys, and of selected pages."""
    r = random.Random(seed)
    yield dict(lens=[r.randrange(1, 9000) for _ in range(r.randrange(1, 9))], mult=r.randrange(1, 9))
    yield dict(lens=[r.randrange(0, 200) for _ in range(r.randrange(100, 300))], mult=r.randrange(1, 4))
    yield dict(lens=[r.choice([0, 0, 0, 1, 64, 65]) for _ in range(r.randrange(2000, 4000))])
    yield dict(lens=[9000 if r.random() < 0.002 else 0 for _ in range(3000)] + [7], mult=r.randrange(1, 3))
    yield dict(lens=[r.randrange(1, 9000) for _ in range(20)], window=r.randrange(1, 3000), mult=2)
    yield dict(lens=[r.randrange(1, 9000) for _ in range(300)], listed=[r.randrange(0, 60) for _ in range(300)], shift=r.choice([4, 6, 8]))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("parts", [1, 152, 304, 456])
def test_every_tile_is_walked_once(check, seed, parts):
    r = random.Random(seed)
    for b in batches(seed):
        new = [r.choice([1, 1, 8, 0]) for _ in b["lens"]]
        assert check(new=new, parts=parts, **b) == 0, (seed, parts, b)


@pytest.mark.parametrize("seed", range(4))
def test_warps_walk_alike_whatever_the_lengths_do(check, seed):
    r = random.Random(seed)
    apart = 0
    for b in batches(seed):
        new = [r.choice([1, 1, 8, 0]) for _ in b["lens"]]
        assert check(new=new, change=True, seed=seed + 1, **b) == 0, (seed, b)
        apart += check(new=new, change=True, own_reads=True, seed=seed + 1, **b) == 1
    assert apart  # the check does see walks that read memory for themselves part


def test_windows_move_on(check):
    """One CTA over thousands of items, most of them without a tile."""
    lens = [64 if i % 300 == 299 else 0 for i in range(5000)]
    assert check(lens, [1] * 5000, parts=1) == 0
    assert check([1] * 5000, [1] * 5000, parts=3) == 0
