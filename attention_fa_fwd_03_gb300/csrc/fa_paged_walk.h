// Which tiles of the split list of fa_paged_fwd a CTA takes: integers only, for the
// device and the host.
//
// All warps of a CTA walk the same segments, each in a role of its own, and meet at
// barriers that do not give up, once per segment. So they have to agree on every
// segment, whatever happens to the lengths in global memory meanwhile: a walk takes
// them from a copy that its CTA has made once (a window of items in shared memory),
// never from global memory itself. (A cluster's CTA has one segment, whatever the
// lengths are.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FA_WALK_FN __host__ __device__ __forceinline__
#else
#define FA_WALK_FN inline
#endif

namespace fa {

// Keys of a tile.
constexpr int kPagedTile = 64;
// Tiles of `units` units of `keys` keys.
inline int64_t paged_tiles(int64_t units, int64_t keys) { return units * ((keys + kPagedTile - 1) / kPagedTile); }
// Places that a unit counts for beside its tiles where the list of up to 16 rows over a cache
// held in 8 bits is cut (fa_paged8.cuh says why), as the host counts it too.
constexpr int kOver8 = 2;
inline int list_over(bool e4m3, int rows) { return e4m3 && rows <= 16 ? kOver8 : 0; }
// Places are counted in 32 bits on the device: whether those of the longest list can be.
inline bool list_fits(int64_t units, int64_t keys, int over) {
  return paged_tiles(units, keys) + units * over <= INT32_MAX;
}
// Items whose lengths a CTA holds at a time.
constexpr int kItemWindow = 128;

FA_WALK_FN int walk_min(int a, int b) { return a < b ? a : b; }
FA_WALK_FN int walk_max(int a, int b) { return a > b ? a : b; }
// of a power of two
FA_WALK_FN int walk_log2(int x) {
#ifdef __CUDA_ARCH__
  return 31 - __clz(x);
#else
  return 31 - __builtin_clz(static_cast<unsigned>(x));
#endif
}

// The list. An item is a sequence (every KV head and row block of it has the same
// tiles) or, with selected pages, a (sequence, KV head); `mult` units each.
struct ListShape {
  int items, mult;
  int sel, window, page_shift;
  int sinks;  // first keys that a window does not hide
  int over;   // tiles that a unit counts for beside its own, where beginning and ending one costs as much
};

// What the kernels read of an item, range-checked: keys, and new tokens (0 to 8)
// beside the number of selected pages (up to 2^20).
struct ItemLens {
  int len, rest;
  FA_WALK_FN static ItemLens of(int len, int n, int listed) { return {len, n | listed << 4}; }
};

struct Item {
  int len, n;  // keys and new tokens
  int listed;  // selected pages
  int head;    // first tiles of the list, kept for their visible first keys,
  int skip;    // and tiles behind them that hold no visible key
  int tiles;   // tiles of each unit
  // place in the list of the unit's tile t
  FA_WALK_FN int tile(int t) const { return head > 0 && t < head ? t : t + skip; }
};
FA_WALK_FN Item make_item(const ListShape& s, const ItemLens& x) {
  Item it;
  it.len = x.len;
  it.n = x.rest & 15;
  it.listed = x.rest >> 4;
  it.head = it.skip = 0;
  int keys = it.len;
  if (s.sel) {
    keys = it.listed << s.page_shift;  // at most 2^20 entries of 2^8 keys
  } else if (s.window > 0) {
    const int first = walk_max(0, it.len - it.n - s.window + 1) / kPagedTile;
    if (s.sinks > 0) it.head = walk_min(first, (s.sinks + kPagedTile - 1) / kPagedTile);
    it.skip = first - it.head;
  }
  it.tiles = it.n > 0 ? (keys + kPagedTile - 1) / kPagedTile - it.skip : 0;
  return it;
}

// What a unit of the item counts for when shares are cut: `over` places, then its tiles.
FA_WALK_FN int unit_places(const ListShape& s, const Item& it) { return it.tiles > 0 ? it.tiles + s.over : 0; }

// One CTA's share of the list: `total` places (tiles, where over is 0) in equal runs, the first total % parts
// of them one longer. (The host has checked that the longest possible list stays
// below 2^31 places.)
struct Share {
  int parts;      // CTAs with a share: every one of them has a tile
  int base, more; // tiles of a share, and how many have one more
  int lo, hi;
  int item, rest; // where lo falls: item, and tiles of it before lo
  FA_WALK_FN void divide(int total, int part, int all_parts) {
    parts = walk_min(total, all_parts);
    base = total / all_parts;
    more = total - base * all_parts;
    lo = part * base + walk_min(part, more);
    hi = lo + base + (part < more ? 1 : 0);
  }
  // CTA whose share holds place x of the list
  FA_WALK_FN int part_of(int x) const {
    const int longer = more * (base + 1);
    return x < longer ? x / (base + 1) : more + (x - longer) / base;
  }
};

// Walks the segments of a share: unit (item, sub), its tiles [t0, t1). `lens(item)`
// gives the CTA's copy of an item's lengths; items are asked for in ascending order,
// the share's first one first.
struct Walk {
  Item it;
  int item, sub;
  int t0, t1, left;
  int used;  // places of the share that the segment takes
  // The segment from place `r` of the unit on: false where the share ends before its first tile.
  FA_WALK_FN bool cut(const ListShape& list, int r) {
    if (list.over == 0) {  // (known where a kernel is compiled)
      t0 = r;
      t1 = walk_min(it.tiles, r + left);
      used = t1 - t0;
      return true;
    }
    const int tiles = walk_max(it.tiles, 1);
    t0 = walk_min(walk_max(r - list.over, 0), tiles - 1);
    t1 = walk_min(it.tiles, walk_max(r + left - list.over, t0));
    used = t1 - t0 + walk_max(walk_min(list.over, r + left) - r, 0);
    return t1 > t0;
  }
  template <class Lens>
  FA_WALK_FN bool start(const ListShape& list, const Share& s, Lens& lens) {
    left = s.hi - s.lo;
    if (left <= 0) return false;
    item = s.item;
    it = make_item(list, lens(item));
    // tiles and sub are in range unless the lengths have changed since the shares
    // were cut, which must not lead out of the buffers either
    const int places = walk_max(unit_places(list, it), 1);
    sub = walk_min(s.rest / places, list.mult - 1);
    return cut(list, walk_min(s.rest - sub * places, places - 1));
  }
  template <class Lens>
  FA_WALK_FN bool next(const ListShape& list, Lens& lens) {
    left -= used;
    if (left <= 0) return false;
    if (++sub == list.mult) {
      sub = 0;
      do {
        if (++item >= list.items) return false;  // (as above)
        it = make_item(list, lens(item));
      } while (it.tiles == 0);
    }
    return cut(list, 0);
  }
  // Clusters: unit `unit` as one segment, whose place does not depend on the lengths.
  // Of its tiles rank `rank` takes every `ranks`-th, a power of two, from its own number
  // on: [t0, t1) counts them.
  FA_WALK_FN void place_unit(const ListShape& list, int unit) {
    item = unit / list.mult;
    sub = unit - item * list.mult;
  }
  FA_WALK_FN void start_unit(const ListShape& list, int rank, int ranks, const ItemLens& x) {
    it = make_item(list, x);
    t0 = 0;
    t1 = (walk_max(it.tiles - rank, 0) + ranks - 1) >> walk_log2(ranks);
    left = t1;
  }
};

}  // namespace fa
