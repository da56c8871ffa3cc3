// Attention of up to 8 new tokens per sequence over the paged cache: the
// forward's online softmax, split over the cache's length and joined.
//
//   S = scale q K^T over visible keys, m = max S, l = sum 2^(S - m) (exp2
//   domain), O = sum 2^(S - m) V / l, LSE = (m + log2 l) ln 2
//
// What bounds it: every visible key's K and V row is read once and used by the
// (Hq / Hkv) * Tq query rows of its KV head, 4 D flops per row for 4 D bytes:
// at most a few tens of flops per byte, far below the tensor cores' ridge. So
// the kernel is built around keeping HBM busy.
//
// Split. A unit is a (sequence, KV head, block of 8 to 64 rows); its keys are cut
// into tiles of 64. Only the device knows the lengths, so every CTA of a grid that
// fills the GPU once sums the tiles of all units and takes an equal share of the
// whole list, whatever the lengths of the sequences. A share is a run of segments;
// those that cover a whole unit write O and LSE themselves, the others (at most the
// first and the last of a CTA) leave (m, l, unnormalised O) in the workspace and a
// second kernel joins them. Short lists skip all that: a cluster of CTAs takes a
// unit, tiles in turn, and joins through distributed shared memory. Either way the
// parts are joined in a fixed order, so results are the same on every run.
//
// Inside a CTA one warp looks up pages and loads tiles by TMA (one box per page
// piece and 64 columns, 128-byte swizzle) into a ring of stages; four warps per
// row block each take 16 keys of a tile and keep a running maximum and sum of
// their own, so tiles need no barrier between warps. Scores and outputs are
// m16n8k16 tensor-core products computed transposed, S^T = K Q^T and O^T = V^T P^T:
// keys and columns of V are the 16 rows of a fragment (read by ldmatrix straight
// from the tile), query rows its 8 columns, so a group of up to 8 heads fills a
// fragment that would be half empty the other way round.
//
// Split lists of more than 16 rows per KV head go to the kernel of fa_paged_tc.cuh,
// whose products are on tcgen05.
//
// Measured with 537 MB of keys and values of 8 units, share of the copy rate (6787
// GB/s): up to 8 rows 89 to 94% (D 64 89, D 96 and 128 91, D 256 94; 131072 keys of
// D 128 86 to 88 us, of which 4.5 are the join's launch and 3 the start), 16 rows 84 to
// 88%. There the tensor pipe is 14% active and the loads bound the kernel: a tcgen05 tile
// with its round trip through TMEM has nothing to gain. With more rows these products
// are bound by issue (about 270 instructions per warp and tile with two warps per
// scheduler): 64 rows of 269 MB took 111 us here, 58 on tcgen05. Such rows come here
// in clusters only.
#pragma once

#include "fa_inst.cuh"
#include "fa_paged_launch.h"
#include "fa_paged_mma.cuh"

namespace fa {

constexpr int kPagedKeyWarps = 4;       // warps that share a tile's keys, 16 each
constexpr int kPagedMaxRanks = 16;      // CTAs of a cluster (above 8: allowed per kernel)

struct PagedFwdArgs {
  PagedView c;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  int Hq, Tq, causal, window;
  float scale_log2;
  const int* new_lens;
  const int *sel, *sel_lens;
  int n_sel;
  int rows, row_blocks;  // query rows of a KV head and their blocks
  // workspace: parts of units, two slots per CTA (0: the unit began in an
  // earlier CTA, 1: it goes on in the next one)
  float* part_o;   // [2 parts][block rows][D]
  float2* part_ml; // [2 parts][block rows] (max, sum)
  // split units: (unit, first part | last part << 16), or unit = -1; by unit where
  // units are no more than CTAs, else by the CTA that began the unit
  int2* joins;
  int by_unit;
  WaitCfg wc;
};

// NT: groups of 8 query rows that a warp holds; RW: warps of other rows beside it.
template <int D_, int NT_, int RW_, bool BF16_, bool CLUSTER_>
struct PagedCfg {
  static constexpr int D = D_, NT = NT_, RW = RW_;
  static constexpr bool BF16 = BF16_;
  static constexpr bool CLUSTER = CLUSTER_;          // a cluster per unit instead of equal shares
  // Tiles per CTA up to which clusters are used. 64 rows, D 128, 16 units of 64 tiles (16
  // per CTA): 28.7 us, split 21.7; of 32 tiles: 18.0 and 18.4; 24 rows, 64 tiles 17.6 and 19.4.
  static constexpr int CLUSTER_TILES = NT == 4 ? 8 : 16;
  static constexpr int KW = kPagedKeyWarps;
  static constexpr int ROWS = 8 * NT * RW;           // rows of a block
  static constexpr int WARPS = KW * RW;              // consumer warps
  // One producer warp beside them; where accumulators need more registers than an
  // equal split leaves, a warpgroup of producers (one works) that gives its own up.
  static constexpr bool SPLIT = RW > 1 && NT * D >= 384;
  static constexpr int THREADS = 32 * (WARPS + (SPLIT ? 4 : 1));
  static constexpr int PRODUCERS = 1;
  static constexpr int REG_PRODUCER = 40, REG_CONSUMER = 224;
  static constexpr int REG_NEEDED = SPLIT ? 128 * REG_PRODUCER + 32 * WARPS * REG_CONSUMER : 0;
  static constexpr int KREG = (D + 63) / 64;         // 64-column regions of a row
  static constexpr int REGION = kPagedTile * 128;
  static constexpr int TILE = KREG * REGION;         // K (or V) rows of a stage
  // Up to 16 rows two CTAs share an SM with about 100 KB in flight each (D = 64 and
  // up to 8 rows: three; with 16, whose registers that would spill, 80% of the copy
  // rate against 84); with more rows, or 64 KB stages, one does.
  static constexpr int CTAS = D == 256 || RW > 1 ? 1 : D == 64 && NT == 1 ? 3 : 2;
  static constexpr int STAGES = D == 256  ? (RW == 1 ? 3 : 2)
                                : D == 64 ? (RW > 1 ? 8 : NT == 1 ? 4 : 6)
                                          : (RW == 1 ? 3 : 5);
  // Queries as B fragments in registers where they fit, else read again each tile
  static constexpr bool QREG = NT * D <= (CTAS == 1 && RW == 1 ? 256 : 128);
  static constexpr int QREGION = ROWS * 128;
  static constexpr int OP = D + 4;                   // row pitch of the merge buffers (floats): no bank conflicts
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = OFF_KV + STAGES * 2 * TILE;
  static constexpr int OFF_O = OFF_Q + KREG * QREGION;
  static constexpr int OFF_ML = OFF_O + ROWS * OP * 4;
  static constexpr int OFF_PML = OFF_ML + KW * ROWS * 8;  // clusters: (max, sum) beside every piece received
  static constexpr int SMEM_BYTES = OFF_PML + (CLUSTER ? ROWS * D : 0) + 1024;
  // clusters: the warps' rows at the end, over the stages and the queries
  static_assert(KW * ROWS * OP * 4 <= OFF_O, "warps' rows");
  static_assert(SMEM_BYTES <= 229000, "shared memory");  // beside the static variables
  static_assert(ROWS * (D / 8) % kPagedMaxRanks == 0, "pieces of a cluster");
};

// Running maxima may be behind by this much (in the exp2 domain) before the sums
// are rescaled: weights then reach 2^8 instead of 1, which costs no precision.
constexpr float kPagedSlack = 8.f;
// Running maximum of a row that has seen no key: finite, so that a hidden score of
// -inf less it is -inf, and the lowest number, so that any score raises it.
constexpr float kNoMax = -3.402823466e38f;
// An exponent is s scale - m in one rounding; m is the rounded s scale of some key, so
// that key's own exponent is up to half a step of m instead of 0. Beyond this magnitude
// of m a step is no longer small and soon past what an exponent can hold: the scores
// are then scaled and rounded first, like m.
constexpr float kLargeMax = 4194304.f;  // 2^22: steps of 1/2
__device__ __forceinline__ bool large_max(float m) { return fabsf(m) > kLargeMax && m != kNoMax; }

// ----------------------------------------------------------------- the list
__device__ __forceinline__ ListShape list_shape(const PagedFwdArgs& p) {
  return {p.sel ? p.c.B * p.c.Hkv : p.c.B, (p.sel ? 1 : p.c.Hkv) * p.row_blocks, p.sel != nullptr, p.window,
          p.c.page_shift};
}
__device__ __forceinline__ int item_seq(const PagedFwdArgs& p, int item) { return p.sel ? item / p.c.Hkv : item; }
__device__ __forceinline__ ItemLens load_lens(const PagedFwdArgs& p, int item) {
  const int listed = p.sel ? p.sel_lens[item] : 0;
  const SeqLens sl = seq_lens(p.c, p.new_lens, item_seq(p, item), p.Tq);
  return ItemLens::of(sl.len, sl.n, p.sel ? checked_count(p.c, listed, p.n_sel) : 0);
}
// Clusters: a warp's own reading of its unit's lengths, one value for all its lanes.
// Warps differ only if somebody writes the lengths under the call. They then wait for
// tiles that never come, up to the time limit, and no longer: barriers without one are
// met the same number of times whatever the lengths are.
__device__ __forceinline__ ItemLens load_lens_warp(const PagedFwdArgs& p, int item) {
  ItemLens x = load_lens(p, item);
  x.len = __shfl_sync(0xffffffffu, x.len, 0);
  x.rest = __shfl_sync(0xffffffffu, x.rest, 0);
  return x;
}
__device__ __forceinline__ int kv_head(const PagedFwdArgs& p, const Walk& w) {
  return p.sel ? w.item % p.c.Hkv : w.sub / p.row_blocks;
}
__device__ __forceinline__ int row_block(const PagedFwdArgs& p, const Walk& w) { return w.sub % p.row_blocks; }

// The CTA's copy of items' lengths, in shared memory: items [base, base + kItemWindow).
// Every warp of the CTA has one of these and walks the whole share with it, so all
// come to the barriers of a window that moves on.
template <int THREADS>
struct ItemWindow {
  const PagedFwdArgs& p;
  ItemLens* slots;
  int items, base;
  // by all threads, with a barrier behind it
  __device__ __forceinline__ void fill(int from) {
    base = from;
    const int i = threadIdx.x;
    if (i < kItemWindow && base + i < items) slots[i] = load_lens(p, base + i);
  }
  __device__ __forceinline__ ItemLens operator()(int item) {
    if (item - base >= kItemWindow) {
      __syncwarp();
      named_bar_sync(2, THREADS);  // all have read what they need of the old window
      fill(item);
      named_bar_sync(2, THREADS);
    }
    return slots[item - base];
  }
};

// A CTA's share, found by all its threads, which also fill the window for its walk.
template <int THREADS>
__device__ __forceinline__ Share find_share(const PagedFwdArgs& p, const ListShape& list, int part, int parts,
                                            ItemWindow<THREADS>& window) {
  static_assert(THREADS >= kItemWindow, "one item per thread");
  __shared__ int sums[THREADS / 32];
  __shared__ int found_rest, found_item;
  const int per = (list.items + THREADS - 1) / THREADS;
  const int i0 = min(list.items, static_cast<int>(threadIdx.x) * per), i1 = min(list.items, i0 + per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool whole = list.items <= kItemWindow;  // the window holds the list: one item per thread
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    const ItemLens x = load_lens(p, i);
    if (whole) window.slots[i] = x;
    mine += make_item(list, x).tiles * list.mult;
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  if (threadIdx.x == 0) found_item = found_rest = 0;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  Share s;
  s.divide(total, part, parts);
  if (s.lo >= before && s.lo < before + mine) {
    int rest = s.lo - before;
    int i = i0;
    for (; i < i1 - 1; ++i) {
      const int n = make_item(list, load_lens(p, i)).tiles * list.mult;
      if (rest < n) break;
      rest -= n;
    }
    found_item = i;
    found_rest = rest;
  }
  __syncthreads();
  s.item = found_item;
  s.rest = found_rest;
  if (!whole) {
    window.fill(s.item);
    __syncthreads();
  }
  return s;
}

// Row 0 of block `rb` of (b, g) among the rows of q, o and lse.
__device__ __forceinline__ int64_t block_row0(const PagedFwdArgs& p, int b, int g, int rb, int block_rows) {
  return (static_cast<int64_t>(b) * p.c.Hkv + g) * p.rows + rb * block_rows;
}

__device__ __forceinline__ void scale4(float4& a, float f) {
  a.x *= f;
  a.y *= f;
  a.z *= f;
  a.w *= f;
}
__device__ __forceinline__ void add4(float4& a, const float4& x, float f) {
  a.x = fmaf(x.x, f, a.x);
  a.y = fmaf(x.y, f, a.y);
  a.z = fmaf(x.z, f, a.z);
  a.w = fmaf(x.w, f, a.w);
}

// O = sum / l and LSE of one row chunk of 8 values.
template <bool BF16>
__device__ __forceinline__ void store_out8(uint16_t* dst, const float4& x, const float4& y, float inv) {
  uint4 w;
  w.x = pack2<BF16>(x.x * inv, x.y * inv);
  w.y = pack2<BF16>(x.z * inv, x.w * inv);
  w.z = pack2<BF16>(y.x * inv, y.y * inv);
  w.w = pack2<BF16>(y.z * inv, y.w * inv);
  *reinterpret_cast<uint4*>(dst) = w;
}
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f || l != l ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

// Maximum and sum of row r over the key warps' own.
template <class C>
__device__ __forceinline__ float2 warps_max_sum(const float2* mls, int r) {
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < C::KW; ++k) m = fmaxf(m, mls[k * C::ROWS + r].x);
#pragma unroll
  for (int k = 0; k < C::KW; ++k) l += mls[k * C::ROWS + r].y * exp2_rel(mls[k * C::ROWS + r].x, m);
  return make_float2(m, l);
}

// Eight columns of a row of a segment, the sums not normalised: the output where the
// segment is the whole unit, else the part `part_slot`.
template <class C>
__device__ __forceinline__ void put_piece(const PagedFwdArgs& p, bool whole, int part_slot, int64_t row0, int r, int ch,
                                          const float4& x, const float4& y, float2 ml) {
  if (whole) {
    store_out8<C::BF16>(p.o + (row0 + r) * C::D + 8 * ch, x, y, ml.y == 0.f ? 0.f : 1.f / ml.y);
    if (ch == 0) p.lse[row0 + r] = row_lse(ml.x, ml.y);
  } else {
    float4* dst = reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(part_slot) * C::ROWS + r) * C::D + 8 * ch);
    dst[0] = x;
    dst[1] = y;
    if (ch == 0) p.part_ml[part_slot * C::ROWS + r] = ml;
  }
}

// By one thread after a segment: whether the unit it began is split, and over which parts.
__device__ __forceinline__ void record_unit(const PagedFwdArgs& p, const ListShape& list, const Share& share,
                                            const Walk& w, int part) {
  const bool ends = w.t1 == w.it.tiles;
  if (w.t0 != 0 || (ends && !p.by_unit)) return;
  const int unit = w.item * list.mult + w.sub;
  // the unit goes on to tile share.hi - t1 + tiles of the list
  const int last = ends ? 0 : min(share.part_of(share.hi - w.t1 + w.it.tiles - 1), share.parts - 1);
  p.joins[p.by_unit ? unit : part] = make_int2(ends ? -1 : unit, part | last << 16);
}

// Units without tiles: nothing is visible to any of their rows.
template <class C>
__device__ __forceinline__ void write_empty_units(const PagedFwdArgs& p, const ListShape& list, int part, int parts, int tid,
                                                  int threads) {
  const int64_t units = static_cast<int64_t>(list.items) * list.mult;
  for (int64_t u = part; u < units; u += parts) {
    const int item = static_cast<int>(u / list.mult), sub = static_cast<int>(u - static_cast<int64_t>(item) * list.mult);
    if (make_item(list, load_lens(p, item)).tiles > 0) continue;
    const int g = p.sel ? item % p.c.Hkv : sub / p.row_blocks, rb = sub % p.row_blocks;
    const int64_t row0 = block_row0(p, item_seq(p, item), g, rb, C::ROWS);
    const int rows = min(C::ROWS, p.rows - rb * C::ROWS);
    for (int i = tid; i < rows * (C::D / 8); i += threads)
      reinterpret_cast<uint4*>(p.o + row0 * C::D)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < rows; i += threads) p.lse[row0 + i] = -INFINITY;
    if (tid == 0 && p.by_unit) p.joins[u] = make_int2(-1, 0);
  }
}

// Stores to CTA `rank`'s shared memory, at the place `at` has in this CTA's.
__device__ __forceinline__ void st_peer_f2(const void* at, uint32_t rank, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_addr(smem_u32(at), rank)), "f"(v.x), "f"(v.y)
               : "memory");
}
__device__ __forceinline__ void st_peer_f4(const void* at, uint32_t rank, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(peer_addr(smem_u32(at), rank)), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// What the lengths will lead to, on its way into L2 before they are known: this
// CTA's part of the page table (or of the selections) and of the queries.
template <class C>
__device__ __forceinline__ void prefetch_inputs(const PagedFwdArgs& p, int part) {
  const PagedView& c = p.c;
  const int64_t t = static_cast<int64_t>(part) * C::THREADS + threadIdx.x;
  const int64_t entries = p.sel ? static_cast<int64_t>(c.B) * c.Hkv * p.n_sel : static_cast<int64_t>(c.B) * c.max_pages;
  const int64_t q_lines = static_cast<int64_t>(c.B) * c.Hkv * p.rows * (C::D / 64);
  if (t * 32 < entries) prefetch_l2((p.sel ? p.sel : c.table) + t * 32);
  if (t < q_lines) prefetch_l2(p.q + t * 64);
}

// Not 0 where one of two packed values is infinite or NaN: exponent bits all set, so
// that one more in the lowest of them carries into the sign's place.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) {
  constexpr uint32_t e = BF16 ? 0x7f807f80u : 0x7c007c00u, one = BF16 ? 0x00800080u : 0x04000400u;
  return ((x & e) + one) & 0x80008000u;
}

// A position no query reaches: the key's slot was not loaded. (Positions end below
// 2^30, and so do windows: differences of any two of these and this stay in 32 bits.)
constexpr int kNoPosition = 1 << 30;

// A producer warp's side of a CTA's ring of K and V tiles: all of them, or with two
// producers (C::PRODUCERS) every other one.
template <class C>
struct TileRing {
  const PagedFwdArgs& p;
  const CUtensorMap &map_k, &map_v;
  uint32_t kv, full, empty;          // shared addresses: stages, barriers
  int (*key_pos)[kPagedKeyWarps];    // position of the first of each 16 keys of a stage
  int* abort_flag;
  int piece, pieces;                 // keys of a page in one tile, pages of a tile
  int lane, producer, issued = 0;      // (those of the other producer count too)
  bool ok = true;
  __device__ __forceinline__ TileRing(const PagedFwdArgs& p_, const CUtensorMap& mk, const CUtensorMap& mv, uint32_t kv_,
                                      uint64_t* full_, uint64_t* empty_, int (*key_pos_)[kPagedKeyWarps], int* abort_,
                                      int producer_ = 0)
      : p(p_), map_k(mk), map_v(mv), kv(kv_), full(smem_u32(full_)), empty(smem_u32(empty_)), key_pos(key_pos_),
        abort_flag(abort_), piece(min(1 << p_.c.page_shift, kPagedTile)), pieces(kPagedTile / piece),
        lane(threadIdx.x & 31), producer(producer_) {}
  __device__ __forceinline__ bool mine(int tile) const { return C::PRODUCERS == 1 || tile % C::PRODUCERS == producer; }
  // One tile of KV head g into the next stage: lane i < pieces has the page (in the
  // sequence, and in the pool or -1) of its piece i, whose first key is key `x` of
  // the list plus i pieces.
  __device__ __forceinline__ void load(int x, int pg, int id, int g) {
    const PagedView& c = p.c;
    if (!mine(issued)) {
      ++issued;
      return;
    }
    const int slot = issued % C::STAGES;
    if (issued >= C::STAGES)
      ok = mbar_wait(empty + 8 * slot, ((issued / C::STAGES) - 1) & 1, p.wc.timeout_cycles, abort_flag, p.wc.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    const int off = (x + lane * piece) & ((1 << c.page_shift) - 1);
    const bool load = lane < pieces && id >= 0;
    if (lane < kPagedKeyWarps) {
      const int pl = (lane * 16) / piece;  // piece that holds these 16 keys
      const int kpage = __shfl_sync(0xfu, pg, pl), kid = __shfl_sync(0xfu, id, pl), koff = __shfl_sync(0xfu, off, pl);
      key_pos[slot][lane] = kid >= 0 ? (kpage << c.page_shift) + koff + lane * 16 - pl * piece : kNoPosition;
    }
    const unsigned loads = __ballot_sync(0xffffffffu, load);
    const uint32_t bar = full + 8 * slot, box = static_cast<uint32_t>(piece) * 128u;
    __syncwarp();  // lane 0 arrives for the positions of all four lanes (a vote orders no memory)
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(loads) * box * 2 * C::KREG);
    __syncwarp();
    if (load) {
      const uint32_t dst = kv + slot * 2 * C::TILE + lane * box;
      const int z = id * c.Hkv + g;
#pragma unroll
      for (int r = 0; r < C::KREG; ++r) {
        tma_load_3d(dst + r * C::REGION, &map_k, bar, r * 64, off, z);
        tma_load_3d(dst + C::TILE + r * C::REGION, &map_v, bar, r * 64, off, z);
      }
    }
    __syncwarp();
    ++issued;
  }
  // Stay until the last loads have landed: the consumers have waited for them too,
  // unless one of their waits gave up.
  __device__ __forceinline__ void drain() const {
    if (lane != 0) return;
    for (int i = max(0, issued - C::STAGES); i < issued; ++i)
      if (mine(i)) mbar_wait(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, p.wc.drain_cycles, nullptr, p.wc.status);
  }
};

// All tiles of a share, by the producer warp. (A wait that gave up ends the loads, not
// the walk: the window moves on with every warp.)
template <class C>
__device__ __forceinline__ void produce_share(const PagedFwdArgs& p, const ListShape& list, const Share& share,
                                              ItemWindow<C::THREADS>& window, TileRing<C>& ring) {
  const PagedView& c = p.c;
  const int lane = ring.lane;
  Walk w;
  for (bool more = w.start(list, share, window); more; more = w.next(list, window)) {
    if (!ring.ok) continue;
    const int b = item_seq(p, w.item), g = kv_head(p, w);
    const int pages = (w.it.len + (1 << c.page_shift) - 1) >> c.page_shift;
    const int64_t u = static_cast<int64_t>(b) * c.Hkv + g;
    const int count = p.sel ? w.it.listed : pages;
    // pages of list entries [e0, e0 + 32) and the next 32, one per lane
    auto look_up = [&](int e, int* page, int* id) {
      *page = -1;
      *id = -1;
      if (e >= count) return;
      int pg = e;
      if (p.sel) {
        pg = p.sel[u * p.n_sel + e];
        if (pg < 0 || pg >= pages) {
          flag_bad_index(c);
          return;
        }
      }
      *page = pg;
      *id = pool_page(c, b, pg);
    };
    int e0 = ((w.it.first + w.t0) * kPagedTile) >> c.page_shift;
    int page0, id0, page1, id1;
    look_up(e0 + lane, &page0, &id0);
    look_up(e0 + 32 + lane, &page1, &id1);
    for (int t = w.t0; t < w.t1 && ring.ok; ++t) {
      const int x = (w.it.first + t) * kPagedTile;  // first key of the tile in the list
      int e = (x >> c.page_shift) - e0;
      if (e >= 32) {
        e0 += 32;
        e -= 32;
        page0 = page1;
        id0 = id1;
        look_up(e0 + 32 + lane, &page1, &id1);
      }
      // lane i looks at piece i of the tile
      const int my = e + ((lane * ring.piece) >> c.page_shift);  // below 32: pages of 16 start tiles at multiples of 4
      ring.load(x, __shfl_sync(0xffffffffu, page0, my & 31), __shfl_sync(0xffffffffu, id0, my & 31), g);
    }
  }
}

// ------------------------------------------------------------------- kernel
template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
fa_paged_fwd_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const PagedFwdArgs p, int ranks) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[C::STAGES], empty[C::STAGES];
  __shared__ int key_pos[C::STAGES][C::KW];  // position of the first of each warp's 16 keys
  __shared__ ItemLens item_lens[C::CLUSTER ? 1 : kItemWindow];
  __shared__ int abort_flag;
  constexpr int D = C::D;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedView& c = p.c;
  const ListShape list = list_shape(p);
  const int part = blockIdx.x, parts = gridDim.x;
  const uint64_t tmo = p.wc.timeout_cycles;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), C::WARPS);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * C::WARPS) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  // (a cluster of one has no peers and needs no barriers)
  if (C::CLUSTER && ranks > 1) cluster_arrive_relaxed();  // waited for before the first store into a peer
  grid_wait_prior();
  grid_release_next();
  prefetch_inputs<C>(p, part);
  const int rank = C::CLUSTER ? part % ranks : 0, unit = C::CLUSTER ? part / ranks : 0;
  Share share;
  ItemWindow<C::THREADS> window{p, item_lens, list.items, 0};
  if constexpr (C::CLUSTER)
    __syncthreads();
  else
    share = find_share<C::THREADS>(p, list, part, parts, window);  // barriers inside

  if (warp >= C::WARPS) {
    // ---------------------------------------------------------- producer warp
    if constexpr (C::SPLIT) {
      regs_release<C::REG_PRODUCER>();
      if (warp > C::WARPS) {
        if (C::CLUSTER && ranks > 1) {
          cluster_wait();
          cluster_barrier();
        }
        return;
      }
    }
    TileRing<C> ring(p, map_k, map_v, sbase + C::OFF_KV, full, empty, key_pos, &abort_flag);
    const int piece = ring.piece, pieces = ring.pieces;
    if constexpr (C::CLUSTER) {
      // Lane k * pieces + i looks up piece i of the k-th tile of a batch of as many of
      // the CTA's tiles as 32 lanes hold, the first batch, where no window moves the
      // first tile, while the lengths that say which of it counts are still on their
      // way: what is read too much is not used.
      Walk w;
      w.place_unit(list, unit);
      const int b = item_seq(p, w.item), g = kv_head(p, w);
      const int64_t u = static_cast<int64_t>(b) * c.Hkv + g;
      const int64_t row = static_cast<int64_t>(b) * c.max_pages;
      const int batch = 32 / pieces, mine = lane / pieces, key = (lane & (pieces - 1)) * piece;
      int first = 0, pg = -1, id = -1, e = 0;
      auto read = [&](int t0) {
        e = (first + (rank + (t0 + mine) * ranks) * kPagedTile + key) >> c.page_shift;
        pg = e;
        id = -1;
        if (p.sel) pg = e < p.n_sel ? p.sel[u * p.n_sel + e] : -1;
        if (static_cast<unsigned>(pg) < static_cast<unsigned>(c.max_pages)) id = c.table[row + pg];
      };
      const bool early = p.sel != nullptr || p.window == 0;
      if (early) read(0);
      w.start_unit(list, rank, ranks, load_lens_warp(p, w.item));
      first = w.it.first * kPagedTile;
      const int pages = (w.it.len + (1 << c.page_shift) - 1) >> c.page_shift;
      const int count = p.sel ? w.it.listed : pages;
      for (int t0 = 0; t0 < w.t1 && ring.ok; t0 += batch) {
        if (t0 > 0 || !early) read(t0);
        const bool counts = t0 + mine < w.t1 && e < count;
        if (counts && static_cast<unsigned>(pg) < static_cast<unsigned>(pages)) {
          id = checked_page(c, id);
        } else {
          if (counts) flag_bad_index(c);  // a selected page that the sequence does not have
          id = -1;
        }
        for (int t = t0; t < min(w.t1, t0 + batch) && ring.ok; ++t) {
          const int from = (t - t0) * pieces + (lane & (pieces - 1));
          ring.load(first + (rank + t * ranks) * kPagedTile, __shfl_sync(0xffffffffu, pg, from),
                    __shfl_sync(0xffffffffu, id, from), g);
        }
      }
    } else {
      produce_share(p, list, share, window, ring);
    }
    ring.drain();
    if (C::CLUSTER && ranks > 1) {  // as the consumers do
      __syncwarp();
      cluster_wait();
      cluster_barrier();
    }
    return;
  }

  // ------------------------------------------------------------ consumer warps
  if constexpr (C::SPLIT) regs_claim<C::REG_CONSUMER>();
  const int kw = warp % C::KW, rw = warp / C::KW;
  const int tid = threadIdx.x;
  float* om = reinterpret_cast<float*>(smem + C::OFF_O);
  float2* mls = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [KW][ROWS]
  auto sync_rows = [&] { named_bar_sync(1, 32 * C::WARPS); };

  if constexpr (!C::CLUSTER) {
    if (tid == 0 && !p.by_unit) p.joins[part] = make_int2(-1, 0);
  }

  // a block's query rows to shared memory, rows behind the last one zero
  auto stage_queries = [&](int64_t row0, int rows) {
    for (int i = tid; i < C::ROWS * (D / 8); i += 32 * C::WARPS) {
      const int r = i / (D / 8), ch = i - r * (D / 8);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < rows) x = reinterpret_cast<const uint4*>(p.q + (row0 + r) * D)[ch];
      *reinterpret_cast<uint4*>(smem + C::OFF_Q + (ch >> 3) * C::QREGION + sw128_offset(r, ch & 7)) = x;
    }
  };
  if constexpr (C::CLUSTER) {  // where the unit's rows are does not depend on the lengths
    const int rb = unit % p.row_blocks;
    stage_queries(static_cast<int64_t>(unit / p.row_blocks) * p.rows + rb * C::ROWS, min(C::ROWS, p.rows - rb * C::ROWS));
  }

  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  bool more = true;  // clusters: one segment, which may be empty
  Walk w;
  if constexpr (C::CLUSTER) {
    w.place_unit(list, unit);
    w.start_unit(list, rank, ranks, load_lens_warp(p, w.item));
  } else {
    more = w.start(list, share, window);
  }
  for (; more; more = !C::CLUSTER && w.next(list, window)) {
    const int g = kv_head(p, w), rb = row_block(p, w);
    const int rows = min(C::ROWS, p.rows - rb * C::ROWS);
    const int64_t row0 = block_row0(p, item_seq(p, w.item), g, rb, C::ROWS);
    // this thread's columns are rows 2 (lane % 4) and the next of each group of 8
    const int group0 = rw * C::NT, col0 = group0 * 8 + 2 * (lane & 3);
    const bool has_rows = group0 * 8 < rows;
    // tokens of this thread's rows, four bits each
    uint64_t tokens = 0;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        tokens |= static_cast<uint64_t>((rb * C::ROWS + col0 + 8 * nt + e) % p.Tq) << (8 * nt + 4 * e);
    auto token = [&](int nt, int e) { return static_cast<int>(tokens >> (8 * nt + 4 * e)) & 15; };
    if constexpr (!C::CLUSTER) stage_queries(row0, rows);
    sync_rows();
    // B fragments of the queries: two products' worth per 8 rows and 32 columns
    const uint32_t qs = sbase + C::OFF_Q;
    auto query_frag = [&](uint32_t (&f)[4], int nt, int k2) {
      const int row = (group0 + nt) * 8 + (lane & 7), ch = 4 * k2 + (lane >> 3);
      ldsm4(f, qs + (ch >> 3) * C::QREGION + sw128_offset(row, ch & 7));
    };
    uint32_t qf[C::QREG ? C::NT : 1][C::QREG ? D / 32 : 1][4];
    if constexpr (C::QREG) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) query_frag(qf[nt][k2], nt, k2);
    }
    float m[C::NT][2], l[C::NT][2], acc[C::NT][D / 16][4];
    bool large = false;  // some row of the warp has a large maximum
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoMax;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }
    const int len = w.it.len, n = w.it.n;
    const int p_lo = len - n, p_hi = len - 1;  // positions of the new tokens

    for (int t = w.t0; t < w.t1; ++t) {
      ok = ok && mbar_wait(smem_u32(&full[slot]), phase, tmo, &abort_flag, p.wc.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int j0 = key_pos[slot][kw];
      const uint32_t ks = sbase + C::OFF_KV + slot * 2 * C::TILE, vs = ks + C::TILE;
      // does any row see any of the 16 keys; do all rows see all of them
      const bool some = has_rows && j0 < len && !(p.window > 0 && j0 + 15 <= p_lo - p.window);
      if (some) {
        const bool all = j0 + 15 < len && !(p.causal && j0 + 15 > p_lo) && !(p.window > 0 && j0 <= p_hi - p.window);
        // S^T = K Q^T: element e of group nt is key j0 + lane / 4 + 8 (e / 2), row
        // col0 + 8 nt + e % 2. One group: two accumulators, half as long a chain.
        float s[C::NT][4], s2[4];
        const int kr = kw * 16 + (lane & 15), kc = lane >> 4;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t a0[4], a1[4];
          ldsm4(a0, ks + (k2 >> 1) * C::REGION + sw128_offset(kr, (4 * k2 + kc) & 7));
          ldsm4(a1, ks + (k2 >> 1) * C::REGION + sw128_offset(kr, (4 * k2 + 2 + kc) & 7));
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt) {
            uint32_t b[4];
            if constexpr (C::QREG) {
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] = qf[nt][k2][e];
            } else {
              query_frag(b, nt, k2);
            }
            if (k2 == 0)
              mma16816_first<C::BF16>(s[nt], a0, b[0], b[1]);
            else
              mma16816<C::BF16>(s[nt], a0, b[0], b[1]);
            if (C::NT == 1 && k2 == 0)
              mma16816_first<C::BF16>(s2, a1, b[2], b[3]);
            else
              mma16816<C::BF16>(C::NT == 1 ? s2 : s[nt], a1, b[2], b[3]);
          }
        }
        if constexpr (C::NT == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] += s2[e];
        }
        uint32_t keep0 = ~0u, keep1 = ~0u;  // keys of this thread's V fragments that some row sees
        const int jv = j0 + 2 * (lane & 3);
        if (!all) {
          // keys [j0 + lo, j0 + lo + span) are seen by a column's row; this thread's are
          // j0 + lane / 4 and 8 behind it
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pos = p_lo + token(nt, h);
              const int lo = p.window > 0 ? pos - p.window + 1 - j0 : -j0;
              const int hi = (p.causal ? min(len, pos + 1) : len) - j0;
              const unsigned span = static_cast<unsigned>(max(hi - lo, 0)), j = (lane >> 2) - lo;
              if (j >= span) s[nt][h] = -INFINITY;
              if (j + 8 >= span) s[nt][2 + h] = -INFINITY;
            }
          auto seen = [&](int j) { return j < len && !(p.window > 0 && j <= p_lo - p.window); };
          keep0 = (seen(jv) ? 0xffffu : 0u) | (seen(jv + 1) ? 0xffff0000u : 0u);
          keep1 = (seen(jv + 8) ? 0xffffu : 0u) | (seen(jv + 9) ? 0xffff0000u : 0u);
        }
        // Exponents against the running maxima of this warp's keys, which are looked
        // at across lanes only when some exponent is above the slack.
        float x[C::NT][4];
        bool above = large;
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[nt][e] = fmaf(s[nt][e], p.scale_log2, -m[nt][e & 1]);
            above |= x[nt][e] > kPagedSlack;
          }
        }
        if (__any_sync(0xffffffffu, above)) {
          bool any_large = false;
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float y = fmaxf(s[nt][h], s[nt][2 + h]);
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
              const float mn = fmaxf(m[nt][h], y * p.scale_log2);
              alpha[h] = ex2(m[nt][h] - mn);
              m[nt][h] = mn;
              any_large |= large_max(mn);
              l[nt][h] *= alpha[h];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[nt][i][0] *= alpha[0];
              acc[nt][i][1] *= alpha[1];
              acc[nt][i][2] *= alpha[0];
              acc[nt][i][3] *= alpha[1];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(s[nt][e], p.scale_log2, -m[nt][e & 1]);
          }
          large = __any_sync(0xffffffffu, any_large);
          if (large) {
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[nt][e] = __fmul_rn(s[nt][e], p.scale_log2) - m[nt][e & 1];
          }
        }
        // Weights in two words of the cache's type, p = hi + lo to 2^-17 (bf16) or
        // 2^-22 (fp16) of p, and transposed into B fragments: with hi alone O would be
        // off by 1.4 times as much as its own rounding makes it. The products with lo
        // cost no time where the tiles' bytes bound the kernel.
        uint32_t pb[C::NT][2], pl[C::NT][2];
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[nt][h] = ex2(x[nt][h]);
            s[nt][2 + h] = ex2(x[nt][2 + h]);
            l[nt][h] += s[nt][h] + s[nt][2 + h];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t hi = pack2<C::BF16>(s[nt][2 * h], s[nt][2 * h + 1]);
            const float2 f = unpack2<C::BF16>(hi);
            pb[nt][h] = transpose8(hi);
            pl[nt][h] = transpose8(pack2<C::BF16>(s[nt][2 * h] - f.x, s[nt][2 * h + 1] - f.y));
          }
        }
        // O^T += V^T P^T. A key hidden from every row gets V = 0 (its slot may hold
        // anything; 0 * NaN would not be 0). Where rows differ in what they see and
        // some of these values are no finite numbers, each token's product is
        // taken with the keys it sees and only its rows are kept.
        const int vr = kw * 16 + ((lane >> 4) << 3) + (lane & 7), vc = (lane >> 3) & 1;
        const bool differ = !all && n > 1 &&
                            ((p.causal && j0 + 15 > p_lo && j0 <= p_hi) ||
                             (p.window > 0 && j0 <= p_hi - p.window && j0 + 15 > p_lo - p.window));
        bool apart = false;
        if (differ) {
          uint32_t odd = 0;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldsm4_trans(a, vs + (i >> 2) * C::REGION + sw128_offset(vr, (2 * i + vc) & 7));
            odd |= not_finite2<C::BF16>(a[0] & keep0) | not_finite2<C::BF16>(a[1] & keep0) |
                   not_finite2<C::BF16>(a[2] & keep1) | not_finite2<C::BF16>(a[3] & keep1);
          }
          apart = __any_sync(0xffffffffu, odd != 0);
        }
        if (!apart) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldsm4_trans(a, vs + (i >> 2) * C::REGION + sw128_offset(vr, (2 * i + vc) & 7));
            a[0] &= keep0;
            a[1] &= keep0;
            a[2] &= keep1;
            a[3] &= keep1;
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt)
              mma16816<C::BF16>(acc[nt][i], a, pb[nt][0], pb[nt][1]);
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt) mma16816<C::BF16>(acc[nt][i], a, pl[nt][0], pl[nt][1]);
          }
        } else {
#pragma unroll 1
          for (int tok = 0; tok < n; ++tok) {
            const int pos = p_lo + tok;
            auto seen = [&](int j) {
              return j < len && !(p.causal && j > pos) && !(p.window > 0 && j <= pos - p.window);
            };
            const uint32_t k0 = (seen(jv) ? 0xffffu : 0u) | (seen(jv + 1) ? 0xffff0000u : 0u);
            const uint32_t k1 = (seen(jv + 8) ? 0xffffu : 0u) | (seen(jv + 9) ? 0xffff0000u : 0u);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint32_t a[4];
              ldsm4_trans(a, vs + (i >> 2) * C::REGION + sw128_offset(vr, (2 * i + vc) & 7));
              a[0] &= k0;
              a[1] &= k0;
              a[2] &= k1;
              a[3] &= k1;
#pragma unroll
              for (int nt = 0; nt < C::NT; ++nt) {
                float x[4] = {acc[nt][i][0], acc[nt][i][1], acc[nt][i][2], acc[nt][i][3]};
                mma16816<C::BF16>(x, a, pb[nt][0], pb[nt][1]);
                mma16816<C::BF16>(x, a, pl[nt][0], pl[nt][1]);
                if (token(nt, 0) == tok) acc[nt][i][0] = x[0], acc[nt][i][2] = x[2];
                if (token(nt, 1) == tok) acc[nt][i][1] = x[1], acc[nt][i][3] = x[3];
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
      if (++slot == C::STAGES) {
        slot = 0;
        phase ^= 1;
      }
    }

    // merge the key warps
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float& x = l[nt][h];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        // padding rows (tokens the sequence does not have) see nothing; a row that has
        // met nothing but NaN keeps it
        if (token(nt, h) >= n || (m[nt][h] == kNoMax && x == 0.f)) {
          m[nt][h] = -INFINITY;
          x = 0.f;
        }
        if (lane < 4) mls[kw * C::ROWS + col0 + 8 * nt + h] = make_float2(m[nt][h], x);
      }
    sync_rows();  // and nobody reads stages any more
    if constexpr (C::CLUSTER) {
      // The warps' rows side by side; a thread adds up the four of an 8-column
      // piece and sends the sum with its maximum and sum of weights to the CTA
      // that owns the piece (i mod ranks), which joins what all CTAs sent.
      float* wm = reinterpret_cast<float*>(smem);  // [KW][ROWS][OP]
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            wm[(kw * C::ROWS + col0 + 8 * nt + (e & 1)) * C::OP + 16 * i + (lane >> 2) + 8 * (e >> 1)] =
                  acc[nt][i][e];
      sync_rows();
      const int pieces = rows * (D / 8), share_of = C::ROWS * (D / 8) / ranks;
      float2* pml = reinterpret_cast<float2*>(smem + C::OFF_PML);  // [ranks][share_of]
      __syncwarp();
      if (ranks > 1) cluster_wait();  // every CTA of the cluster is running
      for (int i = tid; i < pieces; i += 32 * C::WARPS) {
        const int r = i / (D / 8), ch = i - r * (D / 8);
        float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
        const float2 ml = warps_max_sum<C>(mls, r);
#pragma unroll
        for (int k = 0; k < C::KW; ++k) {
          const float mk = mls[k * C::ROWS + r].x;
          if (mk == -INFINITY) continue;  // nothing seen: not even 0 * inf
          const float f = ex2(mk - ml.x);
          const float* x = wm + (k * C::ROWS + r) * C::OP + 8 * ch;
          const float4 u = *reinterpret_cast<const float4*>(x), v = *reinterpret_cast<const float4*>(x + 4);
          add4(s0, u, f);
          add4(s1, v, f);
        }
        if (ranks == 1) {
          store_out8<C::BF16>(p.o + (row0 + r) * D + 8 * ch, s0, s1, ml.y == 0.f ? 0.f : 1.f / ml.y);
          if (ch == 0) p.lse[row0 + r] = row_lse(ml.x, ml.y);
          continue;
        }
        const uint32_t owner = i % ranks;
        const int slot = rank * share_of + i / ranks;
        st_peer_f4(om + 8 * slot, owner, s0);
        st_peer_f4(om + 8 * slot + 4, owner, s1);
        st_peer_f2(pml + slot, owner, ml);
      }
      if (ranks == 1) return;
      __syncwarp();
      cluster_barrier();  // what was sent has arrived; nobody touches a peer after it
      for (int j = tid; rank + j * ranks < pieces; j += 32 * C::WARPS) {
        const int i = rank + j * ranks, r = i / (D / 8), ch = i - r * (D / 8);
        float mt = -INFINITY, lt = 0.f;
        float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
        for (int k = 0; k < ranks; ++k) mt = fmaxf(mt, pml[k * share_of + j].x);
        for (int k = 0; k < ranks; ++k) {
          const float2 ml = pml[k * share_of + j];
          const float f = exp2_rel(ml.x, mt);
          const float* x = om + 8 * (k * share_of + j);
          const float4 u = *reinterpret_cast<const float4*>(x), v = *reinterpret_cast<const float4*>(x + 4);
          lt += ml.y * f;
          add4(s0, u, f);
          add4(s1, v, f);
        }
        store_out8<C::BF16>(p.o + (row0 + r) * D + 8 * ch, s0, s1, lt == 0.f ? 0.f : 1.f / lt);
        if (ch == 0) p.lse[row0 + r] = row_lse(mt, lt);
      }
      return;
    }
    // a common maximum, then each quarter of the columns is summed by the warps in
    // turn (warp q, q - 1, q - 2, q - 3 for quarter q)
    float f[C::NT][2];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mt = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::KW; ++k) mt = fmaxf(mt, mls[k * C::ROWS + col0 + 8 * nt + h].x);
        f[nt][h] = exp2_rel(m[nt][h], mt);
      }
    constexpr int QUARTER = (D / 16 + C::KW - 1) / C::KW;
#pragma unroll 1
    for (int round = 0; round < C::KW; ++round) {
      const int quarter = (kw + round) % C::KW;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if (i / QUARTER != quarter) continue;
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* at = om + (col0 + 8 * nt + (e & 1)) * C::OP + 16 * i + (lane >> 2) + 8 * (e >> 1);
            // nothing seen: not even 0 * inf
            const float x = m[nt][e & 1] == -INFINITY ? 0.f : acc[nt][i][e] * f[nt][e & 1];
            *at = round > 0 ? *at + x : x;
          }
      }
      sync_rows();
    }
    const bool begins = w.t0 == 0, ends = w.t1 == w.it.tiles;
    const int part_slot = 2 * part + (begins ? 1 : 0);
    for (int i = tid; i < rows * (D / 8); i += 32 * C::WARPS) {
      const int r = i / (D / 8), ch = i - r * (D / 8);
      const float4 x = *reinterpret_cast<const float4*>(om + r * C::OP + 8 * ch);
      const float4 y = *reinterpret_cast<const float4*>(om + r * C::OP + 8 * ch + 4);
      const float2 ml = warps_max_sum<C>(mls, r);
      put_piece<C>(p, begins && ends, part_slot, row0, r, ch, x, y, ml);
    }
    if (tid == 0) record_unit(p, list, share, w, part);
    sync_rows();
  }
  if constexpr (!C::CLUSTER) write_empty_units<C>(p, list, part, parts, tid, 32 * C::WARPS);
}

}  // namespace fa

#include "fa_paged_tc.cuh"

namespace fa {

// A launch of its own: in a chain of calls it takes 4.5 us, but a join by the CTA
// that is last with a part (counters in the workspace) took as long, in the fence,
// the counting and one CTA's reading of up to 40 parts (B1 131072 keys 86 us with the
// second launch, 90 without).
// Joins the parts of record blockIdx.x's unit: slot 1 of the CTA that began it and
// slot 0 of the CTAs after it. A row's parts are
// shared by up to 8 warps, four or more each with all their loads in flight, a lane
// 4 columns (D = 256: 8); with few parts the block's warps take several rows at a
// time.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 8;  // blocks per record that split units can have at least
template <int D, int ROWS, bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps)
fa_paged_join_kernel(const PagedFwdArgs p) {
  constexpr int NV = (D / 4 + 31) / 32, UN = 4;
  __shared__ float4 sm_o[kJoinWarps][D / 4];
  __shared__ float2 sm_ml[kJoinWarps];
  __shared__ int2 record;
  grid_wait_prior();
  grid_release_next();
  // read once, and within bounds whatever it holds: lengths that change under the call
  // may leave an old record, and a call that shares the workspace its own
  if (threadIdx.x == 0) record = p.joins[blockIdx.x];
  __syncthreads();
  const int2 join = record;
  const ListShape list = list_shape(p);
  if (join.x < 0 || join.x >= static_cast<int64_t>(list.items) * list.mult) return;
  const int unit = p.by_unit ? blockIdx.x : join.x;
  const int rb = unit % p.row_blocks, rows = min(ROWS, p.rows - rb * ROWS);
  const int64_t row0 = static_cast<int64_t>(unit / p.row_blocks) * p.rows + rb * ROWS;
  constexpr int LAST = paged_max_parts(ROWS) - 1;
  const int first = min(join.y & 0xffff, LAST);
  const int nparts = min(static_cast<int>(static_cast<uint32_t>(join.y) >> 16), LAST) - first + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps of a row, and this warp's place among them
  const int team = nparts <= UN ? 1 : nparts <= 2 * UN ? 2 : nparts <= 4 * UN ? 4 : 8;
  const int mate = warp % team, per_pass = kJoinWarps / team;
  for (int base = blockIdx.y * per_pass; base < rows; base += gridDim.y * per_pass) {
    const int r = base + warp / team;
    const int mine = r < rows ? nparts : 0;
    float m = -INFINITY, l = 0.f;
    float4 acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = mate; i0 < mine; i0 += team * UN) {
      float2 ml[UN];
      float4 x[UN][NV];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * team;
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) x[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= mine) continue;
        const int slot = i == 0 ? 2 * first + 1 : 2 * (first + i);
        ml[u] = p.part_ml[slot * ROWS + r];
        const float4* src = reinterpret_cast<const float4*>(p.part_o + (static_cast<int64_t>(slot) * ROWS + r) * D);
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (lane + 32 * v < D / 4) x[u][v] = src[lane + 32 * v];
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < UN; ++u) mn = fmaxf(mn, ml[u].x);
      const float alpha = exp2_rel(m, mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int v = 0; v < NV; ++v) scale4(acc[v], alpha);
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const float f = exp2_rel(ml[u].x, mn);
        l += ml[u].y * f;
#pragma unroll
        for (int v = 0; v < NV; ++v) add4(acc[v], x[u][v], f);
      }
    }
    if (team > 1) {
      __syncthreads();  // the rows of the pass before are read
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (lane + 32 * v < D / 4) sm_o[warp][lane + 32 * v] = acc[v];
      if (lane == 0) sm_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (mate > 0) continue;
      const float own = m;
      for (int k = 1; k < team; ++k) m = fmaxf(m, sm_ml[warp + k].x);
      const float f0 = exp2_rel(own, m);
      l *= f0;
#pragma unroll
      for (int v = 0; v < NV; ++v) scale4(acc[v], f0);
      for (int k = 1; k < team; ++k) {
        const float2 ml = sm_ml[warp + k];
        const float f = exp2_rel(ml.x, m);
        l += ml.y * f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (lane + 32 * v < D / 4) add4(acc[v], sm_o[warp + k][lane + 32 * v], f);
      }
    }
    if (r >= rows) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (lane + 32 * v >= D / 4) continue;
      uint2 out;
      out.x = pack2<BF16>(acc[v].x * inv, acc[v].y * inv);
      out.y = pack2<BF16>(acc[v].z * inv, acc[v].w * inv);
      *reinterpret_cast<uint2*>(p.o + (row0 + r) * D + 4 * (lane + 32 * v)) = out;
    }
    if (lane == 0) p.lse[row0 + r] = row_lse(m, l);
  }
}

// ------------------------------------------------------------------- launch
inline bool encode_maps(const PagedFwdLaunch& a, int D, CUtensorMap* mk, CUtensorMap* mv) {
  const int page = 1 << a.c.page_shift, piece = page < kPagedTile ? page : kPagedTile;
  return encode_tile_map(mk, a.c.k, a.bf16, D, page, a.c.num_pages * a.c.Hkv, piece) &&
         encode_tile_map(mv, a.c.v, a.bf16, D, page, a.c.num_pages * a.c.Hkv, piece);
}

// Clusters of `ranks` CTAs that run at once on the current device, which is less than
// its CTAs over `ranks`: a cluster stays within a GPC (a CTA per SM, 152 SMs: 36 of 4,
// 15 of 8, 7 of 16). 0 where the size is not possible. Kept per device.
template <class C>
int resident_clusters(int ranks) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][5];  // one more than the answer
  int dev = 0, slot = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  while ((1 << slot) < ranks) ++slot;
  if (dev < kDevices) {
    const int k = known[dev][slot].load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
  }
  auto kern = fa_paged_fwd_kernel<C>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = static_cast<unsigned>(ranks);
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ranks), 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess ||
      (ranks > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < kDevices) known[dev][slot].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <class C>
cudaError_t launch_paged(const PagedFwdLaunch& a, PagedFwdArgs& p, int64_t grid, int ranks) {
  CUtensorMap mk, mv;
  if (!encode_maps(a, C::D, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = fa_paged_fwd_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e == cudaSuccess && ranks > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  if (!register_split_fits(reinterpret_cast<const void*>(kern), C::THREADS, C::REG_NEEDED))
    return cudaErrorInvalidConfiguration;
  return launch_kernel(kern, grid, C::THREADS, C::SMEM_BYTES, a.stream, static_cast<unsigned>(ranks), mk, mv, p, ranks);
}
template <class C>
cudaError_t launch_paged_tc(const PagedFwdLaunch& a, PagedFwdArgs& p, int64_t grid) {
  CUtensorMap mk, mv;
  if (!encode_maps(a, C::D, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = fa_paged_tc_kernel<C>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, C::THREADS, C::SMEM_BYTES, a.stream, 1, mk, mv, p);
}

inline void set_row_blocks(const PagedFwdLaunch& a, PagedFwdArgs& p, int block) {
  p.rows = a.Hq / a.c.Hkv * a.Tq;
  p.row_blocks = (p.rows + block - 1) / block;
}

// The split list and its join, `ctas` CTAs per SM, for units of at most `tiles` tiles
// in earnest.
template <class C, class Launch>
cudaError_t run_split(const PagedFwdLaunch& a, PagedFwdArgs& p, int64_t tiles, int ctas, const Launch& launch) {
  constexpr int max_parts = paged_max_parts(C::ROWS);
  set_row_blocks(a, p, C::ROWS);
  p.part_o = a.ws;
  p.part_ml = reinterpret_cast<float2*>(a.ws + static_cast<size_t>(2 * max_parts) * C::ROWS * C::D);
  p.joins = reinterpret_cast<int2*>(p.part_ml + 2 * max_parts * C::ROWS);
  const int64_t units = static_cast<int64_t>(a.c.B) * a.c.Hkv * p.row_blocks;
  // no more CTAs than the longest possible list has tiles
  const int64_t parts = std::min(std::min<int64_t>(static_cast<int64_t>(device_sm_count()) * ctas, max_parts), units * tiles);
  p.by_unit = units <= parts;
  const cudaError_t e = launch(parts);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  // eight blocks per record, more where records are few (39 units of 35 rows: 24.7 us
  // with 8, 22.7 with 24 and above)
  const int64_t records = std::min(parts, units);
  const int64_t per_record = std::max<int64_t>(kJoinBlocks, kJoinBlocks * device_sm_count() / records);
  cfg.gridDim = dim3(static_cast<unsigned>(records),
                     static_cast<unsigned>(std::min<int64_t>(std::min(p.rows, C::ROWS), per_record)), 1);
  cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
  cfg.stream = a.stream;
  allow_early_launch(&cfg, attrs);
  return cudaLaunchKernelEx(&cfg, fa_paged_join_kernel<C::D, C::ROWS, C::BF16>, p);
}

template <int D, int RG, bool BF16>
cudaError_t run_split_tc(const PagedFwdLaunch& a, PagedFwdArgs& p, int64_t tiles) {
  using C = PagedTcCfg<D, RG, BF16>;
  return run_split<C>(a, p, tiles, 1, [&](int64_t parts) { return launch_paged_tc<C>(a, p, parts); });
}

template <int D, int NT, int RW, bool BF16>
cudaError_t run_paged(const PagedFwdLaunch& a) {
  using C = PagedCfg<D, NT, RW, BF16, true>;
  PagedFwdArgs p = {};
  p.c = a.c;
  p.q = a.q; p.o = a.o; p.lse = a.lse;
  p.Hq = a.Hq; p.Tq = a.Tq; p.causal = a.causal;
  p.window = std::min(a.window, 1 << 30);  // positions end below 2^30: a longer window hides nothing either
  p.scale_log2 = a.scale_log2;
  p.new_lens = a.new_lens;
  p.sel = a.sel; p.sel_lens = a.sel_lens; p.n_sel = a.n_sel;
  p.wc = a.wc;
  set_row_blocks(a, p, C::ROWS);
  // tiles of the longest list a unit can have in earnest (of distinct pages; the
  // kernels take any)
  const int64_t keys = static_cast<int64_t>(a.sel ? std::min(a.n_sel, a.c.max_pages) : a.c.max_pages) << a.c.page_shift;
  int64_t tiles = paged_tiles(1, keys);
  if (a.window > 0 && !a.sel)  // window + Tq - 1 keys, wherever they start in a tile
    tiles = std::min(tiles, (static_cast<int64_t>(a.window) + a.Tq - 2) / kPagedTile + 2);
  const int64_t units = static_cast<int64_t>(a.c.B) * a.c.Hkv * p.row_blocks;
  // Short units: a cluster each, joined in the same launch, where all clusters run at
  // once or one CTA does for a unit. Measured: 16 tiles, 4 units 4.6 us against 12.0
  // with the split list and its join; 64 tiles, 8 units 7.1 us with 16 CTAs, 8.0 with
  // 8 and 11.2 split.
  int ranks = 1;
  while (tiles > 2 && ranks < kPagedMaxRanks && ranks < tiles) ranks *= 2;  // 2 tiles: 5.7 us in one CTA, 6.6 in two
  while (ranks > 1 && units > resident_clusters<C>(ranks)) ranks /= 2;
  if (tiles <= C::CLUSTER_TILES * ranks) return launch_paged<C>(a, p, units * ranks, ranks);
  if constexpr (RW > 1) {  // more than 16 rows
    switch (paged_split_rows(p.rows)) {
      case 32: return run_split_tc<D, 1, BF16>(a, p, tiles);
      case 64: return run_split_tc<D, 2, BF16>(a, p, tiles);
      default: return run_split_tc<D, 4, BF16>(a, p, tiles);
    }
  } else {
    using S = PagedCfg<D, NT, RW, BF16, false>;
    return run_split<S>(a, p, tiles, S::CTAS, [&](int64_t parts) { return launch_paged<S>(a, p, parts, 1); });
  }
}

template <int D, bool BF16>
cudaError_t run_paged_rows(const PagedFwdLaunch& a) {
  switch (paged_block_rows(a.Hq / a.c.Hkv * a.Tq, D)) {
    case 8: return run_paged<D, 1, 1, BF16>(a);
    case 16: return run_paged<D, 2, 1, BF16>(a);
    case 32: return run_paged<D, 2, 2, BF16>(a);
    case 48:
      if constexpr (D < 256) return run_paged<D, 3, 2, BF16>(a);
      break;
    default:
      if constexpr (D < 256) return run_paged<D, 4, 2, BF16>(a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa

#define FA_DEFINE_PAGED_HEAD_DIM(DIM)                                      \
  namespace fa {                                                           \
  cudaError_t launch_paged_fwd_d##DIM(const PagedFwdLaunch& a) {           \
    return a.bf16 ? run_paged_rows<DIM, true>(a) : run_paged_rows<DIM, false>(a); \
  }                                                                        \
  }
