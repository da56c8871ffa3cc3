// Appending new tokens to the paged cache: keys are rotated by their position,
// values copied, the tokens' queries rotated, and the element-wise bounds of
// the keys' pages kept.
//
//   (y_i, y_i') = (x_i cos - x_i' sin, x_i' cos + x_i sin)   per pair (i, i')
//
// in fp32, rounded once to the cache's type (what the page holds is what
// attention reads, so the bounds are taken of the rounded values).
//
// The work is one read and one write of every row. A thread owns units of 16
// elements that close over their rotation pairs (two 16-byte chunks, rot / 2
// apart or adjacent), so a row is D / 16 lanes, and the bounds of a page are
// packed minima and maxima in registers.
//   few new tokens: one unit per thread, so that a single token's latency is two
//     dependent loads and a store (with bounds a thread walks the tokens of its
//     unit of a KV head);
//   many: a warp takes a few consecutive tokens of 4 heads, or with bounds new keys
//     of one page and KV head, with four rows' loads in flight per thread.
// Measured: one token of one sequence 1.4 us, of 96 with bounds 2.2 us (a chain of
// calls; the launch itself); B4 T4096 Hq32 Hkv8 D128 bf16 with bounds, 406 MB, 62.6
// to 63.2 us = 6.4 to 6.5 TB/s, 95% of the copy rate (the 74 bytes that the key path
// spills under three blocks per SM included). That case with (rows, keys in flight, blocks
// per SM): 4/4/3 63.0 us, 4/4/4 73.2, 2/2/4 64.6, 8/4/2 65.0, 2/2/6 90.8.
#include <type_traits>

#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {
namespace {

struct AppendArgs {
  PagedView c;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  TokenStrides ks, vs, qs;
  int Hq, T;
  const int* new_lens;
  const float *cos_table, *sin_table;
  int rope_len, rot_dim, interleaved;
};

constexpr int kAppendThreads = 256;

// The two 16-byte chunks of unit u of a row: element offsets.
struct UnitPos {
  int a, b;
  bool rotated;
};
__device__ __forceinline__ UnitPos unit_pos(const AppendArgs& p, int u) {
  UnitPos r;
  r.rotated = 16 * u < p.rot_dim;
  const bool halves = r.rotated && !p.interleaved;
  r.a = halves ? 8 * u : 16 * u;
  r.b = halves ? 8 * u + p.rot_dim / 2 : 16 * u + 8;
  return r;
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles load_angles(const AppendArgs& p, int pos, int u) {
  Angles g;
  const int64_t at = static_cast<int64_t>(pos) * (p.rot_dim / 2) + 8 * u;
  const float4* c = reinterpret_cast<const float4*>(p.cos_table + at);
  const float4* s = reinterpret_cast<const float4*>(p.sin_table + at);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 x = c[i], y = s[i];
    g.c[4 * i] = x.x; g.c[4 * i + 1] = x.y; g.c[4 * i + 2] = x.z; g.c[4 * i + 3] = x.w;
    g.s[4 * i] = y.x; g.s[4 * i + 1] = y.y; g.s[4 * i + 2] = y.z; g.s[4 * i + 3] = y.w;
  }
  return g;
}

// Rotate a unit in place (fp32 arithmetic, one rounding per value).
template <bool BF16>
__device__ __forceinline__ void rotate_unit(uint4& a, uint4& b, const Angles& g, bool interleaved) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF16>(wa[i]), y = unpack2<BF16>(wb[i]);
    if (interleaved) {  // pairs (x.x, x.y) and (y.x, y.y)
      wa[i] = pack2<BF16>(x.x * g.c[i] - x.y * g.s[i], x.y * g.c[i] + x.x * g.s[i]);
      wb[i] = pack2<BF16>(y.x * g.c[4 + i] - y.y * g.s[4 + i], y.y * g.c[4 + i] + y.x * g.s[4 + i]);
    } else {  // pairs (x.x, y.x) and (x.y, y.y)
      const float c0 = g.c[2 * i], c1 = g.c[2 * i + 1], s0 = g.s[2 * i], s1 = g.s[2 * i + 1];
      wa[i] = pack2<BF16>(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
      wb[i] = pack2<BF16>(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
  using T2 = std::conditional_t<BF16, __nv_bfloat162, __half2>;
  T2 r = __hmin2(*reinterpret_cast<T2*>(&x), *reinterpret_cast<T2*>(&y));
  return *reinterpret_cast<uint32_t*>(&r);
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  using T2 = std::conditional_t<BF16, __nv_bfloat162, __half2>;
  T2 r = __hmax2(*reinterpret_cast<T2*>(&x), *reinterpret_cast<T2*>(&y));
  return *reinterpret_cast<uint32_t*>(&r);
}

struct Unit {
  uint4 a, b;
};
__device__ __forceinline__ Unit load_unit(const uint16_t* src, const UnitPos& at) {
  return {*reinterpret_cast<const uint4*>(src + at.a), *reinterpret_cast<const uint4*>(src + at.b)};
}
__device__ __forceinline__ void shuffle_unit(const Unit& x, int lane, Unit* y) {
  const uint32_t* s = reinterpret_cast<const uint32_t*>(&x);
  uint32_t* d = reinterpret_cast<uint32_t*>(y);
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = __shfl_sync(0xffffffffu, s[i], lane);
}
__device__ __forceinline__ void store_unit(uint16_t* dst, const UnitPos& at, const Unit& x) {
  *reinterpret_cast<uint4*>(dst + at.a) = x.a;
  *reinterpret_cast<uint4*>(dst + at.b) = x.b;
}

// Packed element-wise minima and maxima of a unit.
template <bool BF16>
struct UnitBounds {
  Unit mn, mx;
  __device__ __forceinline__ void start(const Unit& x) { mn = mx = x; }
  __device__ __forceinline__ void widen(const Unit& lo, const Unit& hi) {
    const uint32_t* l = reinterpret_cast<const uint32_t*>(&lo);
    const uint32_t* h = reinterpret_cast<const uint32_t*>(&hi);
    uint32_t* m = reinterpret_cast<uint32_t*>(&mn);
    uint32_t* x = reinterpret_cast<uint32_t*>(&mx);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = min2<BF16>(m[i], l[i]);
      x[i] = max2<BF16>(x[i], h[i]);
    }
  }
};

__device__ __forceinline__ uint16_t* bounds_row(const PagedView& c, int id, int g) {
  return c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * c.D;
}

// The new tokens of a sequence that have a place: [t0, t1) of its rows, token t at
// position first + t.
struct NewTokens {
  int first, t0, t1;
};
__device__ __forceinline__ NewTokens new_tokens(const AppendArgs& p, int b) {
  const SeqLens sl = seq_lens(p.c, p.new_lens, b, p.T);
  NewTokens r;
  r.first = sl.len - sl.n;
  r.t0 = max(0, -r.first);
  r.t1 = p.rot_dim > 0 ? min(sl.n, p.rope_len - r.first) : sl.n;
  if (r.t0 > 0 || r.t1 < sl.n) flag_bad_index(p.c);
  return r;
}

// One value, query or (without bounds) key row's unit: token t, row `row` of the
// token: values, then queries, then keys.
template <bool BF16>
__device__ __forceinline__ void append_row(const AppendArgs& p, const NewTokens& nt, int b, int t, int row, int u,
                                           const UnitPos& at, const Angles& g) {
  const PagedView& c = p.c;
  const int hq = p.Hq;  // 0 without queries
  const bool there = t >= nt.t0 && t < nt.t1;
  if (row >= c.Hkv && row < c.Hkv + hq) {
    const int h = row - c.Hkv;
    Unit x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (there) {
      x = load_unit(p.q + b * p.qs.b + h * p.qs.h + t * p.qs.t, at);
      if (at.rotated) rotate_unit<BF16>(x.a, x.b, g, p.interleaved);
    }
    store_unit(p.q_out + ((static_cast<int64_t>(b) * p.Hq + h) * p.T + t) * c.D, at, x);
    return;
  }
  if (!there) return;
  const int pos = nt.first + t;
  const int id = pool_page(c, b, pos >> c.page_shift);
  if (id < 0) return;
  const int slot = pos & ((1 << c.page_shift) - 1);
  if (row < c.Hkv) {
    store_unit(c.v + pool_row(c, id, row, slot), at, load_unit(p.v + b * p.vs.b + row * p.vs.h + t * p.vs.t, at));
  } else {
    const int gk = row - c.Hkv - hq;
    Unit x = load_unit(p.k + b * p.ks.b + gk * p.ks.h + t * p.ks.t, at);
    if (at.rotated) rotate_unit<BF16>(x.a, x.b, g, p.interleaved);
    store_unit(c.k + pool_row(c, id, gk, slot), at, x);
  }
}

// Few tokens. Grid: x = sequence, y = blocks of kAppendThreads units of all rows
// of the sequence's T tokens (keys with bounds: of its KV heads).
template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads)
fa_kv_append_kernel(const AppendArgs p) {
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int units = c.D / 16;
  const int b = blockIdx.x;
  const int item = blockIdx.y * kAppendThreads + threadIdx.x;
  const int r = item / units, u = item - r * units;
  const bool bounds = c.bounds != nullptr;
  const int heads = c.Hkv + p.Hq + (bounds ? 0 : c.Hkv);  // rows of a token without its bounded keys
  const UnitPos at = unit_pos(p, u);
  if (r < p.T * heads) {
    const int t = r / heads;
    const NewTokens nt = new_tokens(p, b);
    Angles g = {};
    if (at.rotated && r - t * heads >= c.Hkv && t >= nt.t0 && t < nt.t1) g = load_angles(p, nt.first + t, u);
    append_row<BF16>(p, nt, b, t, r - t * heads, u, at, g);
    return;
  }
  const int gk = r - p.T * heads;
  if (!bounds || gk >= c.Hkv) return;
  const NewTokens nt = new_tokens(p, b);
  const int page_mask = (1 << c.page_shift) - 1;
  for (int t = nt.t0; t < nt.t1;) {  // a page at a time
    const int pos = nt.first + t;
    const int stop = min(nt.t1, t + page_mask + 1 - (pos & page_mask));
    const int id = pool_page(c, b, pos >> c.page_shift);
    if (id >= 0) {
      uint16_t* br = bounds_row(c, id, gk);
      const bool fresh = (pos & page_mask) == 0;
      Unit old_mn = {}, old_mx = {};
      if (!fresh) {
        old_mn = {*reinterpret_cast<const uint4*>(br + at.a), *reinterpret_cast<const uint4*>(br + at.b)};
        old_mx = {*reinterpret_cast<const uint4*>(br + c.D + at.a), *reinterpret_cast<const uint4*>(br + c.D + at.b)};
      }
      UnitBounds<BF16> bd;
      for (int s = t; s < stop; ++s) {
        Unit x = load_unit(p.k + b * p.ks.b + gk * p.ks.h + s * p.ks.t, at);
        if (at.rotated) rotate_unit<BF16>(x.a, x.b, load_angles(p, nt.first + s, u), p.interleaved);
        store_unit(c.k + pool_row(c, id, gk, (nt.first + s) & page_mask), at, x);
        if (s == t)
          bd.start(x);
        else
          bd.widen(x, x);
      }
      if (!fresh) bd.widen(old_mn, old_mx);
      store_unit(br, at, bd.mn);
      store_unit(br + c.D, at, bd.mx);
    }
    t = stop;
  }
}

// Many tokens. Blocks in order of work: first, with bounds, new keys by (sequence,
// page, KV head), shared by one to eight warps; then, a warp each, (sequence, group of consecutive tokens, rows of a few heads).
constexpr int kRowBatch = 4;  // rows of a thread, all loads in flight
constexpr int kKeyBatch = 4;  // keys of a page likewise
constexpr int kManyBlocks = 3;  // blocks per SM that registers are to allow
constexpr int kAppendWarps = kAppendThreads / 32;
template <int D, bool BF16>
__global__ void __launch_bounds__(kAppendThreads, kManyBlocks)
fa_kv_append_many_kernel(const AppendArgs p, int pages_per_seq, int key_blocks, int key_warps, int groups_per_seq,
                         int row_chunks, int64_t row_items) {
  constexpr int U = D / 16, TL = 32 / U;  // lanes of a row, rows side by side
  __shared__ UnitBounds<BF16> sums[kAppendWarps][U];
  __shared__ int filled[kAppendWarps];
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % U, tl = lane / U;
  const UnitPos at = unit_pos(p, u);
  if (blockIdx.x < key_blocks) {
    // key_warps warps share an item, each the rows share * TL + tl, then key_warps * TL on
    const int share = warp % key_warps;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kAppendWarps / key_warps) + warp / key_warps;
    const int g = static_cast<int>(item % c.Hkv);
    const int bp = static_cast<int>(item / c.Hkv);
    const int b = bp / pages_per_seq;
    UnitBounds<BF16> bd;
    int id = -1, lo = 0;
    bool any = false;
    if (b < c.B) {
      const NewTokens nt = new_tokens(p, b);
      const int first = nt.first + nt.t0;  // first position written
      const int page = (first >> c.page_shift) + (bp - b * pages_per_seq);
      const int base = page << c.page_shift;
      lo = max(first - base, 0);
      const int hi = min(nt.first + nt.t1 - base, 1 << c.page_shift);
      if (lo < hi && nt.t0 < nt.t1) id = pool_page(c, b, page);
      if (id >= 0 && tl < TL) {
        const uint16_t* src = p.k + b * p.ks.b + g * p.ks.h + static_cast<int64_t>(base - nt.first) * p.ks.t;
        uint16_t* dst = c.k + pool_row(c, id, g, 0);
        const int step = key_warps * TL;
        for (int s0 = lo + share * TL + tl; s0 < hi; s0 += kKeyBatch * step) {
          Unit x[kKeyBatch];
#pragma unroll
          for (int i = 0; i < kKeyBatch; ++i)
            if (s0 + i * step < hi) x[i] = load_unit(src + (s0 + i * step) * p.ks.t, at);
#pragma unroll
          for (int i = 0; i < kKeyBatch; ++i) {
            const int s = s0 + i * step;
            if (s >= hi) break;
            if (at.rotated) rotate_unit<BF16>(x[i].a, x[i].b, load_angles(p, base + s, u), p.interleaved);
            store_unit(dst + s * D, at, x[i]);
            if (!any)
              bd.start(x[i]);
            else
              bd.widen(x[i], x[i]);
            any = true;
          }
        }
      }
    }
    // join the rows side by side (lanes without a key take lane u's, which has one
    // if any of its warp's has), then the item's warps
    Unit mn0, mx0;
    shuffle_unit(bd.mn, u, &mn0);
    shuffle_unit(bd.mx, u, &mx0);
    const bool warp_any = __any_sync(0xffffffffu, any);
    if (!any) {
      bd.mn = mn0;
      bd.mx = mx0;
    }
#pragma unroll
    for (int k = 1; k < TL; ++k) {
      Unit m, x;
      shuffle_unit(bd.mn, (u + k * U) & 31, &m);
      shuffle_unit(bd.mx, (u + k * U) & 31, &x);
      if (tl == 0) bd.widen(m, x);
    }
    if (tl == 0) sums[warp][u] = bd;
    if (lane == 0) filled[warp] = warp_any;
    __syncthreads();
    if (share == 0 && tl == 0 && id >= 0) {  // the item's first warp has its first key
      for (int k = 1; k < key_warps; ++k)
        if (filled[warp + k]) bd.widen(sums[warp + k][u].mn, sums[warp + k][u].mx);
      uint16_t* br = bounds_row(c, id, g);
      if (lo > 0) {
        const Unit om = {*reinterpret_cast<const uint4*>(br + at.a), *reinterpret_cast<const uint4*>(br + at.b)};
        const Unit ox = {*reinterpret_cast<const uint4*>(br + D + at.a), *reinterpret_cast<const uint4*>(br + D + at.b)};
        bd.widen(om, ox);
      }
      store_unit(br, at, bd.mn);
      store_unit(br + D, at, bd.mx);
    }
    return;
  }
  const int64_t r = static_cast<int64_t>(blockIdx.x - key_blocks) * kAppendWarps + warp;
  if (r >= row_items) return;
  int chunk = static_cast<int>(r % row_chunks);
  const int bg = static_cast<int>(r / row_chunks);
  const int b = bg / groups_per_seq;
  const int t = (bg - b * groups_per_seq) * TL + tl;
  if (tl >= TL || t >= p.T) return;
  const NewTokens nt = new_tokens(p, b);
  const bool there = t >= nt.t0 && t < nt.t1;
  const int pos = nt.first + t;
  // chunks of value rows, of query rows, of key rows
  const int v_chunks = (c.Hkv + kRowBatch - 1) / kRowBatch, q_chunks = (p.Hq + kRowBatch - 1) / kRowBatch;
  const bool is_v = chunk < v_chunks, is_q = !is_v && chunk < v_chunks + q_chunks;
  chunk -= is_v ? 0 : is_q ? v_chunks : v_chunks + q_chunks;
  const TokenStrides& st = is_v ? p.vs : is_q ? p.qs : p.ks;
  const int h0 = chunk * kRowBatch, count = min(kRowBatch, (is_q ? p.Hq : c.Hkv) - h0);
  const uint16_t* src = (is_v ? p.v : is_q ? p.q : p.k) + b * st.b + h0 * st.h + t * st.t;
  uint16_t* dst;
  int64_t step;  // from head to head
  if (is_q) {
    dst = p.q_out + ((static_cast<int64_t>(b) * p.Hq + h0) * p.T + t) * D;
    step = static_cast<int64_t>(p.T) * D;
  } else {
    if (!there) return;
    const int id = pool_page(c, b, pos >> c.page_shift);
    if (id < 0) return;
    dst = (is_v ? c.v : c.k) + pool_row(c, id, h0, pos & ((1 << c.page_shift) - 1));
    step = static_cast<int64_t>(D) << c.page_shift;
  }
  Unit x[kRowBatch];
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    x[i] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (there && i < count) x[i] = load_unit(src + i * st.h, at);
  }
  if (there && at.rotated && !is_v) {
    const Angles g = load_angles(p, pos, u);
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) rotate_unit<BF16>(x[i].a, x[i].b, g, p.interleaved);
  }
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i)
    if (i < count) store_unit(dst + i * step, at, x[i]);
}

// Up to this many new tokens per sequence, one unit per thread.
constexpr int kFewTokens = 8;

template <int D, bool BF16>
cudaError_t run_append_many(const AppendLaunch& a, const AppendArgs& p) {
  constexpr int TL = 32 / (D / 16);
  const bool bounds = a.c.bounds != nullptr;
  const int page = 1 << a.c.page_shift;
  const int pages = (a.T + page - 2) / page + 1;  // that T tokens can touch
  const int64_t key_items = bounds ? static_cast<int64_t>(a.c.B) * pages * a.c.Hkv : 0;
  // Few pages: more warps each, down to 16 keys (B2 T413, 128 keys a page: 19.3 us
  // with one, 5.3 with eight); one warp each where that fills the GPU (B4 T4096, 64
  // keys a page: 63.0 us with one, 68.2 with four).
  int key_warps = 1;
  while (key_warps < kAppendWarps && 16 * key_warps < page && key_items * key_warps < 8 * device_sm_count()) key_warps *= 2;
  const int64_t key_blocks = (key_items * key_warps + kAppendWarps - 1) / kAppendWarps;
  const int groups = (a.T + TL - 1) / TL;
  const int kv_chunks = (a.c.Hkv + kRowBatch - 1) / kRowBatch;
  const int chunks = (bounds ? 1 : 2) * kv_chunks + (p.Hq + kRowBatch - 1) / kRowBatch;
  const int64_t row_items = static_cast<int64_t>(a.c.B) * groups * chunks;
  const int64_t blocks = key_blocks + (row_items + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_kernel(fa_kv_append_many_kernel<D, BF16>, blocks, kAppendThreads, 0, a.stream, 1, p, pages,
                       static_cast<int>(key_blocks), key_warps, groups, chunks, row_items);
}

template <bool BF16>
cudaError_t run_append(const AppendLaunch& a) {
  AppendArgs p;
  p.c = a.c;
  p.k = a.k; p.v = a.v; p.q = a.q;
  p.q_out = a.q_out;
  p.ks = a.ks; p.vs = a.vs; p.qs = a.qs;
  p.Hq = a.q != nullptr ? a.Hq : 0;
  p.T = a.T;
  p.new_lens = a.new_lens;
  p.cos_table = a.cos_table; p.sin_table = a.sin_table;
  p.rope_len = a.rope_len; p.rot_dim = a.rot_dim; p.interleaved = a.interleaved;
  if (a.T > kFewTokens) {
    switch (a.c.D) {
      case 64: return run_append_many<64, BF16>(a, p);
      case 96: return run_append_many<96, BF16>(a, p);
      case 128: return run_append_many<128, BF16>(a, p);
      default: return run_append_many<256, BF16>(a, p);
    }
  }
  const bool bounds = a.c.bounds != nullptr;
  const int rows = a.T * (a.c.Hkv + p.Hq + (bounds ? 0 : a.c.Hkv)) + (bounds ? a.c.Hkv : 0);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.gridDim = dim3(static_cast<unsigned>(a.c.B),
                     static_cast<unsigned>((rows * (a.c.D / 16) + kAppendThreads - 1) / kAppendThreads), 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = a.stream;
  allow_early_launch(&cfg, attrs);
  return cudaLaunchKernelEx(&cfg, fa_kv_append_kernel<BF16>, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendLaunch& a) {
  return a.bf16 ? run_append<true>(a) : run_append<false>(a);
}

}  // namespace fa
