// Appending new tokens to a cache held in 8 bits: keys rotated by their position, keys and
// values of a page and KV head brought to a common scale and rounded to e4m3, the tokens'
// queries rotated.
//
//   s = min { 2^e : |x| <= 448 2^e for the page's new x },  at least the page's old s
//   held = round(x / s)
//
// Why a power of two: e4m3 is floating point, so a scale moves its range and buys no
// precision; and when a later token raises the scale of a page that is partly filled, the
// older rows keep their values exactly, but for what falls below 2^-6 s (the smallest
// normal number). With any other factor every such step would round all of them again.
// One scale per page and head: 18 binades of range are more than a page's rows need, and
// attention then has one factor for the 16 keys that a warp takes of a tile. The rotated
// key is rounded once, from fp32 to 8 bits.
//
// The work is one read (16 bits) and one write (8 bits) of every row. Keys and values are
// items of a page and KV head each, whose rows are read, their largest magnitude agreed
// on, and written:
//   few new tokens: a warp per item, its lanes some rows side by side; a row of a page from
//     before is read again only where the scale rises;
//   many: one to eight warps per item with two rows of a thread in registers, as they
//     come (so that loads are under way while others wait at the item's barrier), so that
//     rows are read once where a page has no more (64 x 128 elements, 256 threads: 2);
//     longer pages are read twice, the second time from L2. Query rows have blocks of
//     their own, in turn with the items': they keep the memory busy meanwhile.
//
// Measured (bf16, Hq32 Hkv8 D128): one token 3.2 us, CPU time of the call; 4 x 4096 tokens
// into pages of 64 67.7 us, 81% of the copy rate for their 371 MB. Three blocks per SM with
// 80 registers: 21 warps of 64 active, a warp waits 3.6 of its 10 cycles per instruction for
// loads; four blocks spill 140 bytes a thread.
#include <climits>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_append.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// The scale of rows whose largest magnitude is `most` (448 = 1.75 2^8), and its inverse:
// 2^-126 to 2^120, so that both are normal numbers.
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t b = __float_as_uint(most);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}
__device__ __forceinline__ float inverse_scale(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// The larger of m and |x|; a NaN counts as nothing. FINITE: an infinity neither. (It is
// looked for in a second pass, where the first one finds it.)
template <bool FINITE>
__device__ __forceinline__ float widen_max(float m, float x) {
  const float a = fabsf(x);
  return !FINITE || a < INFINITY ? fmaxf(m, a) : m;
}

__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
__device__ __forceinline__ void unpack4_e4m3(uint32_t x, float* y) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(x >> (16 * i))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
}

// A unit's 16 values in fp32, chunk a's eight before chunk b's.
struct Values {
  float x[16];
};
template <bool BF16>
__device__ __forceinline__ Values unit_values(const Unit& u) {
  Values v;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    v.x[2 * i] = f.x;
    v.x[2 * i + 1] = f.y;
  }
  return v;
}
__device__ __forceinline__ void rotate_values(Values& v, const Angles& g, bool interleaved) {
  auto turn = [&](float& a, float& b, int i) {
    const float x = a, y = b;
    a = x * g.c[i] - y * g.s[i];
    b = y * g.c[i] + x * g.s[i];
  };
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(v.x[2 * i], v.x[2 * i + 1], i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(v.x[i], v.x[i + 8], i);
  }
}
// Rounded and stored (a finite value is at most 448 s). `odd`: some are infinite, and are
// to become NaN.
__device__ __forceinline__ void store_values(uint8_t* dst, const UnitPos& at, const Values& v, float inv, bool odd) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = v.x[4 * i + e] * inv;
    if (odd) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fabsf(y[e]) <= 448.f ? y[e] : NAN;
    }
    w[i] = pack4_e4m3(y[0], y[1], y[2], y[3]);
  }
  if (at.b == at.a + 8) {
    *reinterpret_cast<uint4*>(dst + at.a) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(dst + at.a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(dst + at.b) = make_uint2(w[2], w[3]);
  }
}

// Row chunks [first, n) of 16 held values, every step-th, times `f` = old scale / new one.
__device__ __forceinline__ void rescale_chunks(uint8_t* rows, int first, int n, int step, float f) {
  for (int i0 = first; i0 < n; i0 += 4 * step) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * step < n) x[k] = reinterpret_cast<const uint4*>(rows)[i0 + k * step];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k * step >= n) break;
      uint32_t* w = reinterpret_cast<uint32_t*>(&x[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y[4];
        unpack4_e4m3(w[e], y);
        w[e] = pack4_e4m3(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
      }
      reinterpret_cast<uint4*>(rows)[i0 + k * step] = x[k];
    }
  }
}

// Keys (or values) of one KV head: where its new rows come from and go to.
struct Source {
  const uint16_t* src;  // of sequence b and head g
  int64_t step;         // from token to token
  uint8_t* pool;
  float* scales;
  bool turn;            // rotate
};
__device__ __forceinline__ Source source_of(const AppendArgs& p, int b, int g, bool values, const UnitPos& at) {
  if (values)
    return {p.v + b * p.vs.b + g * p.vs.h, p.vs.t, reinterpret_cast<uint8_t*>(p.c.v), p.c.v_scales, false};
  return {p.k + b * p.ks.b + g * p.ks.h, p.ks.t, reinterpret_cast<uint8_t*>(p.c.k), p.c.k_scales, at.rotated};
}
// Values are units of adjacent chunks: their rotation pairs do not matter.
__device__ __forceinline__ UnitPos item_unit(const AppendArgs& p, int u, bool values) {
  return values ? UnitPos{16 * u, 16 * u + 8, false} : unit_pos(p, u);
}
template <bool BF16>
__device__ __forceinline__ Values load_values(const AppendArgs& p, const Source& s, const UnitPos& at, int t, int pos, int u) {
  Values v = unit_values<BF16>(load_unit(s.src + t * s.step, at));
  if (s.turn) rotate_values(v, load_angles(p, pos, u), p.interleaved);
  return v;
}

template <bool BF16>
__device__ __forceinline__ void append_query(const AppendArgs& p, const NewTokens& nt, int b, int t, int h, int u,
                                             const UnitPos& at) {
  Unit x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (t >= nt.t0 && t < nt.t1) {
    x = load_unit(p.q + b * p.qs.b + h * p.qs.h + t * p.qs.t, at);
    if (at.rotated) rotate_unit<BF16>(x.a, x.b, load_angles(p, nt.first + t, u), p.interleaved);
  }
  store_unit(p.q_out + ((static_cast<int64_t>(b) * p.Hq + h) * p.T + t) * p.c.D, at, x);
}

// Few tokens. Grid: x = sequence, y = blocks of warps: 2 Hkv of keys and values, a head
// each, then units of the query rows, one per thread.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
fa_kv_append8_kernel(const AppendArgs p) {
  constexpr int U = D / 16, TL = 32 / U;  // lanes of a row, rows side by side
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int w = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (w >= 2 * c.Hkv) {
    const int i = (w - 2 * c.Hkv) * 32 + lane, r = i / U, u = i - r * U;
    if (r >= p.T * p.Hq) return;
    append_query<BF16>(p, new_tokens(p, b), b, r / p.Hq, r % p.Hq, u, unit_pos(p, u));
    return;
  }
  const bool values = w < c.Hkv;
  const int g = values ? w : w - c.Hkv, u = lane % U, tl = lane / U;
  const UnitPos at = item_unit(p, u, values);
  const Source src = source_of(p, b, g, values, at);
  const NewTokens nt = new_tokens(p, b);
  const int page_mask = (1 << c.page_shift) - 1;
  for (int t = nt.t0; t < nt.t1;) {  // a page at a time
    const int pos = nt.first + t, slot = pos & page_mask;
    const int stop = min(nt.t1, t + page_mask + 1 - slot);
    // the first rows of the lanes while the page is looked up
    Values v;
    const int mine = t + tl;
    const bool one = tl < TL && mine < stop;
    if (one) v = load_values<BF16>(p, src, at, mine, nt.first + mine, u);
    const int id = pool_page(c, b, pos >> c.page_shift);
    if (id >= 0) {
      float* scale = src.scales + static_cast<int64_t>(id) * c.Hkv + g;
      const float old = __shfl_sync(0xffffffffu, slot > 0 && lane == 0 ? *scale : 0.f, 0);
      auto largest = [&](auto finite) {
        float most = 0.f;
        if (one) {
#pragma unroll
          for (int e = 0; e < 16; ++e) most = widen_max<finite.value>(most, v.x[e]);
        }
        for (int s = mine + TL; tl < TL && s < stop; s += TL) {
          const Values x = load_values<BF16>(p, src, at, s, nt.first + s, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) most = widen_max<finite.value>(most, x.x[e]);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
        return most;
      };
      float most = largest(std::false_type());
      const bool odd = most == INFINITY;
      if (odd) most = largest(std::true_type());
      const float s0 = scale_for(most), sc = slot > 0 ? fmaxf(s0, old) : s0, inv = inverse_scale(sc);
      uint8_t* rows = src.pool + pool_row(c, id, g, 0);
      if (one) store_values(rows + static_cast<int64_t>(slot + tl) * D, at, v, inv, odd);
      for (int s = mine + TL; tl < TL && s < stop; s += TL)
        store_values(rows + static_cast<int64_t>(slot + s - t) * D, at, load_values<BF16>(p, src, at, s, nt.first + s, u), inv,
                     odd);
      if (slot > 0 && s0 > old) rescale_chunks(rows, lane, slot * U, 32, old * inv);
      if (lane == 0 && !(slot > 0 && sc == old)) *scale = sc;
    }
    t = stop;
  }
}

// A warp's query rows `r`: of a sequence, group of consecutive tokens and a few heads.
constexpr int kRowBatch = 4;  // rows of a thread, all loads in flight
template <int D, bool BF16>
__device__ __forceinline__ void append_queries(const AppendArgs& p, uint32_t r, uint32_t groups_per_seq, uint32_t row_chunks,
                                               uint32_t row_items) {
  constexpr int U = D / 16, TL = 32 / U;
  const int lane = threadIdx.x & 31, u = lane % U, tl = lane / U;
  if (r >= row_items) return;
  const uint32_t bg = r / row_chunks, seq = bg / groups_per_seq;
  const int chunk = r - bg * row_chunks, b = seq, t = (bg - seq * groups_per_seq) * TL + tl;
  if (tl >= TL || t >= p.T) return;
  const UnitPos at = unit_pos(p, u);
  const NewTokens nt = new_tokens(p, b);
  const bool there = t >= nt.t0 && t < nt.t1;
  const int h0 = chunk * kRowBatch, count = min(kRowBatch, p.Hq - h0);
  const uint16_t* q = p.q + b * p.qs.b + h0 * p.qs.h + t * p.qs.t;
  uint16_t* dst = p.q_out + ((static_cast<int64_t>(b) * p.Hq + h0) * p.T + t) * D;
  Unit x[kRowBatch];
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i) {
    x[i] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (there && i < count) x[i] = load_unit(q + i * p.qs.h, at);
  }
  if (there && at.rotated) {
    const Angles g = load_angles(p, nt.first + t, u);
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) rotate_unit<BF16>(x[i].a, x[i].b, g, p.interleaved);
  }
#pragma unroll
  for (int i = 0; i < kRowBatch; ++i)
    if (i < count) store_unit(dst + static_cast<int64_t>(i) * p.T * D, at, x[i]);
}

// Many tokens. Keys and values by (sequence, page, KV head, which), `warps` of a block each;
// query rows of (sequence, group of consecutive tokens, a few heads), a warp each. Blocks of
// the two kinds take turns evenly over the grid: items are chains of dependent loads and a
// barrier, rows keep the memory busy meanwhile.
constexpr int kRows = 2;      // rows of a thread in registers
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 3)
fa_kv_append8_many_kernel(const AppendArgs p, uint32_t pages_per_seq, uint64_t items_per_block, int warps_log2,
                          uint32_t groups_per_seq, uint32_t row_chunks, uint32_t row_items) {
  constexpr int U = D / 16, TL = 32 / U;
  __shared__ float tops[2][kWarps];
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = lane % U, tl = lane / U;
  // blocks of items before this one (items_per_block: of 2^32; divisions of 64 bits would
  // take longer than an item's rows)
  const uint32_t items_before = static_cast<uint32_t>(blockIdx.x * items_per_block >> 32);
  if (static_cast<uint32_t>((blockIdx.x + 1) * items_per_block >> 32) > items_before) {
    const int warps = 1 << warps_log2, share = warp & (warps - 1);
    const uint32_t item = items_before * (kWarps >> warps_log2) + (warp >> warps_log2);
    const uint32_t bp = item / (2u * c.Hkv), seq = bp / pages_per_seq;
    const int head = item - bp * (2u * c.Hkv), g = head >> 1, b = seq;
    const bool values = head & 1;
    const UnitPos at = item_unit(p, u, values);
    int page = 0, base = 0, lo = 0, hi = 0, first = 0;
    if (seq < static_cast<uint32_t>(c.B)) {
      const NewTokens nt = new_tokens(p, b);
      first = nt.first;
      const int from = nt.first + nt.t0;  // first position written
      page = (from >> c.page_shift) + static_cast<int>(bp - seq * pages_per_seq);
      base = page << c.page_shift;
      lo = max(from - base, 0);
      hi = nt.t0 < nt.t1 ? min(nt.first + nt.t1 - base, 1 << c.page_shift) : 0;
    }
    const bool there = lo < hi;
    const Source src = there ? source_of(p, b, g, values, at) : Source{};
    const int step = warps * TL, slot0 = lo + share * TL + tl;  // this thread's rows: slot0, slot0 + step, ...
    const bool works = there && tl < TL;
    // rows as they come, so that many are under way; turned when they are needed, twice
    Unit x[kRows];
    auto load = [&](int s0) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (s0 + i * step < hi) x[i] = load_unit(src.src + static_cast<int64_t>(base + s0 + i * step - first) * src.step, at);
    };
    auto row_values = [&](int i, int s) {
      Values v = unit_values<BF16>(x[i]);
      if (src.turn) rotate_values(v, load_angles(p, base + s, u), p.interleaved);
      return v;
    };
    if (works) load(slot0);  // the page's lookup waits beside it
    const int id = there ? pool_page(c, b, page) : -1;
    const bool kept = slot0 + kRows * step >= hi;  // all of its rows are in registers
    auto largest = [&](auto finite) {  // of the item, by all of the block's warps
      float most = 0.f;
      if (works) {
        for (int s0 = slot0; s0 < hi; s0 += kRows * step) {
          if (!kept) load(s0);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            if (s0 + i * step >= hi) break;
            const Values v = row_values(i, s0 + i * step);
#pragma unroll
            for (int e = 0; e < 16; ++e) most = widen_max<finite.value>(most, v.x[e]);
          }
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
      if (lane == 0) tops[finite.value][warp] = most;
      __syncthreads();
      for (int i = 0; i < warps; ++i) most = fmaxf(most, tops[finite.value][warp - share + i]);
      return most;
    };
    float* scale = id >= 0 ? src.scales + static_cast<int64_t>(id) * c.Hkv + g : nullptr;
    const float old = id >= 0 && lo > 0 ? *scale : 0.f;
    float most = largest(std::false_type());
    const bool odd = most == INFINITY;
    bool any_odd = false;  // of the block's items
#pragma unroll
    for (int i = 0; i < kWarps; ++i) any_odd |= tops[0][i] == INFINITY;
    if (any_odd) {
      const float finite = largest(std::true_type());
      if (odd) most = finite;
    }
    if (id < 0) return;
    const float s0 = scale_for(most), sc = lo > 0 ? fmaxf(s0, old) : s0, inv = inverse_scale(sc);
    uint8_t* rows = src.pool + pool_row(c, id, g, 0);
    if (works) {
      for (int s = slot0; s < hi; s += kRows * step) {
        if (!kept) load(s);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (s + i * step >= hi) break;
          store_values(rows + static_cast<int64_t>(s + i * step) * D, at, row_values(i, s + i * step), inv, odd);
        }
      }
    }
    if (lo > 0 && s0 > old) rescale_chunks(rows, share * 32 + lane, lo * U, warps * 32, old * inv);
    if (share == 0 && lane == 0) *scale = sc;
    return;
  }
  append_queries<D, BF16>(p, (blockIdx.x - items_before) * kWarps + warp, groups_per_seq, row_chunks, row_items);
}

template <int D, bool BF16>
cudaError_t run_append8(const AppendLaunch& a) {
  constexpr int U = D / 16, TL = 32 / U;
  const AppendArgs p = append_args(a);
  if (a.T <= kFewTokens) {
    const int warps = 2 * a.c.Hkv + (a.T * p.Hq * U + 31) / 32;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(static_cast<unsigned>(a.c.B), static_cast<unsigned>((warps + kWarps - 1) / kWarps), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = a.stream;
    allow_early_launch(&cfg, attrs);
    return cudaLaunchKernelEx(&cfg, fa_kv_append8_kernel<D, BF16>, p);
  }
  const int page = 1 << a.c.page_shift;
  const int pages = (a.T + page - 2) / page + 1;  // that T tokens can touch
  const int64_t items = static_cast<int64_t>(a.c.B) * pages * a.c.Hkv * 2;
  int log2 = 0;  // warps of an item: so many that its rows fit the registers
  while ((1 << log2) < kWarps && (TL * kRows << log2) < page) ++log2;
  const int64_t item_blocks = ((items << log2) + kWarps - 1) / kWarps;
  const int groups = (a.T + TL - 1) / TL, chunks = (p.Hq + kRowBatch - 1) / kRowBatch;
  const int64_t row_items = static_cast<int64_t>(a.c.B) * groups * chunks;
  const int64_t blocks = item_blocks + (row_items + kWarps - 1) / kWarps;
  if (items > INT32_MAX || row_items > INT32_MAX || blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const uint64_t per_block = ((static_cast<uint64_t>(item_blocks) << 32) + blocks - 1) / blocks;
  return launch_kernel(fa_kv_append8_many_kernel<D, BF16>, blocks, kThreads, 0, a.stream, 1, p, static_cast<uint32_t>(pages),
                       per_block, log2, static_cast<uint32_t>(groups), static_cast<uint32_t>(chunks),
                       static_cast<uint32_t>(row_items));
}

}  // namespace

cudaError_t launch_kv_append8(const AppendLaunch& a) {
  switch (a.c.D) {
    case 64: return a.bf16 ? run_append8<64, true>(a) : run_append8<64, false>(a);
    case 96: return a.bf16 ? run_append8<96, true>(a) : run_append8<96, false>(a);
    case 128: return a.bf16 ? run_append8<128, true>(a) : run_append8<128, false>(a);
    default: return a.bf16 ? run_append8<256, true>(a) : run_append8<256, false>(a);
  }
}

}  // namespace fa
