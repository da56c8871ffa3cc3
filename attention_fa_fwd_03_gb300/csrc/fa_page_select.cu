// Choosing the pages that the attention of a new token reads, from the
// element-wise bounds of each page's keys.
//
//   score(page) = max_h sum_d max(q_hd min_d, q_hd max_d)
//               = max_h sum_d (q_hd > 0 ? q_hd max_d : q_hd min_d)
//
// One launch: a cluster of CTAs per (sequence, KV head) scores its pages in fp32
// (bound by reading 4 D bytes of bounds per page and KV head) and leaves the
// scores in the shared memory of its first CTA, which finds the n_sel best.
//
// A score is the sum of q+ max_d + q- min_d with q+ = max(q, 0), q- = min(q, 0),
// both exact in 16 bits: a product of 16 pages' bounds with up to 8 query heads on
// the tensor cores. Which dimension meets which index of the product is free as
// long as both operands agree, so a thread's fragment is whole 16-byte chunks
// loaded straight from global memory.
//
// The choice is the one that scores in 64 bits give although nearly all the work
// is done in 32: with A the largest of sum_d max_h |q_hd| max(|min_d|, |max_d|)
// over the pages, a score is off by at most E = D 2^-23 A + 2 D 2^-126: the products are
// exact unless they are below fp32's normal numbers (bf16: what becomes of those, and of
// sums below 2^-126, is left open, at most 2^-126 each), the D additions at least single
// precision in an order and with a rounding that are left open. With tau the last place's value among the fp32 scores, its true
// value is within E of tau: pages above tau + 2 E are chosen, pages under tau - 2 E
// are not. Where those in between are more than the places left, they are computed
// again as exact products summed in two fp32 words (E2 = D 2^-45 A + 2^-130, the
// latter for products that underflow), and those that this leaves open too in 64
// bits, ranked by (score, lower page): the 64-bit units are so few that one page
// costs microseconds. Where more pages are in between than can be ranked directly, or
// bounds are no numbers, each gets a 64-bit score from sums of three fp32 words, eight
// pages to a warp. Where their scores are all one (a query of zeros, as padding has),
// the lower pages win and nothing is computed again.
//
// Measured in a chain of calls: 12 units of 126 pages 6.6 us, 8 units of 2048 pages
// (8.4 MB) 10.9 us, both bound by dependent loads, barriers and instruction fetch
// (scoring 7 K cycles, search 4 K, places 4 K); 256 ragged units of up to 1024 pages (67
// MB) 26 to 27 us, of which scoring moves 5.5 TB/s and the largest units and their choice
// are the rest. L2 prefetch of the next pass's bounds made that 28 us.
// 8 units of 2048 pages that all tie: 9.8 us with a query of zeros, 344 with equal bounds
// in bf16 (156 in fp16, which need no look-out for products beyond fp32); 2634 when each
// page's score was summed in 64 bits.
#include "fa_inst.cuh"
#include "fa_paged_launch.h"
#include "fa_paged_mma.cuh"

namespace fa {
namespace {

struct SelectArgs {
  PagedView c;
  const uint16_t* q;
  int Hq, n_sel, keep_first, keep_last;
  int *sel, *sel_lens;
  uint32_t* scores;          // [B * Hkv, max_pages] keys of scores beyond kHeld pages
  unsigned long long* keys;  // [B * Hkv, max_pages] 64-bit scores where they are needed
  int head_chunk;            // query heads held at a time
};

__device__ __forceinline__ int page_count(const PagedView& c, int b) {
  return (seq_lens(c, nullptr, b, 0).len + (1 << c.page_shift) - 1) >> c.page_shift;
}

// Larger of two with NaN the largest.
__device__ __forceinline__ float max_or_nan(float x, float y) { return y > x || y != y ? y : x; }

constexpr int kSelectRanks = 8;       // CTAs of a cluster at most
constexpr int kHeld = 12 * 1024;      // pages whose scores are held in shared memory
constexpr int kFewTies = 256;         // pages in between that are ranked directly
constexpr int kQuerySmem = 36 * 1024;

// Query heads in shared memory: rows of q+, rows of q-, then the row of largest
// magnitudes, 16-bit, padded by 16 bytes so that 8 rows' chunks have other banks.
__host__ __device__ constexpr int query_pitch(int D) { return 2 * D + 16; }
inline int query_bytes(int heads, int D) { return (2 * heads + 1) * query_pitch(D); }

// Order-preserving maps (NaN highest, -0 as +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return ~0u;
  const uint32_t i = __float_as_uint(x + 0.f);
  return i >> 31 ? ~i : i | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const unsigned long long i = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  return i >> 63 ? ~i : i | (1ull << 63);
}

// What a CTA found beside the scores.
struct ScoreStats {
  float a;            // largest A
  int odd;            // a score or bound that is no number
  uint32_t lo, hi;    // smallest and largest key
};

template <bool BF16>
__device__ __forceinline__ uint32_t abs_max2(uint32_t x, uint32_t y) {
  using T2 = std::conditional_t<BF16, __nv_bfloat162, __half2>;
  const T2 r = __hmax2(__habs2(*reinterpret_cast<T2*>(&x)), __habs2(*reinterpret_cast<T2*>(&y)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Pool pages of the rows that this thread of CTA `rank` takes in its first pass, as
// the page table has them: read before the lengths are known, checked after.
struct FirstRows {
  int id[2];
};
template <int T>
__device__ __forceinline__ FirstRows first_rows(const SelectArgs& p, int b, int rank) {
  FirstRows f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int page = p.keep_first + rank * (T / 2) + 16 * (threadIdx.x >> 5) + ((threadIdx.x & 31) >> 2) + 8 * k;
    f.id[k] = page < p.c.max_pages ? p.c.table[static_cast<int64_t>(b) * p.c.max_pages + page] : -1;
  }
  return f;
}

// Scores of the pages keep_first + i, i < end, of (b, g) that are rank `rank`'s of
// `ranks`: passes of T / 2 in turn. put(i, key) for each, by one lane; get(i) gives
// back what was put (heads beyond head_chunk).
template <int T, int D, bool BF16, class Put, class Get>
__device__ __forceinline__ ScoreStats score_pages(const SelectArgs& p, uint8_t* qs, int b, int g, int rank, int ranks,
                                                  int end, const FirstRows& firsts, const Put& put, const Get& get) {
  constexpr int CH = D / 32, BATCH = CH == 3 ? 3 : 2;  // a thread's chunks of a row, and how many at a time
  constexpr int PITCH = query_pitch(D);
  const PagedView& c = p.c;
  const int reps = p.Hq / c.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane >> 2, col = lane & 3;
  uint8_t* qmag = qs + 2 * p.head_chunk * PITCH;
  ScoreStats st = {0.f, 0, ~0u, 0u};
  // this thread's rows of a pass: pages base + row and base + row + 8
  const uint4* src[2];
  bool there[2];
  uint4 lo[2][BATCH], hi[2][BATCH];
  const int begin = rank * (T / 2), step = ranks * (T / 2);
  auto find_rows = [&](int base) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = base + row + 8 * k;
      int id = -1;
      if (base == begin + 16 * warp)
        id = i < end ? checked_page(c, firsts.id[k]) : -1;
      else if (i < end)
        id = pool_page(c, b, p.keep_first + i);
      there[k] = id >= 0;
      src[k] = reinterpret_cast<const uint4*>(c.bounds + (static_cast<int64_t>(max(id, 0)) * c.Hkv + g) * 2 * D) + col;
    }
  };
  auto load_rows = [&](int i0) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        lo[k][i] = there[k] ? src[k][4 * (i0 + i)] : make_uint4(0, 0, 0, 0);
        hi[k][i] = there[k] ? src[k][D / 8 + 4 * (i0 + i)] : make_uint4(0, 0, 0, 0);
      }
  };
  for (int h0 = 0; h0 < reps; h0 += p.head_chunk) {
    const int heads = min(p.head_chunk, reps - h0), tiles = (heads + 7) / 8;
    const bool last = h0 + heads == reps;
    if (h0 > 0) __syncthreads();
    find_rows(begin + 16 * warp);  // under way while the queries are laid out
    load_rows(0);
    // behind the last head it again, which changes no maximum
    for (int i = threadIdx.x; i < tiles * 8 * (D / 2); i += T) {
      const int r = i / (D / 2), d2 = i - r * (D / 2);
      const uint32_t x = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + h0 + min(r, heads - 1)) * D)[d2];
      const float2 f = unpack2<BF16>(x);
      *reinterpret_cast<uint32_t*>(qs + r * PITCH + 4 * d2) = pack2<BF16>(f.x < 0.f ? 0.f : f.x, f.y < 0.f ? 0.f : f.y);
      *reinterpret_cast<uint32_t*>(qs + (p.head_chunk + r) * PITCH + 4 * d2) =
          pack2<BF16>(f.x > 0.f ? 0.f : f.x, f.y > 0.f ? 0.f : f.y);
    }
    __syncthreads();
    for (int d2 = threadIdx.x; d2 < D / 2; d2 += T) {
      uint32_t m = 0;
      for (int r = 0; r < heads; ++r) {
        m = abs_max2<BF16>(m, *reinterpret_cast<const uint32_t*>(qs + r * PITCH + 4 * d2));
        m = abs_max2<BF16>(m, *reinterpret_cast<const uint32_t*>(qs + (p.head_chunk + r) * PITCH + 4 * d2));
      }
      *reinterpret_cast<uint32_t*>(qmag + 4 * d2) = m;
    }
    __syncthreads();
    for (int base = begin + 16 * warp; base < end; base += step) {
      if (base != begin + 16 * warp) {
        find_rows(base);
        load_rows(0);
      }
      float best[2] = {-INFINITY, -INFINITY}, most[2] = {0.f, 0.f};
      for (int t = 0; t < tiles; ++t) {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i0 = 0; i0 < CH; i0 += BATCH) {
          if (CH > BATCH && (i0 > 0 || t > 0)) load_rows(i0);
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int at = 16 * (col + 4 * (i0 + i));
            const uint4 up = *reinterpret_cast<const uint4*>(qs + (8 * t + row) * PITCH + at);
            const uint4 down = *reinterpret_cast<const uint4*>(qs + (p.head_chunk + 8 * t + row) * PITCH + at);
            const uint32_t h0f[4] = {hi[0][i].x, hi[1][i].x, hi[0][i].y, hi[1][i].y};
            const uint32_t h1f[4] = {hi[0][i].z, hi[1][i].z, hi[0][i].w, hi[1][i].w};
            const uint32_t l0f[4] = {lo[0][i].x, lo[1][i].x, lo[0][i].y, lo[1][i].y};
            const uint32_t l1f[4] = {lo[0][i].z, lo[1][i].z, lo[0][i].w, lo[1][i].w};
            mma16816<BF16>(s, h0f, up.x, up.y);
            mma16816<BF16>(s, h1f, up.z, up.w);
            mma16816<BF16>(s, l0f, down.x, down.y);
            mma16816<BF16>(s, l1f, down.z, down.w);
            if (t == 0) {
              const uint4 mag = *reinterpret_cast<const uint4*>(qmag + at);
              uint32_t m0[4], m1[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                m0[e] = abs_max2<BF16>(h0f[e], l0f[e]);
                m1[e] = abs_max2<BF16>(h1f[e], l1f[e]);
              }
              mma16816<BF16>(a, m0, mag.x, mag.y);
              mma16816<BF16>(a, m1, mag.z, mag.w);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          best[k] = max_or_nan(best[k], max_or_nan(s[2 * k], s[2 * k + 1]));
          if (t == 0) most[k] = a[2 * k];  // every column has it
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        best[k] = max_or_nan(best[k], __shfl_xor_sync(0xffffffffu, best[k], 1));
        best[k] = max_or_nan(best[k], __shfl_xor_sync(0xffffffffu, best[k], 2));
        const int i = base + row + 8 * k;
        if (col != 0 || i >= end) continue;
        float x = best[k];
        if (there[k]) {
          st.odd |= x != x || isinf(x) || !(most[k] < INFINITY);
          st.a = fmaxf(st.a, most[k]);
        } else {
          x = -INFINITY;  // a bad page
        }
        uint32_t key = order_key(x);
        if (h0 > 0) key = max(key, get(i));
        put(i, key);
        if (last) {
          st.lo = min(st.lo, key);
          st.hi = max(st.hi, key);
        }
      }
      __syncwarp();
    }
  }
  return st;
}

// ------------------------------------------------------------------- choice
// Sums over the block of three counts of every thread.
struct BlockCounts {
  int (*c)[3];  // three sets in shared memory, all zero at first
  int round;
  // one barrier a round: set k is read after barrier k, and cleared after
  // barrier k + 1, before barrier k + 2 lets anyone add to it again
  __device__ __forceinline__ void add(int x0, int x1, int x2, int (&sum)[3]) {
    int* set = c[round % 3];
    x0 = __reduce_add_sync(0xffffffffu, x0);
    x1 = __reduce_add_sync(0xffffffffu, x1);
    x2 = __reduce_add_sync(0xffffffffu, x2);
    if ((threadIdx.x & 31) == 0) {
      if (x0) atomicAdd(set, x0);
      if (x1) atomicAdd(set + 1, x1);
      if (x2) atomicAdd(set + 2, x2);
    }
    __syncthreads();
    sum[0] = set[0];
    sum[1] = set[1];
    sum[2] = set[2];
    if (threadIdx.x < 3) c[(round + 2) % 3][threadIdx.x] = 0;
    ++round;
  }
};

// The need-th largest of the keys that get(i, &key) gives for i in [0, n), all of
// them in [lo, hi]: the largest T with at least `need` keys >= T, two bits at a
// time from the first bit in which lo and hi differ.
template <int T, class K, class Get>
__device__ __forceinline__ K kth_largest(BlockCounts& counts, int n, int need, K lo, K hi, const Get& get) {
  if (lo == hi) return lo;
  int bit = 63 - __clzll(static_cast<long long>(lo ^ hi));
  bit -= bit & 1;
  K t = hi >> bit >> 2 << bit << 2;  // shifts of 2 apart: bit + 2 may be the type's width
#pragma unroll 1
  for (; bit >= 0; bit -= 2) {
    const K t1 = t | (static_cast<K>(1) << bit), t2 = t | (static_cast<K>(2) << bit), t3 = t | (static_cast<K>(3) << bit);
    int a = 0, b = 0, e = 0;
    for (int i = threadIdx.x; i < n; i += T) {
      K k;
      if (!get(i, &k)) continue;
      a += k >= t1;
      b += k >= t2;
      e += k >= t3;
    }
    int sum[3];
    counts.add(a, b, e, sum);
    t = sum[2] >= need ? t3 : sum[1] >= need ? t2 : sum[0] >= need ? t1 : t;
  }
  return t;
}

// Exclusive prefix sum over the block's threads, and the total. One barrier: calls
// in a row take the two halves of warp_sums in turn.
template <int T>
__device__ __forceinline__ int block_before(int x, int (*halves)[T / 32], int turn, int* total) {
  int* warp_sums = halves[turn & 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  static_assert(T / 32 <= 32, "one warp adds the warps' sums");
  int sums = lane < (T / 32) ? warp_sums[lane] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sums, off);
    if (lane >= off) sums += y;
  }
  *total = __shfl_sync(0xffffffffu, sums, 31);
  const int before = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
  return incl - x + (warp > 0 ? before : 0);
}

// The need-th largest of the n keys in [lo, hi] that get(i) gives: a histogram of
// kBins equal ranges, the range of the wanted place, again within it until it
// holds few keys, which are ranked against each other. Bins of scores are nearly
// evenly filled, so one round is the rule; each round divides the range by kBins.
// Up to kDirectKeys of them, `held` in shared memory, are ranked at once (123 keys:
// 2.5 K cycles against 3.3 K; 343: 8.8 K).
constexpr int kBins = 2048;
constexpr int kFewKeys = 256;
constexpr int kDirectKeys = 128;
template <int T>
struct SearchSmem {
  int bins[kBins];
  uint32_t keys[kFewKeys];
  int warp_sums[2][T / 32];
  int bin, above, inside, count;
  uint32_t found;
};
template <int T, class Get>
__device__ __forceinline__ uint32_t kth_largest_score(SearchSmem<T>& sm, int n, int need, uint32_t lo, uint32_t hi,
                                                      const uint32_t* held, const Get& get) {
  constexpr int PER = kBins / T;
  if (lo == hi) return lo;
  if (held != nullptr && n <= kDirectKeys) {
    // few keys: each against all of them
    const int i = threadIdx.x;
    if (i < n) {
      const uint32_t k = held[i];
      int more = 0, equal = 0;
#pragma unroll 2
      for (int j = 0; j + 3 < n; j += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(held + j);
        more += (x.x > k) + (x.y > k) + (x.z > k) + (x.w > k);
        equal += (x.x == k) + (x.y == k) + (x.z == k) + (x.w == k);
      }
#pragma unroll 1
      for (int j = n & ~3; j < n; ++j) {
        more += held[j] > k;
        equal += held[j] == k;
      }
      if (more < need && need <= more + equal) sm.found = k;  // equal keys write the same value
    }
    __syncthreads();
    return sm.found;
  }
  int turn = 0;
  // A round leaves a range of at most 2^21 keys, then 2^10, then one. (The limit is for
  // keys in a workspace that somebody else writes.)
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    if (lo == hi) return lo;
    const int shift = max(0, 32 - __clz(hi - lo) - 11);
    static_assert(kBins == 1 << 11, "bins cover the range");
#pragma unroll
    for (int i = 0; i < PER; ++i) sm.bins[threadIdx.x + i * T] = 0;
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += T) {
      const uint32_t k = get(i);
      if (k >= lo && k <= hi) atomicAdd(&sm.bins[(k - lo) >> shift], 1);
    }
    __syncthreads();
    // thread t: bins from the top, kBins - 1 - PER t down
    int mine = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += sm.bins[kBins - 1 - PER * threadIdx.x - i];
    int above = block_before<T>(mine, sm.warp_sums, turn++, &total);
    if (above < need && need <= above + mine) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int bin = kBins - 1 - PER * threadIdx.x - i, x = sm.bins[bin];
        if (above < need && need <= above + x) {
          sm.bin = bin;
          sm.above = above;
          sm.inside = x;
        }
        above += x;
      }
    }
    __syncthreads();
    need -= sm.above;
    lo += static_cast<uint32_t>(sm.bin) << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
    const int inside = sm.inside;
    if (inside <= kFewKeys) {
      for (int i = threadIdx.x; i < n; i += T) {
        const uint32_t k = get(i);
        if (k < lo || k > hi) continue;
        const int at = atomicAdd(&sm.count, 1);
        if (at < kFewKeys) sm.keys[at] = k;
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < inside) {
        const uint32_t k = sm.keys[threadIdx.x];
        int more = 0, equal = 0;
        for (int i = 0; i < inside; ++i) {
          more += sm.keys[i] > k;
          equal += sm.keys[i] == k;
        }
        if (more < need && need <= more + equal) sm.found = k;  // equal keys write the same value
      }
      __syncthreads();
      return sm.found;
    }
    __syncthreads();  // before the bins are cleared again
  }
  return lo;
}

// Store to the first CTA of the cluster, at the place `at` has in this one's
// shared memory.
__device__ __forceinline__ void st_first(const uint32_t* at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(smem_u32(at), 0)), "r"(v) : "memory");
}

// The 64-bit key of page i of the competing ones, by a whole warp.
template <int D, bool BF16>
__device__ __forceinline__ unsigned long long exact_key(const SelectArgs& p, int b, int g, int page) {
  const PagedView& c = p.c;
  const int lane = threadIdx.x & 31, reps = p.Hq / c.Hkv;
  const int id = pool_page(c, b, page);
  if (id < 0) return 0;
  const uint16_t* lo = c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * D;
  double x[D / 32][2];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    x[i][0] = unpack2<BF16>(lo[lane + 32 * i]).x;
    x[i][1] = unpack2<BF16>(lo[D + lane + 32 * i]).x;
  }
  double best = 0.0;
  for (int r = 0; r < reps; ++r) {
    const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + r) * D;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const double y = unpack2<BF16>(q[lane + 32 * i]).x;
      const double u = y * x[i][0], v = y * x[i][1];
      s += u > v || u != u ? u : v;
    }
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (r == 0 || s > best || s != s) best = s;
    if (best != best) break;
  }
  return order_key(best);
}

// s + e exactly, as the rounded sum and its error.
__device__ __forceinline__ void two_sum(float a, float b, float* s, float* e) {
  *s = __fadd_rn(a, b);
  const float t = __fsub_rn(*s, a);
  *e = __fadd_rn(__fsub_rn(a, __fsub_rn(*s, t)), __fsub_rn(b, t));
}

// The score of a page that is there, as the sum of two fp32 words, by a whole
// warp: products are exact in fp32 (16-bit factors), errors of the sums are kept.
template <int D, bool BF16>
__device__ __forceinline__ float2 two_word_score(const SelectArgs& p, int b, int g, int page) {
  const PagedView& c = p.c;
  const int lane = threadIdx.x & 31, reps = p.Hq / c.Hkv;
  const int id = max(pool_page(c, b, page), 0);
  const uint16_t* lo = c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * D;
  float x[D / 32][2];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    x[i][0] = unpack2<BF16>(lo[lane + 32 * i]).x;
    x[i][1] = unpack2<BF16>(lo[D + lane + 32 * i]).x;
  }
  float2 best = make_float2(-INFINITY, 0.f);
#pragma unroll 4
  for (int r = 0; r < reps; ++r) {
    const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + r) * D;
    float s = 0.f, e = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float y = unpack2<BF16>(q[lane + 32 * i]).x;
      float err;
      two_sum(s, __fmul_rn(y, y < 0.f ? x[i][0] : x[i][1]), &s, &err);
      e = __fadd_rn(e, err);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      // both lanes of a pair add in the same order, so all lanes agree
      const float s2 = __shfl_xor_sync(0xffffffffu, s, off), e2 = __shfl_xor_sync(0xffffffffu, e, off);
      const bool low = (lane & off) == 0;
      float err;
      two_sum(low ? s : s2, low ? s2 : s, &s, &err);
      e = __fadd_rn(__fadd_rn(e, e2), err);
    }
    float hi, rest;
    two_sum(s, e, &hi, &rest);
    if (hi > best.x || (hi == best.x && rest > best.y)) best = make_float2(hi, rest);
  }
  return best;
}

// The 64-bit key of a page (-1: none) by 4 lanes, eight pages to a warp: sums in three
// fp32 words, s + e + f, which hold more than 64 bits' 53, made one number at the end.
// Terms that are no finite numbers are summed apart, where they decide. `lossy`: a bf16 product was too small or too large for fp32. Which
// lane adds which dimensions depends on the page's bounds and the query only, so pages
// with the same bounds get the same key. Called by whole warps.
template <int D, bool BF16>
__device__ __forceinline__ unsigned long long three_word_key(const SelectArgs& p, int b, int g, int page, bool* lossy) {
  const PagedView& c = p.c;
  const int lane = threadIdx.x & 31, col = lane & 3, reps = p.Hq / c.Hkv;
  const int id = page >= 0 ? pool_page(c, b, page) : -1;
  const uint4* lo4 = reinterpret_cast<const uint4*>(c.bounds + (static_cast<int64_t>(max(id, 0)) * c.Hkv + g) * 2 * D);
  bool lost = false;
  double best = 0.0;
  for (int r = 0; r < reps; ++r) {
    const uint4* q4 = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + r) * D);
    float s = 0.f, e = 0.f, f = 0.f, special = 0.f;
#pragma unroll 1
    for (int ch = col; ch < D / 8; ch += 4) {
      const uint4 xl = lo4[ch], xh = lo4[D / 8 + ch], xq = q4[ch];
      const uint32_t wl[4] = {xl.x, xl.y, xl.z, xl.w}, wh[4] = {xh.x, xh.y, xh.z, xh.w}, wq[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 l2 = unpack2<BF16>(wl[i / 2]), h2 = unpack2<BF16>(wh[i / 2]), q2 = unpack2<BF16>(wq[i / 2]);
        const float l = i & 1 ? l2.y : l2.x, h = i & 1 ? h2.y : h2.x, y = i & 1 ? q2.y : q2.x;
        const float u = __fmul_rn(y, l), v = __fmul_rn(y, h);
        const float t = u > v || u != u ? u : v;
        if (BF16) {
          // 2^-125: a product of 16 bits above it is exact
          lost |= y != 0.f && ((l != 0.f && fabsf(u) < 2.3509887e-38f) || (h != 0.f && fabsf(v) < 2.3509887e-38f));
          lost |= fabsf(y) < INFINITY && ((fabsf(l) < INFINITY && isinf(u)) || (fabsf(h) < INFINITY && isinf(v)));
        }
        const bool finite = fabsf(t) < INFINITY;
        if (!finite) special += t;
        float e1, e2;
        two_sum(s, finite ? t : 0.f, &s, &e1);
        two_sum(e, e1, &e, &e2);
        f = __fadd_rn(f, e2);
      }
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      // both lanes of a pair add in the same order, so both have the same words
      const float s2 = __shfl_xor_sync(0xffffffffu, s, off), e2 = __shfl_xor_sync(0xffffffffu, e, off);
      const float f2 = __shfl_xor_sync(0xffffffffu, f, off);
      special += __shfl_xor_sync(0xffffffffu, special, off);
      const bool low = (lane & off) == 0;
      float s_err, e_err, e_err2;
      two_sum(low ? s : s2, low ? s2 : s, &s, &s_err);
      two_sum(low ? e : e2, low ? e2 : e, &e, &e_err);
      two_sum(e, s_err, &e, &e_err2);
      f = __fadd_rn(__fadd_rn(low ? f : f2, low ? f2 : f), __fadd_rn(e_err, e_err2));
    }
    if (BF16) lost |= special == 0.f && !(fabsf(s) < INFINITY);  // finite terms beyond fp32
    const double x = special != 0.f ? static_cast<double>(special)
                                    : static_cast<double>(s) + (static_cast<double>(e) + static_cast<double>(f));
    if (r == 0 || x > best || x != x) best = x;  // a NaN stays
  }
  lost |= __shfl_xor_sync(0xffffffffu, lost, 1);
  lost |= __shfl_xor_sync(0xffffffffu, lost, 2);
  *lossy = lost && id >= 0;
  return id < 0 ? 0ull : order_key(best);
}

// The chosen of pages i < n into their places, in ascending order: a thread takes runs
// of four. state(i, key): 2 chosen, 0 not, 1 (where `ties`) chosen if among the first
// `equal` of its kind. (There are as many chosen as places, unless the scores changed
// under the call.)
template <int T, class Get4, class State>
__device__ __forceinline__ void place_pages(int* sel, int first, int limit, int n, int (*warp_sums)[T / 32], bool ties,
                                            int equal, const Get4& get4, const State& state) {
  int turn = 0;
  int at = first, seen = 0;  // places given and equals met before this stretch
  for (int base = 0; base < n; base += 4 * T) {
    const int i0 = base + 4 * threadIdx.x;
    uint32_t k[4] = {0, 0, 0, 0};
    get4(i0, k);
    int st[4], same = 0, total;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      st[j] = i0 + j < n ? state(i0 + j, k[j]) : 0;
      same += st[j] == 1;
    }
    if (ties) {
      int t = seen + block_before<T>(same, warp_sums, turn++, &total);
      seen += total;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (st[j] == 1) st[j] = t++ < equal ? 2 : 0;
    }
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += st[j] == 2;
    int to = at + block_before<T>(mine, warp_sums, turn++, &total);
    at += total;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (st[j] == 2 && to < limit) sel[to++] = first + i0 + j;
  }
}

// The choice where many pages compete for the last places: those with an fp32 key in
// [low, high] are ranked by their 64-bit keys, left in the workspace. By all threads, as
// the kernel's last step. (A function of its own, called where nothing is needed after
// it: its registers and code are not the common path's.)
template <int T>
struct WideSmem {
  int (*counters)[3];
  int round;
  int (*warp_sums)[T / 32];
  unsigned long long* key_range;
};
template <int T, int D, bool BF16>
__device__ __noinline__ void choose_wide(const SelectArgs& p, WideSmem<T> sm, const uint32_t* keys32, int unit, int b,
                                         int g, int n, int places, uint32_t low, uint32_t high, bool odd) {
  BlockCounts counts{sm.counters, sm.round};
  unsigned long long* key_range = sm.key_range;
  unsigned long long* keys = p.keys + static_cast<int64_t>(unit) * p.c.max_pages;
  int* sel = p.sel + static_cast<int64_t>(unit) * p.n_sel;
  auto keys4 = [&](int i, uint32_t (&k)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) k[j] = keys32[i + j];
  };
  // one score for all of them: bad pages only, or a query of zeros over numbers
  const int reps = p.Hq / p.c.Hkv;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(b) * p.Hq + g * reps) * D);
  uint32_t any = 0;
  for (int i = threadIdx.x; i < reps * (D / 2); i += T) any |= q[i] & 0x7fff7fffu;
  const bool zero = !__syncthreads_or(any != 0);
  if (!odd && (zero || high == order_key(-INFINITY))) {
    place_pages<T>(sel, p.keep_first, p.n_sel - p.keep_last, n, sm.warp_sums, true, places, keys4,
                   [&](int, uint32_t k) { return k > high ? 2 : k < low ? 0 : 1; });
    return;
  }
  const int lane = threadIdx.x & 31;
  for (int i0 = 8 * (threadIdx.x >> 5); i0 < n; i0 += 8 * (T / 32)) {
    const int i = i0 + (lane >> 2);
    const uint32_t k = i < n ? keys32[i] : 0;
    const bool mine = i < n && k >= low && k <= high;
    if (!__any_sync(0xffffffffu, mine)) continue;
    bool lossy;
    const unsigned long long k64 = three_word_key<D, BF16>(p, b, g, mine ? p.keep_first + i : -1, &lossy);
    if (mine && (lane & 3) == 0) keys[i] = k64;
    for (unsigned left = __ballot_sync(0xffffffffu, lossy && (lane & 3) == 0); left != 0; left &= left - 1) {
      const int at = i0 + ((__ffs(left) - 1) >> 2);
      const unsigned long long x = exact_key<D, BF16>(p, b, g, p.keep_first + at);
      if (lane == 0) keys[at] = x;
    }
  }
  __syncthreads();
  auto key64 = [&](int i, unsigned long long* k) {
    const uint32_t k32 = keys32[i];
    if (k32 < low || k32 > high) return false;
    *k = keys[i];
    return true;
  };
  // the range they are in, often one value
  if (threadIdx.x == 0) {
    key_range[0] = ~0ull;
    key_range[1] = 0ull;
  }
  __syncthreads();
  unsigned long long least = ~0ull, most = 0ull;
  for (int i = threadIdx.x; i < n; i += T) {
    unsigned long long k;
    if (!key64(i, &k)) continue;
    least = min(least, k);
    most = max(most, k);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    least = min(least, __shfl_xor_sync(0xffffffffu, least, off));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  }
  if (lane == 0) {
    atomicMin(&key_range[0], least);
    atomicMax(&key_range[1], most);
  }
  __syncthreads();
  const unsigned long long cut = kth_largest<T, unsigned long long>(counts, n, places, key_range[0], key_range[1], key64);
  int above = 0;
  for (int i = threadIdx.x; i < n; i += T) {
    unsigned long long k;
    above += key64(i, &k) && k > cut;
  }
  int sum[3];
  counts.add(above, 0, 0, sum);
  place_pages<T>(sel, p.keep_first, p.n_sel - p.keep_last, n, sm.warp_sums, true, places - sum[0], keys4,
                 [&](int i, uint32_t k) { return k > high ? 2 : k < low ? 0 : keys[i] > cut ? 2 : keys[i] == cut ? 1 : 0; });
}

// T = 512: few sequences, the block alone on its SM; T = 256: three blocks share
// one, so that one's choice overlaps the others' loads.
template <int T, int D, bool BF16>
__global__ void __launch_bounds__(T, T == 512 ? 1 : 3)
fa_page_select_kernel(const __grid_constant__ SelectArgs p, int ranks) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ int counters[3][3];
  __shared__ SearchSmem<T> search;
  __shared__ uint32_t warp_stats[(T / 32)][4], rank_stats[kSelectRanks][5];
  __shared__ int cta_pages;
  __shared__ unsigned long long tie_key[kFewTies], key_range[2];
  __shared__ float2 tie_score[kFewTies], tie_cut;
  __shared__ int tie_page[kFewTies], ties_found;
  uint8_t* qs = dyn;
  uint32_t* held = reinterpret_cast<uint32_t*>(dyn + (2 * p.head_chunk + 1) * query_pitch(D));
  if (threadIdx.x < 9) counters[threadIdx.x / 3][threadIdx.x % 3] = 0;
  if (threadIdx.x == 9) ties_found = 0;
  cluster_arrive_relaxed();  // waited for before the first store into the first CTA
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int unit = blockIdx.x / ranks, rank = blockIdx.x - unit * ranks;
  const int b = unit / c.Hkv, g = unit - b * c.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const FirstRows firsts = first_rows<T>(p, b, rank);
  // One reading of the length for the whole CTA, whose threads meet at barriers that
  // depend on it. CTAs of a cluster that read different ones (somebody writes them under
  // the call) find that out below.
  if (threadIdx.x == 0) cta_pages = page_count(c, b);
  __syncthreads();
  const int pages = cta_pages;
  // pages keep_first + i, i < n, compete for `need` places
  const int need = p.n_sel - p.keep_first - p.keep_last;
  const int n = pages - p.keep_first - p.keep_last;
  const bool all = pages <= p.n_sel;
  // scores go to the first CTA's shared memory where they fit and are final at once
  const bool local = n <= kHeld && p.Hq / c.Hkv <= p.head_chunk;
  uint32_t* far = p.scores + static_cast<int64_t>(unit) * c.max_pages;
  cluster_wait();
  if (!all && need > 0) {
    ScoreStats st = score_pages<T, D, BF16>(
        p, qs, b, g, rank, ranks, n, firsts,
        [&](int i, uint32_t k) {
          if (local)
            st_first(held + i, k);
          else
            far[i] = k;
        },
        [&](int i) { return far[i]; });
    st.a = warp_max(st.a);
    st.odd = __any_sync(0xffffffffu, st.odd);
    st.lo = __reduce_min_sync(0xffffffffu, st.lo);
    st.hi = __reduce_max_sync(0xffffffffu, st.hi);
    if (lane == 0) {
      warp_stats[warp][0] = __float_as_uint(st.a);
      warp_stats[warp][1] = static_cast<uint32_t>(st.odd);
      warp_stats[warp][2] = st.lo;
      warp_stats[warp][3] = st.hi;
    }
    __syncthreads();
    if (threadIdx.x < 4) {
      uint32_t x = warp_stats[0][threadIdx.x];
      for (int w = 1; w < (T / 32); ++w) {
        const uint32_t y = warp_stats[w][threadIdx.x];
        x = threadIdx.x == 2 ? min(x, y) : max(x, y);  // A is not negative: its bits order like it
      }
      st_first(&rank_stats[rank][threadIdx.x], x);
    }
  }
  if (threadIdx.x == 32) st_first(&rank_stats[rank][4], static_cast<uint32_t>(pages));
  __syncwarp();
  if (ranks > 1)
    cluster_barrier();  // every CTA's scores are with the first
  else
    __syncthreads();
  if (rank != 0) return;

  int* sel = p.sel + static_cast<int64_t>(unit) * p.n_sel;
  if (threadIdx.x == 0) p.sel_lens[unit] = min(pages, p.n_sel);
  float a_max = 0.f;
  uint32_t odd = 0, key_lo = ~0u, key_hi = 0u;
  bool agree = true;
#pragma unroll
  for (int r = 0; r < kSelectRanks; ++r) {
    if (r >= ranks) break;
    a_max = fmaxf(a_max, __uint_as_float(rank_stats[r][0]));
    odd |= rank_stats[r][1];
    key_lo = min(key_lo, rank_stats[r][2]);
    key_hi = max(key_hi, rank_stats[r][3]);
    agree &= rank_stats[r][4] == static_cast<uint32_t>(pages);
  }
  if (all || !agree) {
    for (int i = threadIdx.x; i < p.n_sel; i += T) sel[i] = i < pages ? i : -1;
    return;
  }
  for (int i = threadIdx.x; i < p.keep_first; i += T) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += T) sel[p.n_sel - p.keep_last + i] = pages - p.keep_last + i;
  if (need == 0) return;
  auto key32 = [&](int i) { return local ? held[i] : far[i]; };
  BlockCounts counts{counters, 0};
  uint32_t low = 0, high = ~0u;  // keys above `high` are in, under `low` out
  int sum[3];
  int sure = 0, between = n;
  if (!odd) {
    const uint32_t tau = kth_largest_score<T>(search, n, need, key_lo, key_hi, local ? held : nullptr, key32);
    const float t = order_value(tau);
    // 2 E, with room for the error of A itself and the roundings of t -+ err
    const float err = 2.02f * D * 1.1920929e-7f * a_max + fabsf(t) * 2.4e-7f + (BF16 ? 5.f * D * 1.1754944e-38f : 0.f);
    if (t > -INFINITY) {
      low = order_key(t - err);
      high = order_key(t + err);
    } else {
      low = high = tau;  // bad pages
    }
    int in = 0, mid = 0;
    for (int i = threadIdx.x; i < n; i += T) {
      const uint32_t k = key32(i);
      in += k > high;
      if (k >= low && k <= high) {
        ++mid;
        const int at = atomicAdd(&ties_found, 1);
        if (at < kFewTies) tie_page[at] = i;
      }
    }
    counts.add(in, mid, 0, sum);
    sure = sum[0];
    between = sum[1];
  }
  const int places = need - sure;   // for the pages in between
  const bool ranked = between > places;
  const bool few = ranked && !odd && between <= kFewTies && local && low != order_key(-INFINITY);
  if (few) {
    // Each against the others; the keys of those that win or lose leave
    // [low, high]. A bad page is in between only where all of them are.
    const int t = threadIdx.x;
    for (int i = warp; i < between; i += (T / 32)) {
      const float2 x = two_word_score<D, BF16>(p, b, g, p.keep_first + tie_page[i]);
      if (lane == 0) tie_score[i] = x;
    }
    __syncthreads();
    // the last place's score, and which are within 2 E2 of it
    auto minus = [](float2 x, float2 y) { return (x.x - y.x) + (x.y - y.y); };
    if (t < between) {
      const float2 x = tie_score[t];
      int above = 0;
      for (int i = 0; i < between; ++i) {
        const float2 y = tie_score[i];
        above += y.x > x.x || (y.x == x.x && (y.y > x.y || (y.y == x.y && i < t)));
      }
      if (above == places - 1) tie_cut = x;
    }
    __syncthreads();
    const float err2 = 2.02f * (D * 2.8421709e-14f * a_max + 7.3468397e-40f);
    int in = 0, open = 0;
    if (t < between) {
      const float d = minus(tie_score[t], tie_cut);
      in = d > err2;
      open = fabsf(d) <= err2;
    }
    counts.add(in, open, 0, sum);
    const int left = places - sum[0];
    const bool exact = sum[1] > left;
    if (exact) {
      for (int i = warp; i < between; i += (T / 32)) {
        if (!(fabsf(minus(tie_score[i], tie_cut)) <= err2)) continue;
        const unsigned long long k = exact_key<D, BF16>(p, b, g, p.keep_first + tie_page[i]);
        if (lane == 0) tie_key[i] = k;
      }
      __syncthreads();
    }
    if (t < between) {
      if (open && exact) {
        const int page = tie_page[t];
        const unsigned long long k = tie_key[t];
        int above = 0;
        for (int i = 0; i < between; ++i) {
          if (!(fabsf(minus(tie_score[i], tie_cut)) <= err2)) continue;
          above += tie_key[i] > k || (tie_key[i] == k && tie_page[i] < page);
        }
        in = above < left;
      } else {
        in |= open;
      }
      held[tie_page[t]] = in ? ~0u : 0u;
    }
    __syncthreads();
  } else if (ranked) {
    return choose_wide<T, D, BF16>(p, {counts.c, counts.round, search.warp_sums, key_range}, local ? held : far, unit, b, g,
                                   n, places, low, high, odd != 0);
  }
  place_pages<T>(
      sel, p.keep_first, p.n_sel - p.keep_last, n, search.warp_sums, false, 0,
      [&](int i, uint32_t (&k)[4]) {
        if (local && i + 3 < n) {
          const uint4 x = *reinterpret_cast<const uint4*>(held + i);
          k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n) k[j] = key32(i + j);
        }
      },
      [&](int, uint32_t k) { return k > high ? 2 : k < low ? 0 : !ranked || k == ~0u ? 2 : 0; });
}

template <int T, int D, bool BF16>
cudaError_t run_select(const SelectLaunch& a) {
  SelectArgs p;
  p.c = a.c;
  p.q = a.q;
  p.Hq = a.Hq; p.n_sel = a.n_sel; p.keep_first = a.keep_first; p.keep_last = a.keep_last;
  p.sel = a.sel; p.sel_lens = a.sel_lens;
  const int64_t units = static_cast<int64_t>(a.c.B) * a.c.Hkv;
  p.keys = static_cast<unsigned long long*>(a.ws);
  p.scores = reinterpret_cast<uint32_t*>(p.keys + units * a.c.max_pages);
  // query heads in eights, as many as shared memory is set aside for
  p.head_chunk = std::min((a.Hq / a.c.Hkv + 7) / 8, (kQuerySmem / query_pitch(D) - 1) / 16) * 8;
  // a cluster large enough that each CTA has one pass of T / 2 pages, but not many
  // more CTAs than the GPU holds at a time (B32 ragged to 1024 pages, T = 256: 35 us
  // with one CTA per unit, 26 with two, 32 with four)
  int ranks = 1;
  while (ranks < kSelectRanks && ranks * (T / 2) < a.c.max_pages && units * ranks < 3 * device_sm_count()) ranks *= 2;
  const int64_t held = std::min<int64_t>(kHeld, a.c.max_pages);
  const size_t smem = static_cast<size_t>(query_bytes(p.head_chunk, D)) + held * 4;
  auto kern = fa_page_select_kernel<T, D, BF16>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kQuerySmem + kHeld * 4);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, units * ranks, T, static_cast<int>(smem), a.stream, static_cast<unsigned>(ranks), p,
                       ranks);
}

// Few units: more threads each (one sequence of 2048 pages and 8 KV heads: 11.4
// us with 512, 13.7 with 256); many: more blocks per SM (B32 ragged: 35 and 26).
template <int D, bool BF16>
cudaError_t run_select_threads(const SelectLaunch& a) {
  const bool few = static_cast<int64_t>(a.c.B) * a.c.Hkv * kSelectRanks <= device_sm_count();
  return few ? run_select<512, D, BF16>(a) : run_select<256, D, BF16>(a);
}

template <bool BF16>
cudaError_t run_select_dt(const SelectLaunch& a) {
  switch (a.c.D) {
    case 64: return run_select_threads<64, BF16>(a);
    case 96: return run_select_threads<96, BF16>(a);
    case 128: return run_select_threads<128, BF16>(a);
    default: return run_select_threads<256, BF16>(a);
  }
}

}  // namespace

cudaError_t launch_page_select(const SelectLaunch& a) {
  return a.bf16 ? run_select_dt<true>(a) : run_select_dt<false>(a);
}

}  // namespace fa
