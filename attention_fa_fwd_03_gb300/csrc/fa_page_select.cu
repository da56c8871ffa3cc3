// Choosing the pages that the attention of a new token reads, from the
// element-wise bounds of each page's keys.
//
//   score(page) = max_h sum_d max(q_hd min_d, q_hd max_d)
//               = max_h sum_d (q_hd > 0 ? q_hd max_d : q_hd min_d)
//
// Two kernels: scores of every page in fp32 (bound by reading 4 D bytes of bounds
// per page and KV head), then one block per (sequence, KV head) that finds the
// n_sel best.
//
// The choice is the one that scores in 64 bits give although nearly all the work
// is done in 32: beside each score the first kernel leaves A = sum_d max_h |q_hd|
// max(|min_d|, |max_d|), and its score is off by at most E = 40 * 2^-24 A (at most
// 24 fused additions in a lane, one more for its two halves, four joining up to
// 16 lanes; the rest covers the rounding of A). With tau the wanted
// place's value among the fp32 scores and E the largest such bound, the true
// place's value is within E of tau: pages above tau + 2 E are chosen, pages under
// tau - 2 E are not, and only the few in between are computed again in 64 bits
// and ranked by (score, lower page). Without near ties there are no more of them
// than places, and nothing is computed again.
#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {
namespace {

struct SelectArgs {
  PagedView c;
  const uint16_t* q;
  int Hq, n_sel, keep_first, keep_last;
  int *sel, *sel_lens;
  float2* scores;                 // [B * Hkv, max_pages] (score, A); a bad page has (-inf, 0)
  unsigned long long* keys;       // [B * Hkv, max_pages] 64-bit scores where they are needed
  int group, head_chunk, chunk;   // KV heads of a block, query heads held at a time, pages of a block
};

__device__ __forceinline__ int page_count(const PagedView& c, int b) {
  return (cache_len(c, b) + (1 << c.page_shift) - 1) >> c.page_shift;
}

// Larger of two with NaN the largest.
__device__ __forceinline__ float max_or_nan(float x, float y) { return y > x || y != y ? y : x; }

// ------------------------------------------------------------------- scores
// A few lanes share a (page, KV head), 16 (D = 96: 24) dimensions each in
// 16-byte chunks; a thread takes two pages at a time so that a query value read
// from shared memory is used twice. Query heads are held as fp32 rows, then the
// row of their largest magnitudes.
constexpr int kScoreThreads = 256;
template <int D>
constexpr int kScoreLanes = D == 96 ? 4 : D / 16;
template <int D>
constexpr int kScoreSlots = kScoreThreads / kScoreLanes<D>;
constexpr int kScorePages = 2;            // pages per thread at a time
constexpr int kScoreSmem = 48 * 1024;

inline int score_pitch(int heads, int D) { return (heads + 1) * D + 4; }  // floats per KV head; + 4: other banks

template <int D, bool BF16>
__global__ void __launch_bounds__(kScoreThreads)
fa_page_score_kernel(const SelectArgs p) {
  extern __shared__ __align__(16) float qs[];
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int b = blockIdx.x, g0 = blockIdx.z * p.group;
  const int pages = page_count(c, b);
  const int end = min(pages - p.keep_last, static_cast<int>(blockIdx.y + 1) * p.chunk);
  int begin = blockIdx.y * p.chunk;
  if (pages <= p.n_sel || begin >= end) return;
  const int groups = min(p.group, c.Hkv - g0);
  const int reps = p.Hq / c.Hkv;
  const int pitch = (p.head_chunk + 1) * D + 4;
  constexpr int L = kScoreLanes<D>, CH = D / 8 / L;  // lanes of a page, chunks of a lane
  const int slot = threadIdx.x / L, lane = threadIdx.x % L;
  // the lanes of a slot run together, the slots of a warp need not
  const unsigned mates = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
  const int per_pass = kScoreSlots<D> / groups;  // pages side by side
  const int gi = slot % groups, ps = slot / groups;
  const int g = g0 + gi;
  float2* out = p.scores + (static_cast<int64_t>(b) * c.Hkv + g) * c.max_pages;
  for (int h0 = 0; h0 < reps; h0 += p.head_chunk) {
    const int heads = min(p.head_chunk, reps - h0);
    if (h0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < groups * heads * (D / 8); i += kScoreThreads) {
      const int ch = i % (D / 8), r = i / (D / 8), hi = r % heads, gg = r / heads;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(
                                p.q + (static_cast<int64_t>(b) * p.Hq + (g0 + gg) * reps + h0 + hi) * D) + ch);
      float4* dst = reinterpret_cast<float4*>(qs + gg * pitch + hi * D + 8 * ch);
      const float2 a = unpack2<BF16>(x.x), e = unpack2<BF16>(x.y), f = unpack2<BF16>(x.z), k = unpack2<BF16>(x.w);
      dst[0] = make_float4(a.x, a.y, e.x, e.y);
      dst[1] = make_float4(f.x, f.y, k.x, k.y);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * D; i += kScoreThreads) {
      const int gg = i / D, d = i - gg * D;
      float m = 0.f;
      for (int r = 0; r < heads; ++r) m = fmaxf(m, fabsf(qs[gg * pitch + r * D + d]));
      qs[gg * pitch + p.head_chunk * D + d] = m;
    }
    __syncthreads();
    if (ps >= per_pass) continue;
    const float* qg = qs + gi * pitch;
    for (int base = begin + ps; base < end; base += per_pass * kScorePages) {
      const uint4* src[kScorePages];
      bool there[kScorePages];
#pragma unroll
      for (int k = 0; k < kScorePages; ++k) {
        const int pg = base + k * per_pass;
        const int id = pg < end ? pool_page(c, b, pg) : -1;
        there[k] = id >= 0;
        src[k] = reinterpret_cast<const uint4*>(c.bounds + (static_cast<int64_t>(max(id, 0)) * c.Hkv + g) * 2 * D);
      }
      // the bounds' chunks of this lane: lane, lane + L, ...
      uint4 lo[kScorePages][CH], hi[kScorePages][CH];
#pragma unroll
      for (int k = 0; k < kScorePages; ++k)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          lo[k][i] = there[k] ? __ldg(src[k] + lane + L * i) : make_uint4(0, 0, 0, 0);
          hi[k][i] = there[k] ? __ldg(src[k] + D / 8 + lane + L * i) : make_uint4(0, 0, 0, 0);
        }
      float best[kScorePages], most[kScorePages];
#pragma unroll
      for (int k = 0; k < kScorePages; ++k) {
        best[k] = -INFINITY;
        most[k] = 0.f;
      }
      for (int r = 0; r <= heads; ++r) {
        const bool mags = r == heads;
        const float4* qr = reinterpret_cast<const float4*>(qg + (mags ? p.head_chunk : r) * D);
        uint64_t s2[kScorePages];
#pragma unroll
        for (int k = 0; k < kScorePages; ++k) s2[k] = f2_pack(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const float4 qa = qr[2 * (lane + L * i)], qb = qr[2 * (lane + L * i) + 1];
          const float qv[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = qv[2 * e], y = qv[2 * e + 1];
            const uint64_t up = f2_pack(fmaxf(x, 0.f), fmaxf(y, 0.f)), down = f2_pack(fminf(x, 0.f), fminf(y, 0.f));
#pragma unroll
            for (int k = 0; k < kScorePages; ++k) {
              const float2 l = unpack2<BF16>(reinterpret_cast<const uint32_t*>(&lo[k][i])[e]);
              const float2 h = unpack2<BF16>(reinterpret_cast<const uint32_t*>(&hi[k][i])[e]);
              if (mags) {
                s2[k] = ffma2(f2_pack(x, y), f2_pack(fmaxf(fabsf(l.x), fabsf(h.x)), fmaxf(fabsf(l.y), fabsf(h.y))), s2[k]);
              } else {
                s2[k] = ffma2(up, f2_pack(h.x, h.y), s2[k]);
                s2[k] = ffma2(down, f2_pack(l.x, l.y), s2[k]);
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kScorePages; ++k) {
          const float2 v = f2_unpack(s2[k]);
          float s = v.x + v.y;
#pragma unroll
          for (int off = 1; off < L; off <<= 1) s += __shfl_xor_sync(mates, s, off);
          if (mags)
            most[k] = s;
          else
            best[k] = max_or_nan(best[k], s);
        }
      }
#pragma unroll
      for (int k = 0; k < kScorePages; ++k) {
        const int pg = base + k * per_pass;
        if (lane != 0 || pg >= end) continue;
        float2 r = there[k] ? make_float2(best[k], most[k]) : make_float2(-INFINITY, 0.f);
        if (h0 > 0) {
          const float2 before = out[pg];
          r = make_float2(max_or_nan(before.x, r.x), max_or_nan(before.y, r.y));
        }
        out[pg] = r;
      }
    }
  }
}

// ------------------------------------------------------------------- choice
constexpr int kPickThreads = 512;
constexpr int kPickSmem = 12 * 1024;  // pages whose scores are held in shared memory

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

// The need-th largest of the keys that get(i, &key) gives for i in [0, n):
// largest T with at least `need` keys >= T, two bits at a time.
template <class K, class Get>
__device__ __forceinline__ K kth_largest(BlockCounts& counts, int n, int need, const Get& get) {
  K t = 0;
#pragma unroll 1
  for (int bit = static_cast<int>(sizeof(K)) * 8 - 2; bit >= 0; bit -= 2) {
    const K t1 = t | (static_cast<K>(1) << bit), t2 = t | (static_cast<K>(2) << bit), t3 = t | (static_cast<K>(3) << bit);
    int a = 0, b = 0, e = 0;
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
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

// Exclusive prefix sum over the block's threads.
__device__ __forceinline__ int block_before(int x, int* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = incl - x;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  return before;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPickThreads)
fa_page_pick_kernel(const SelectArgs p) {
  __shared__ uint32_t held[kPickSmem];
  __shared__ int counters[3][3], warp_sums[kPickThreads / 32];
  __shared__ float warp_max_a[kPickThreads / 32];
  if (threadIdx.x < 9) counters[threadIdx.x / 3][threadIdx.x % 3] = 0;
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int unit = blockIdx.x, b = unit / c.Hkv, g = unit - b * c.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pages = page_count(c, b);
  int* sel = p.sel + static_cast<int64_t>(unit) * p.n_sel;
  if (threadIdx.x == 0) p.sel_lens[unit] = min(pages, p.n_sel);
  if (pages <= p.n_sel) {
    for (int i = threadIdx.x; i < p.n_sel; i += kPickThreads) sel[i] = i < pages ? i : -1;
    return;
  }
  for (int i = threadIdx.x; i < p.keep_first; i += kPickThreads) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += kPickThreads) sel[p.n_sel - p.keep_last + i] = pages - p.keep_last + i;
  const int need = p.n_sel - p.keep_first - p.keep_last;
  if (need == 0) return;
  // pages keep_first + i, i < n, compete for `need` places
  const int n = pages - p.keep_first - p.keep_last;
  const float2* scores = p.scores + static_cast<int64_t>(unit) * c.max_pages + p.keep_first;
  unsigned long long* keys = p.keys + static_cast<int64_t>(unit) * c.max_pages + p.keep_first;

  float a_max = 0.f;
  bool odd = false;  // a score or bound that is no number
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const float2 s = scores[i];
    odd |= s.x != s.x || !(s.y < INFINITY) || (isinf(s.x) && s.y != 0.f);
    a_max = fmaxf(a_max, s.y);
    if (i < kPickSmem) held[i] = order_key(s.x);
  }
  a_max = warp_max(a_max);
  if (lane == 0) warp_max_a[warp] = a_max;
  odd = __syncthreads_or(odd);
  for (int w = 0; w < kPickThreads / 32; ++w) a_max = fmaxf(a_max, warp_max_a[w]);
  auto key32 = [&](int i) { return i < kPickSmem ? held[i] : order_key(scores[i].x); };

  BlockCounts counts{counters, 0};
  uint32_t low = 0, high = ~0u;  // keys above `high` are in, under `low` out
  int sum[3];
  int sure = 0, between = n;
  if (!odd) {
    const uint32_t tau = kth_largest<uint32_t>(counts, n, need, [&](int i, uint32_t* k) {
      *k = key32(i);
      return true;
    });
    const float t = order_value(tau);
    const float err = 2.02f * 40.f * 5.9604645e-8f * a_max + fabsf(t) * 2.4e-7f;
    if (t > -INFINITY) {
      low = order_key(t - err);
      high = order_key(t + err);
    } else {
      low = high = tau;
    }
    int in = 0, mid = 0;
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
      const uint32_t k = key32(i);
      in += k > high;
      mid += k >= low && k <= high;
    }
    counts.add(in, mid, 0, sum);
    sure = sum[0];
    between = sum[1];
  } else {
    high = ~0u;  // every page is computed again; no key is above ~0
  }
  const int places = need - sure;  // for the pages in between
  unsigned long long cut = 0;      // their keys above `cut` are in, and the first `equal` at it
  int equal = between;
  if (between > places) {
    const int reps = p.Hq / c.Hkv;
    for (int i = warp; i < n; i += kPickThreads / 32) {
      const uint32_t k = key32(i);
      if (k < low || k > high) continue;
      const int id = pool_page(c, b, p.keep_first + i);
      unsigned long long key = 0;
      if (id >= 0) {
        const uint16_t* lo = c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * D;
        double best = 0.0;
        for (int r = 0; r < reps; ++r) {
          const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + r) * D;
          double s = 0.0;
          for (int d = lane; d < D; d += 32) {
            const double x = unpack2<BF16>(q[d]).x;
            const double u = x * unpack2<BF16>(lo[d]).x, v = x * unpack2<BF16>(lo[D + d]).x;
            s += u > v || u != u ? u : v;
          }
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (r == 0 || s > best || s != s) best = s;
          if (best != best) break;
        }
        key = order_key(best);
      }
      if (lane == 0) keys[i] = key;
    }
    __syncthreads();
    auto key64 = [&](int i, unsigned long long* k) {
      const uint32_t k32 = key32(i);
      if (k32 < low || k32 > high) return false;
      *k = keys[i];
      return true;
    };
    cut = kth_largest<unsigned long long>(counts, n, places, key64);
    int above = 0;
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
      unsigned long long k;
      above += key64(i, &k) && k > cut;
    }
    counts.add(above, 0, 0, sum);
    equal = places - sum[0];
  }
  // places in ascending order: a thread takes a run of pages
  const int per = (n + kPickThreads - 1) / kPickThreads;
  const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
  const bool ranked = between > places;
  // 2: in, 1: in if early enough among its equals, 0: out
  auto state = [&](int i) {
    const uint32_t k = key32(i);
    if (k > high) return 2;
    if (k < low) return 0;
    if (!ranked) return 2;
    const unsigned long long k64 = keys[i];
    return k64 > cut ? 2 : k64 == cut ? 1 : 0;
  };
  int ties = 0;
  if (ranked) {
    for (int i = i0; i < i1; ++i) ties += state(i) == 1;
    ties = block_before(ties, warp_sums);
  }
  int mine = 0, t = ties;
  for (int i = i0; i < i1; ++i) {
    const int s = state(i);
    mine += s == 2 || (s == 1 && t++ < equal);
  }
  int at = p.keep_first + block_before(mine, warp_sums);
  t = ties;
  for (int i = i0; i < i1; ++i) {
    const int s = state(i);
    if (s == 2 || (s == 1 && t++ < equal)) sel[at++] = p.keep_first + i;
  }
}

template <int D, bool BF16>
cudaError_t run_select(const SelectLaunch& a) {
  SelectArgs p;
  p.c = a.c;
  p.q = a.q;
  p.Hq = a.Hq; p.n_sel = a.n_sel; p.keep_first = a.keep_first; p.keep_last = a.keep_last;
  p.sel = a.sel; p.sel_lens = a.sel_lens;
  const int64_t units = static_cast<int64_t>(a.c.B) * a.c.Hkv;
  p.scores = static_cast<float2*>(a.ws);
  p.keys = reinterpret_cast<unsigned long long*>(p.scores + units * a.c.max_pages);
  // as many query heads, then KV heads, as shared memory holds
  const int reps = a.Hq / a.c.Hkv;
  p.head_chunk = std::min(reps, kScoreSmem / 4 / D - 2);
  const int pitch_bytes = 4 * score_pitch(p.head_chunk, D);
  p.group = std::max(1, std::min(std::min(a.c.Hkv, kScoreSlots<D>), kScoreSmem / pitch_bytes));
  const int per_pass = kScoreSlots<D> / p.group * kScorePages;
  // enough blocks to fill the GPU a few times over, but few enough that loading
  // the queries stays small beside the bounds
  const int64_t group_blocks = (a.c.Hkv + p.group - 1) / p.group;
  const int64_t want = std::max<int64_t>(1, static_cast<int64_t>(device_sm_count()) * 4 / std::max<int64_t>(1, a.c.B * group_blocks));
  int64_t chunk = (a.c.max_pages + want - 1) / want;
  chunk = std::max<int64_t>((chunk + per_pass - 1) / per_pass, 1) * per_pass;
  while ((a.c.max_pages + chunk - 1) / chunk > 65535) chunk *= 2;
  p.chunk = static_cast<int>(chunk);
  if (group_blocks > 65535) return cudaErrorInvalidConfiguration;
  if (a.c.max_pages > a.n_sel) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(static_cast<unsigned>(a.c.B), static_cast<unsigned>((a.c.max_pages + chunk - 1) / chunk),
                       static_cast<unsigned>(group_blocks));
    cfg.blockDim = dim3(kScoreThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.group) * pitch_bytes;
    cfg.stream = a.stream;
    allow_early_launch(&cfg, attrs);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_page_score_kernel<D, BF16>, p);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(fa_page_pick_kernel<D, BF16>, units, kPickThreads, 0, a.stream, 1, p);
}

template <bool BF16>
cudaError_t run_select_dt(const SelectLaunch& a) {
  switch (a.c.D) {
    case 64: return run_select<64, BF16>(a);
    case 96: return run_select<96, BF16>(a);
    case 128: return run_select<128, BF16>(a);
    default: return run_select<256, BF16>(a);
  }
}

}  // namespace

cudaError_t launch_page_select(const SelectLaunch& a) {
  return a.bf16 ? run_select_dt<true>(a) : run_select_dt<false>(a);
}

}  // namespace fa
