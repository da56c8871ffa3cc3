// Appending new tokens to the paged cache: keys are rotated by their position,
// values copied, the tokens' queries rotated, and the element-wise bounds of
// the keys' pages kept.
//
//   (y_i, y_i') = (x_i cos - x_i' sin, x_i' cos + x_i sin)   per pair (i, i')
//
// in fp32, rounded once to the cache's type (what the page holds is what
// attention reads, so the bounds are taken of the rounded values).
//
// The work is one read and one write of every row. A thread owns a unit of 16
// elements that closes over its rotation pairs (two 16-byte chunks, rot / 2
// apart or adjacent), so a row is D / 16 threads.
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
    const float4 x = __ldg(c + i), y = __ldg(s + i);
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

// Whether position `pos` of sequence b has a slot and angles.
__device__ __forceinline__ bool position_ok(const AppendArgs& p, int pos) {
  if (pos >= 0 && (p.rot_dim == 0 || pos < p.rope_len)) return true;
  flag_bad_index(p.c);
  return false;
}

// Grid: x = (sequence, token), y = blocks of kAppendThreads units of the
// token's rows (values, queries, then keys).
template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads)
fa_kv_append_kernel(const AppendArgs p) {
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int units = c.D / 16;
  const int b = blockIdx.x / p.T, t = blockIdx.x - b * p.T;
  const int item = blockIdx.y * kAppendThreads + threadIdx.x;
  const int row = item / units, u = item - row * units;
  const int hq = p.q != nullptr ? p.Hq : 0;
  if (row >= 2 * c.Hkv + hq) return;
  const SeqLens sl = seq_lens(c, p.new_lens, b, p.T);
  const int n = sl.n, pos = sl.len - n + t;
  const bool valid = t < n && position_ok(p, pos);
  const bool is_v = row < c.Hkv, is_q = !is_v && row < c.Hkv + hq;
  UnitPos at = unit_pos(p, u);
  if (is_q) {
    const int h = row - c.Hkv;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (valid) {
      const uint16_t* src = p.q + b * p.qs.b + h * p.qs.h + t * p.qs.t;
      x = *reinterpret_cast<const uint4*>(src + at.a);
      y = *reinterpret_cast<const uint4*>(src + at.b);
      if (at.rotated) rotate_unit<BF16>(x, y, load_angles(p, pos, u), p.interleaved);
    }
    uint16_t* dst = p.q_out + ((static_cast<int64_t>(b) * p.Hq + h) * p.T + t) * c.D;
    *reinterpret_cast<uint4*>(dst + at.a) = x;
    *reinterpret_cast<uint4*>(dst + at.b) = y;
    return;
  }
  if (!valid) return;
  const int id = pool_page(c, b, pos >> c.page_shift);
  if (id < 0) return;
  const int slot = pos & ((1 << c.page_shift) - 1);
  if (is_v) {
    const uint16_t* src = p.v + b * p.vs.b + row * p.vs.h + t * p.vs.t;
    uint16_t* dst = c.v + pool_row(c, id, row, slot);
    reinterpret_cast<uint4*>(dst)[2 * u] = reinterpret_cast<const uint4*>(src)[2 * u];
    reinterpret_cast<uint4*>(dst)[2 * u + 1] = reinterpret_cast<const uint4*>(src)[2 * u + 1];
    return;
  }
  const int g = row - c.Hkv - hq;
  const uint16_t* src = p.k + b * p.ks.b + g * p.ks.h + t * p.ks.t;
  uint4 x = *reinterpret_cast<const uint4*>(src + at.a);
  uint4 y = *reinterpret_cast<const uint4*>(src + at.b);
  if (at.rotated) rotate_unit<BF16>(x, y, load_angles(p, pos, u), p.interleaved);
  uint16_t* dst = c.k + pool_row(c, id, g, slot);
  *reinterpret_cast<uint4*>(dst + at.a) = x;
  *reinterpret_cast<uint4*>(dst + at.b) = y;
}

// Bounds of every page that received a token, read back from the pool: one
// block per (sequence, page, KV head), a thread per pair of elements.
template <bool BF16>
__global__ void __launch_bounds__(128)
fa_kv_bounds_kernel(const AppendArgs p, int pages_per_seq) {
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int g = blockIdx.x % c.Hkv;
  const int bp = blockIdx.x / c.Hkv;
  const int b = bp / pages_per_seq;
  const SeqLens sl = seq_lens(c, p.new_lens, b, p.T);
  int first = sl.len - sl.n, last = sl.len;  // positions written
  if (first < 0) first = 0;
  if (p.rot_dim > 0 && last > p.rope_len) last = p.rope_len;
  const int page = (first >> c.page_shift) + (bp - b * pages_per_seq);
  const int base = page << c.page_shift;
  const int lo = max(first - base, 0), hi = min(last - base, 1 << c.page_shift);
  if (lo >= hi) return;
  const int id = pool_page(c, b, page);
  if (id < 0) return;
  uint32_t* bounds = reinterpret_cast<uint32_t*>(c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * c.D);
  for (int d = threadIdx.x; d < c.D / 2; d += 128) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(c.k + pool_row(c, id, g, 0)) + d;
    uint32_t mn = lo > 0 ? bounds[d] : src[lo * (c.D / 2)];
    uint32_t mx = lo > 0 ? bounds[c.D / 2 + d] : src[lo * (c.D / 2)];
    for (int s = lo; s < hi; ++s) {
      const uint32_t x = src[s * (c.D / 2)];
      mn = min2<BF16>(mn, x);
      mx = max2<BF16>(mx, x);
    }
    bounds[d] = mn;
    bounds[c.D / 2 + d] = mx;
  }
}

template <bool BF16>
cudaError_t run_append(const AppendLaunch& a) {
  AppendArgs p;
  p.c = a.c;
  p.k = a.k; p.v = a.v; p.q = a.q;
  p.q_out = a.q_out;
  p.ks = a.ks; p.vs = a.vs; p.qs = a.qs;
  p.Hq = a.Hq; p.T = a.T;
  p.new_lens = a.new_lens;
  p.cos_table = a.cos_table; p.sin_table = a.sin_table;
  p.rope_len = a.rope_len; p.rot_dim = a.rot_dim; p.interleaved = a.interleaved;
  const int rows = 2 * a.c.Hkv + (a.q != nullptr ? a.Hq : 0);
  const int64_t items = static_cast<int64_t>(rows) * (a.c.D / 16);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.gridDim = dim3(static_cast<unsigned>(a.c.B * a.T),
                     static_cast<unsigned>((items + kAppendThreads - 1) / kAppendThreads), 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = a.stream;
  allow_early_launch(&cfg, attrs);
  cudaError_t e = cudaLaunchKernelEx(&cfg, fa_kv_append_kernel<BF16>, p);
  if (e != cudaSuccess || a.c.bounds == nullptr) return e;
  const int page = 1 << a.c.page_shift;
  const int pages = (a.T + page - 2) / page + 1;
  return launch_kernel(fa_kv_bounds_kernel<BF16>, static_cast<int64_t>(a.c.B) * pages * a.c.Hkv, 128,
                       0, a.stream, 1, p, pages);
}

}  // namespace

cudaError_t launch_kv_append(const AppendLaunch& a) {
  return a.bf16 ? run_append<true>(a) : run_append<false>(a);
}

}  // namespace fa
