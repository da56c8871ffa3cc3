// Choosing the pages that the attention of a new token reads, from the
// element-wise bounds of each page's keys.
#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {
namespace {

struct SelectArgs {
  PagedView c;
  const uint16_t* q;
  int Hq, n_sel, keep_first, keep_last;
  int *sel, *sel_lens;
  unsigned long long* keys;  // [B * Hkv, max_pages]
};

constexpr int kSelectThreads = 256;

// Order-preserving map of a double (NaN highest, -0 as +0).
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const long long i = __double_as_longlong(x + 0.0);
  return i < 0 ? ~static_cast<unsigned long long>(i) : static_cast<unsigned long long>(i) | (1ull << 63);
}

template <bool BF16>
__global__ void __launch_bounds__(kSelectThreads)
fa_page_select_kernel(const SelectArgs p) {
  __shared__ int count;
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int unit = blockIdx.x, b = unit / c.Hkv, g = unit - b * c.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int reps = p.Hq / c.Hkv;
  const int pages = (cache_len(c, b) + (1 << c.page_shift) - 1) >> c.page_shift;
  int* sel = p.sel + static_cast<int64_t>(unit) * p.n_sel;
  unsigned long long* keys = p.keys + static_cast<int64_t>(unit) * c.max_pages;
  if (threadIdx.x == 0) p.sel_lens[unit] = min(pages, p.n_sel);
  for (int i = threadIdx.x; i < p.n_sel; i += kSelectThreads) sel[i] = pages <= p.n_sel && i < pages ? i : -1;
  if (pages <= p.n_sel) return;
  for (int pg = warp; pg < pages; pg += kSelectThreads / 32) {
    unsigned long long key = ~0ull;
    if (pg >= p.keep_first && pg < pages - p.keep_last) {
      const int id = pool_page(c, b, pg);
      double best = 0.0;
      key = 0;
      if (id >= 0) {
        const uint16_t* lo = c.bounds + (static_cast<int64_t>(id) * c.Hkv + g) * 2 * c.D;
        const uint16_t* hi = lo + c.D;
        for (int r = 0; r < reps; ++r) {
          const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.Hq + g * reps + r) * c.D;
          double s = 0.0;
          for (int d = lane; d < c.D; d += 32) {
            const float x = unpack2<BF16>(q[d]).x;
            const double u = static_cast<double>(x) * unpack2<BF16>(lo[d]).x;
            const double v = static_cast<double>(x) * unpack2<BF16>(hi[d]).x;
            s += u > v || u != u ? u : v;
          }
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (r == 0 || s > best || s != s) best = s;
          if (best != best) break;
        }
        key = order_key(best);
      }
    }
    if (lane == 0) keys[pg] = key;
  }
  __syncthreads();
  // rank of each page by (key, lower index first); then ascending places
  for (int base = 0; base < pages; base += kSelectThreads) {
    const int i = base + threadIdx.x;
    bool in = false;
    if (i < pages) {
      const unsigned long long k = keys[i];
      const bool kept = i < p.keep_first || i >= pages - p.keep_last;
      int above = p.keep_first + p.keep_last;
      if (!kept)
        for (int j = p.keep_first; j < pages - p.keep_last; ++j) above += keys[j] > k || (keys[j] == k && j < i);
      in = kept || above < p.n_sel;
    }
    if (threadIdx.x == 0 && base == 0) count = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
      __syncthreads();
      const int at = count;
      __syncthreads();
      if (warp == w) {
        const unsigned ballot = __ballot_sync(0xffffffffu, in);
        if (in) sel[at + __popc(ballot & ((1u << lane) - 1))] = i;
        if (lane == 0) count = at + __popc(ballot);
      }
    }
  }
}

template <bool BF16>
cudaError_t run_select(const SelectLaunch& a) {
  SelectArgs p;
  p.c = a.c;
  p.q = a.q;
  p.Hq = a.Hq; p.n_sel = a.n_sel; p.keep_first = a.keep_first; p.keep_last = a.keep_last;
  p.sel = a.sel; p.sel_lens = a.sel_lens;
  p.keys = static_cast<unsigned long long*>(a.ws);
  return launch_kernel(fa_page_select_kernel<BF16>, static_cast<int64_t>(a.c.B) * a.c.Hkv, kSelectThreads,
                       0, a.stream, 1, p);
}

}  // namespace

cudaError_t launch_page_select(const SelectLaunch& a) {
  return a.bf16 ? run_select<true>(a) : run_select<false>(a);
}

}  // namespace fa
