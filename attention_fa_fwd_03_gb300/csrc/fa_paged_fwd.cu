// Attention of up to 8 new tokens per sequence over the paged cache.
#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {
namespace {

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
};

constexpr int kWarps = 4;

// One block per (sequence, query head, token); a warp takes every kWarps-th
// key, a lane pairs of dimensions.
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarps)
fa_paged_fwd_kernel(const PagedFwdArgs p) {
  constexpr int NP = (D / 2 + 31) / 32;
  __shared__ float sm_o[kWarps][D], sm_m[kWarps], sm_l[kWarps];
  grid_wait_prior();
  grid_release_next();
  const PagedView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x;  // (b * Hq + h) * Tq + t
  const int t = row % p.Tq, bh = row / p.Tq, b = bh / p.Hq;
  const int g = (bh - b * p.Hq) / (p.Hq / c.Hkv);
  const int len = cache_len(c, b), n = new_len(c, p.new_lens, b, p.Tq);
  const int pos = len - n + t;
  const int pages = (len + (1 << c.page_shift) - 1) >> c.page_shift;
  int list = pages;
  const int64_t u = static_cast<int64_t>(b) * c.Hkv + g;
  if (p.sel != nullptr) {
    list = p.sel_lens[u];
    if (list < 0 || list > p.n_sel) {
      flag_bad_index(c);
      list = list < 0 ? 0 : p.n_sel;
    }
  }
  if (t >= n) list = 0;
  float qf[NP][2], acc[NP][2], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int d = lane + 32 * i;
    float2 x = make_float2(0.f, 0.f);
    if (d < D / 2) x = unpack2<BF16>(reinterpret_cast<const uint32_t*>(p.q)[static_cast<int64_t>(row) * (D / 2) + d]);
    qf[i][0] = x.x * p.scale_log2;
    qf[i][1] = x.y * p.scale_log2;
    acc[i][0] = acc[i][1] = 0.f;
  }
  for (int e = 0; e < list; ++e) {
    int page = e;
    if (p.sel != nullptr) {
      page = p.sel[u * p.n_sel + e];
      if (page < 0 || page >= pages) {
        flag_bad_index(c);
        continue;
      }
    }
    const int id = pool_page(c, b, page);
    if (id < 0) continue;
    for (int s = warp; s < (1 << c.page_shift); s += kWarps) {
      const int j = (page << c.page_shift) + s;
      if (j >= len || (p.causal && j > pos) || (p.window > 0 && pos >= j && pos - j >= p.window)) continue;
      const int64_t r = pool_row(c, id, g, s);
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(c.k + r);
      const uint32_t* vr = reinterpret_cast<const uint32_t*>(c.v + r);
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int d = lane + 32 * i;
        if (d < D / 2) {
          const float2 f = unpack2<BF16>(kr[d]);
          x = fmaf(qf[i][0], f.x, fmaf(qf[i][1], f.y, x));
        }
      }
      x = warp_sum(x);
      const float mn = fmaxf(m, x), alpha = exp2_rel(m, mn), w = exp2_rel(x, mn);
      m = mn;
      l = l * alpha + w;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int d = lane + 32 * i;
        const float2 f = d < D / 2 ? unpack2<BF16>(vr[d]) : make_float2(0.f, 0.f);
        acc[i][0] = fmaf(w, f.x, acc[i][0] * alpha);
        acc[i][1] = fmaf(w, f.y, acc[i][1] * alpha);
      }
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int d = lane + 32 * i;
    if (d < D / 2) {
      sm_o[warp][2 * d] = acc[i][0];
      sm_o[warp][2 * d + 1] = acc[i][1];
    }
  }
  __syncthreads();
  float mt = -INFINITY, lt = 0.f;
  for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm_m[w]);
  for (int w = 0; w < kWarps; ++w) lt += sm_l[w] * exp2_rel(sm_m[w], mt);
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
  for (int d = threadIdx.x; d < D / 2; d += 32 * kWarps) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2_rel(sm_m[w], mt);
      x += sm_o[w][2 * d] * f;
      y += sm_o[w][2 * d + 1] * f;
    }
    reinterpret_cast<uint32_t*>(p.o)[static_cast<int64_t>(row) * (D / 2) + d] = pack2<BF16>(x * inv, y * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = lt > 0.f ? (mt + log2f(lt)) * kLn2 : -INFINITY;
}

template <int D, bool BF16>
cudaError_t run_paged(const PagedFwdLaunch& a) {
  PagedFwdArgs p;
  p.c = a.c;
  p.q = a.q; p.o = a.o; p.lse = a.lse;
  p.Hq = a.Hq; p.Tq = a.Tq; p.causal = a.causal; p.window = a.window;
  p.scale_log2 = a.scale_log2;
  p.new_lens = a.new_lens;
  p.sel = a.sel; p.sel_lens = a.sel_lens; p.n_sel = a.n_sel;
  return launch_kernel(fa_paged_fwd_kernel<D, BF16>, static_cast<int64_t>(a.c.B) * a.Hq * a.Tq,
                       32 * kWarps, 0, a.stream, 1, p);
}

template <int D>
cudaError_t run_paged_dt(const PagedFwdLaunch& a) {
  return a.bf16 ? run_paged<D, true>(a) : run_paged<D, false>(a);
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedFwdLaunch& a) {
  switch (a.c.D) {
    case 64: return run_paged_dt<64>(a);
    case 96: return run_paged_dt<96>(a);
    case 128: return run_paged_dt<128>(a);
    default: return run_paged_dt<256>(a);
  }
}

}  // namespace fa
