// Page tables and slot maps from the requests' lengths.
//
// Sequence b holds the pages [0, h0) and [f0, e0) and wants [0, h) and [f, e), where h
// covers the first keys that a window leaves visible, f is the page of the first key it
// shows and e the page behind the last key. What it gives back is a union of four
// intervals of pages, what it gets of two (see Plan), so both counts are a few
// comparisons per sequence; an exclusive sum over the sequences places each of its
// pages on the stack of free pages. No atomics: the order is that of the sequences.
//
// The work is a few words per sequence and per page that changes hands, microseconds
// of launch and dependent loads (lengths and states, then tables and stack). So one
// cluster does it: every CTA sums over all sequences for itself, 1024 at a time, then
// its warps take sequences in turn, several of them one where there are few. Pages given back have to be on the stack before
// any is taken from it, and states are written when nobody reads them any more: a
// barrier each. Slots of a few tokens are written by the same cluster, of many by a
// second launch that fills the GPU.
#include <algorithm>
#include <climits>

#include "../../include/fa.h"
#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {
namespace {

constexpr int kAssignThreads = 1024;
// Up to so many sequences and tokens one CTA does all, without a cluster's barriers. (Pages of 16, one
// CTA and eight, us: 8 sequences and a token each 5.1, 6.3; 64: 6.3, 6.5; 128: 8.3, 6.6. One
// sequence, 1024 tokens 5.0, 5.6; 8192: 6.6, 6.4.)
constexpr int kLoneB = 64, kLoneTokens = 4096;
// Up to so many tokens the cluster writes their slots. (Here and apart, us: 4 x 2048 6.4, 7.7;
// 16 x 1024 6.7, 7.4; 64 x 1024 8.7, 7.6; 256 x 8192 60, 15.6, of which the slots' bytes are 2.5.)
constexpr int kSlotsHere = 16384;

struct AssignArgs {
  int *table, *held, *free_pages, *free_count;
  const int *lens, *new_lens;
  int64_t* slots;  // null: none
  int B, num_pages, page_shift, max_pages, T, window, sinks;
  int slots_here;  // the cluster writes the slots
  uint32_t* status;
};

__device__ __forceinline__ int in_range(const AssignArgs& p, int x, int lo, int hi) {
  const int y = min(max(x, lo), hi);
  if (y != x) atomicOr(p.status, kStatusBadIndex);
  return y;
}

struct Lens {
  int len, n;
};
__device__ __forceinline__ Lens lens_of(const AssignArgs& p, int b) {
  const int len = p.lens[b], n = p.new_lens ? p.new_lens[b] : p.T;
  return {in_range(p, len, 0, p.max_pages << p.page_shift), in_range(p, n, 0, p.T)};
}

__device__ __forceinline__ int span(int lo, int hi) { return max(hi - lo, 0); }

// What a sequence holds and wants.
struct Plan {
  int h0, f0, e0, h, f, e;
  // given back, in ascending order: [h, min(h0, f)), [max(f0, h), min(e0, f)), [e, h0),
  // [max(f0, e), e0). (The second and the third are not both there.)
  __device__ __forceinline__ int back() const {
    return span(h, min(h0, f)) + span(max(f0, h), min(e0, f)) + span(e, h0) + span(max(f0, e), e0);
  }
  __device__ __forceinline__ int back_page(int i) const {
    int n = span(h, min(h0, f));
    if (i < n) return h + i;
    i -= n;
    n = span(max(f0, h), min(e0, f));
    if (i < n) return max(f0, h) + i;
    i -= n;
    n = span(e, h0);
    return i < n ? e + i : max(f0, e) + i - n;
  }
  // got: [e0, h), [max(e0, f), e)
  __device__ __forceinline__ int more() const { return span(e0, h) + span(max(e0, f), e); }
  __device__ __forceinline__ int more_page(int i) const {
    const int n = span(e0, h);
    return i < n ? e0 + i : max(e0, f) + i - n;
  }
};

__device__ __forceinline__ Plan make_plan(const AssignArgs& p, int b) {
  const Lens l = lens_of(p, b);
  const int a0 = p.held[3 * b], a1 = p.held[3 * b + 1], a2 = p.held[3 * b + 2];
  Plan x;
  x.h0 = in_range(p, a0, 0, p.max_pages);
  x.f0 = in_range(p, a1, x.h0, p.max_pages);
  x.e0 = in_range(p, a2, x.f0, p.max_pages);
  const bool gap = x.f0 > x.h0;
  const int page = 1 << p.page_shift;
  x.e = (l.len + page - 1) >> p.page_shift;
  if (p.window > 0) {
    x.h = min(x.e, (p.sinks + page - 1) >> p.page_shift);
    x.f = max(0, l.len - l.n - p.window + 1) >> p.page_shift;
    if (gap) {
      x.h = min(x.h, x.h0);
      x.f = max(x.f, x.f0);
    }
  } else {
    x.h = gap ? min(x.e, x.h0) : 0;
    x.f = gap ? x.f0 : 0;
  }
  x.f = max(min(x.f, x.e), x.h);
  return x;
}

struct Sums {
  int back, more;
};

// A window of sequences, each with its plan and the pages of the sequences before it.
struct AssignShared {
  Plan plan[kAssignThreads];
  Sums before[kAssignThreads];
  Sums warp[kAssignThreads / 32];
};

// Window [base, base + kAssignThreads) by all threads, `carry` the sums before it;
// returns those behind it.
__device__ __forceinline__ Sums plan_window(const AssignArgs& p, AssignShared& sm, int base, Sums carry) {
  const int b = base + threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Sums mine = {0, 0};
  Plan x = {};
  if (b < p.B) {
    x = make_plan(p, b);
    mine = {x.back(), x.more()};
  }
  Sums incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl.back, off), v = __shfl_up_sync(0xffffffffu, incl.more, off);
    if (lane >= off) {
      incl.back += u;
      incl.more += v;
    }
  }
  __syncthreads();  // the window before is no longer read
  if (lane == 31) sm.warp[warp] = incl;
  sm.plan[threadIdx.x] = x;
  __syncthreads();
  Sums all = carry, upto = carry;
#pragma unroll 8
  for (int w = 0; w < kAssignThreads / 32; ++w) {
    const Sums s = sm.warp[w];
    if (w < warp) {
      upto.back += s.back;
      upto.more += s.more;
    }
    all.back += s.back;
    all.more += s.more;
  }
  sm.before[threadIdx.x] = {upto.back + incl.back - mine.back, upto.more + incl.more - mine.more};
  __syncthreads();
  return all;
}

// One token's slot.
__device__ __forceinline__ int64_t slot_of(const AssignArgs& p, int b, int t, const Lens& l) {
  const int pos = l.len - l.n + t;
  if (t >= l.n || pos < 0) return -1;
  const int id = p.table[static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift)];
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) return -1;
  return (static_cast<int64_t>(id) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

__global__ void __launch_bounds__(kAssignThreads, 1) fa_page_assign_kernel(const AssignArgs p, int ranks) {
  __shared__ AssignShared sm;
  grid_wait_prior();
  grid_release_next();
  const int rank = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int count = in_range(p, p.free_count[0], 0, p.num_pages);
  const bool one = p.B <= kAssignThreads;  // the only window stays in shared memory
  Sums all = {0, 0};
  auto meet = [&] {
    if (ranks > 1) {
      __syncwarp();
      cluster_barrier();
    } else {
      __syncthreads();
    }
  };
  // f(b, plan, before, i0, step): sequence b's work i0, i0 + step, ... by one warp, or by several
  // where there are more warps than sequences; the sums are those of all sequences
  auto sweep = [&](bool planned, bool replaces, const auto& f) {
    Sums carry = {0, 0};
    for (int base = 0; base < p.B; base += kAssignThreads) {
      if (!planned) carry = plan_window(p, sm, base, carry);
      if (!planned && replaces) meet();  // every CTA has read this window's states
      const int n = min(kAssignThreads, p.B - base);
      const int warps = ranks * (kAssignThreads / 32), w = rank + ranks * warp;
      const int per = max(walk_log2(warps) - walk_log2(2 * n - 1), 0);  // warps of a sequence: 2^per
      for (int i = w >> per; i < n; i += warps >> per)
        f(base + i, sm.plan[i], sm.before[i], 32 * (w & ((1 << per) - 1)) + lane, 32 << per);
    }
    if (!planned) all = carry;
  };
  // pages given back, to the stack
  sweep(false, false, [&](int b, const Plan& x, const Sums& before, int i0, int step) {
    int* row = p.table + static_cast<int64_t>(b) * p.max_pages;
    const int n = x.back();
    for (int i = i0; i < n; i += step) {
      const int pg = x.back_page(i), id = row[pg];
      const int64_t at = static_cast<int64_t>(count) + before.back + i;
      const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages);
      if (at < p.num_pages) p.free_pages[at] = good ? id : -1;
      if (!good || at >= p.num_pages) atomicOr(p.status, kStatusBadIndex);
      row[pg] = -1;
    }
  });
  const int total = static_cast<int>(min(static_cast<int64_t>(count) + all.back, static_cast<int64_t>(p.num_pages)));
  meet();
  // pages wanted, from its top
  sweep(one, false, [&](int b, const Plan& x, const Sums& before, int i0, int step) {
    int* row = p.table + static_cast<int64_t>(b) * p.max_pages;
    const int n = x.more();
    for (int i = i0; i < n; i += step) {
      const int at = total - 1 - (before.more + i);
      row[x.more_page(i)] = at >= 0 ? p.free_pages[at] : -1;
    }
  });
  meet();
  // what each sequence holds now, and the slots
  sweep(one, true, [&](int b, const Plan& x, const Sums& before, int i0, int step) {
    const int more = x.more(), want = x.h + x.e - x.f;
    const int got = want - more + min(more, max(0, total - before.more));
    if (p.slots_here) {
      const Lens l = lens_of(p, b);
      for (int t = i0; t < p.T; t += step) p.slots[static_cast<int64_t>(b) * p.T + t] = slot_of(p, b, t, l);
    }
    if (i0 < 3) {
      const int h = min(x.h, got), end = got > h ? x.f + got - h : h;
      const int f = got < want ? min(x.f, end) : x.f, e = got < want ? end : x.e;
      p.held[3 * b + i0] = i0 == 0 ? h : i0 == 1 ? f : e;
    }
  });
  if (rank == 0 && threadIdx.x == 0) {
    p.free_count[0] = max(total - all.more, 0);
    p.free_count[1] = max(all.more - total, 0);
  }
}

// Slots of many tokens: a block writes adjacent ones, each thread every 256th.
constexpr int kSlotThreads = 256, kSlotsEach = 8;
__global__ void __launch_bounds__(kSlotThreads) fa_page_slots_kernel(const AssignArgs p, int per_seq) {
  grid_wait_prior();
  grid_release_next();
  const int b = blockIdx.x / per_seq;
  const Lens l = lens_of(p, b);
  const int t0 = (blockIdx.x - b * per_seq) * kSlotThreads * kSlotsEach + threadIdx.x;
  int64_t slot[kSlotsEach];
#pragma unroll
  for (int i = 0; i < kSlotsEach; ++i) slot[i] = slot_of(p, b, t0 + i * kSlotThreads, l);  // (-1 behind the last token)
#pragma unroll
  for (int i = 0; i < kSlotsEach; ++i)
    if (t0 + i * kSlotThreads < p.T) p.slots[static_cast<int64_t>(b) * p.T + t0 + i * kSlotThreads] = slot[i];
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" fa_status fa_page_assign(int* page_table, const int* kv_lens, int* held, int* free_pages, int* free_count,
                                    int B, int num_pages, int page_size, int max_pages, int T, const int* new_lens,
                                    int window, int sinks, int64_t* slots, cudaStream_t stream) {
  const int ps = page_size;
  if (B < 1 || B > 65536 || num_pages < 1 || num_pages > (1 << 30) || max_pages < 1 || T < 1 || T > (1 << 22))
    return FA_ERR_INVALID_ARG;
  if (!(ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256)) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * ps > (1 << 30) || static_cast<int64_t>(B) * max_pages > INT32_MAX ||
      static_cast<int64_t>(B) * T > INT32_MAX)
    return FA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!page_table || !kv_lens || !held || !free_pages || !free_count) return FA_ERR_INVALID_ARG;
  const void* words[6] = {page_table, kv_lens, held, free_pages, free_count, new_lens};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return FA_ERR_MISALIGNED;
  // the first five are written
  const void* at[7] = {page_table, held, free_pages, free_count, slots, kv_lens, new_lens};
  const size_t n = static_cast<size_t>(B) * 4;
  const size_t bytes[7] = {n * max_pages, 3 * n, static_cast<size_t>(num_pages) * 4, 8, 2 * n * T, n, n};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (at[i] && at[j] && overlap(at[i], bytes[i], at[j], bytes[j])) return FA_ERR_INVALID_ARG;
  WaitCfg wc;
  if (!launch_waits(&wc)) return FA_ERR_LAUNCH;
  AssignArgs p;
  p.table = page_table; p.held = held; p.free_pages = free_pages; p.free_count = free_count;
  p.lens = kv_lens; p.new_lens = new_lens;
  p.slots = slots;
  p.B = B; p.num_pages = num_pages; p.max_pages = max_pages; p.T = T;
  p.page_shift = 0;
  while ((1 << p.page_shift) < ps) ++p.page_shift;
  p.window = std::min(window, 1 << 30);
  p.sinks = std::min(sinks, 1 << 30);
  p.status = wc.status;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  p.slots_here = slots && tokens <= kSlotsHere;
  const int ranks = B <= kLoneB && tokens <= kLoneTokens ? 1 : 8;
  cudaError_t e = launch_kernel(fa_page_assign_kernel, ranks, kAssignThreads, 0, stream, static_cast<unsigned>(ranks), p, ranks);
  if (e == cudaSuccess && slots && !p.slots_here) {
    const int per_seq = (T + kSlotThreads * kSlotsEach - 1) / (kSlotThreads * kSlotsEach);
    e = launch_kernel(fa_page_slots_kernel, static_cast<int64_t>(B) * per_seq, kSlotThreads, 0, stream, 1, p, per_seq);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}
