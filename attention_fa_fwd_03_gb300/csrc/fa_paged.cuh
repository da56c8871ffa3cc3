// Shared definitions of the paged-cache kernels (fa_kv_append, fa_paged_fwd,
// fa_page_select): the device view of the cache and the checks of everything
// that only the device can see. The pages of the sources describe training
// only; these kernels serve, with the forward's mathematics.
#pragma once

#include <cstdint>

#include "fa_common.cuh"

namespace fa {

// The kernels start before the one ahead of them in the stream has ended
// (programmatic serialisation) and may read what it writes: the lengths, the rotated
// queries, the selection, the bounds. So they read global memory by ordinary loads
// behind grid_wait_prior(): the read-only path (__ldg) is for memory that nobody writes
// while the kernel runs, and its loads may be moved above the wait.

// Bit of the device status word beside those of sm103_ptx.cuh: a page, length,
// position or selected page out of range. The access is skipped.
constexpr uint32_t kStatusBadIndex = 4u;

struct PagedView {
  uint16_t* k;       // [num_pages, Hkv, page, D], 16-bit values (with scales: e4m3)
  uint16_t* v;
  uint16_t* bounds;  // [num_pages, Hkv, 2, D] or null
  float *k_scales, *v_scales;  // [num_pages, Hkv], or null where the cache holds 16-bit values
  const int* table;  // [B, max_pages]
  const int* lens;   // [B]
  int B, Hkv, D, num_pages, page_shift, max_pages;
  uint32_t* status;
};

__device__ __forceinline__ void flag_bad_index(const PagedView& c) {
  atomicOr(c.status, kStatusBadIndex);
}

// A count that has to be in [0, most], clamped to it.
__device__ __forceinline__ int checked_count(const PagedView& c, int n, int most) {
  if (static_cast<unsigned>(n) <= static_cast<unsigned>(most)) return n;
  flag_bad_index(c);
  return n < 0 ? 0 : most;
}

// Keys of sequence b (new ones included) and new tokens among the call's T rows,
// loaded together: callers wait for both once.
struct SeqLens {
  int len, n;
};
__device__ __forceinline__ SeqLens seq_lens(const PagedView& c, const int* new_lens, int b, int T) {
  const int len = c.lens[b], n = new_lens ? new_lens[b] : T;
  return {checked_count(c, len, c.max_pages << c.page_shift), checked_count(c, n, T)};
}

// A pool page, or -1 where the table holds none.
__device__ __forceinline__ int checked_page(const PagedView& c, int id) {
  if (static_cast<unsigned>(id) < static_cast<unsigned>(c.num_pages)) return id;
  flag_bad_index(c);
  return -1;
}

// Pool page of page `p` of sequence b (0 <= p < max_pages), or -1.
__device__ __forceinline__ int pool_page(const PagedView& c, int b, int p) {
  return checked_page(c, c.table[static_cast<int64_t>(b) * c.max_pages + p]);
}

// First element of row `slot` of KV head g in pool page `id`.
__device__ __forceinline__ int64_t pool_row(const PagedView& c, int id, int g, int slot) {
  return ((((static_cast<int64_t>(id) * c.Hkv + g) << c.page_shift) + slot)) * c.D;
}

}  // namespace fa
