// Host-side launch interface between the C ABI of the paged cache
// (fa_paged_api.cu) and its kernels' units. Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include "fa_paged.cuh"
#include "fa_paged_walk.h"

namespace fa {

// Strides in elements of the batch, head and token index.
struct TokenStrides {
  int64_t b, h, t;
};

struct AppendLaunch {
  PagedView c;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  TokenStrides ks, vs, qs;
  int Hq, T;
  const int* new_lens;
  const float *cos_table, *sin_table;
  int rope_len, rot_dim, interleaved;
  bool bf16;
  cudaStream_t stream;
};

struct PagedFwdLaunch {
  PagedView c;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  int Hq, Tq, causal, window, sinks;
  float scale_log2;
  const int* new_lens;
  const int *sel, *sel_lens;
  int n_sel;
  float* ws;
  WaitCfg wc;
  bool bf16;
  cudaStream_t stream;
};

struct SelectLaunch {
  PagedView c;
  const uint16_t* q;
  int Hq, n_sel, keep_first, keep_last;
  int *sel, *sel_lens;
  void* ws;
  bool bf16;
  cudaStream_t stream;
};

cudaError_t launch_kv_append(const AppendLaunch& a);
cudaError_t launch_kv_append8(const AppendLaunch& a);  // the cache has scales
cudaError_t launch_paged_fwd_d64(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_d96(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_d128(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_d256(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_window_d64(const PagedFwdLaunch& a);  // with a window
cudaError_t launch_paged_fwd_window_d96(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_window_d128(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_window_d256(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_sinks_d64(const PagedFwdLaunch& a);  // and first keys beside it
cudaError_t launch_paged_fwd_sinks_d96(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_sinks_d128(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd_sinks_d256(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd8_d64(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd8_d96(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd8_d128(const PagedFwdLaunch& a);
cudaError_t launch_paged_fwd8_d256(const PagedFwdLaunch& a);

// Query rows of a block where a cluster takes a unit: 8 (usual decoding), 16, 32, 48
// or 64 where a KV head has more, so that its keys are loaded once for all of them
// (D = 256: at most 32, what registers hold).
inline int paged_block_rows(int rows, int D) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || D == 256 ? 32 : rows <= 48 ? 48 : 64;
}
// The same where the list is split: above 16 rows by tcgen05, up to 128.
inline int paged_split_rows(int rows) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

// CTAs of a split list at most: they leave parts of units to be joined.
__host__ __device__ constexpr int paged_max_parts(int block_rows) { return block_rows <= 16 ? 608 : 192; }

// Device workspace of launch_paged_fwd_d* in bytes: per CTA two parts of a
// block (fp32 rows, maximum and sum) and a record of what is to be joined.
inline size_t paged_fwd_workspace(int rows, int D) {
  const int block = paged_split_rows(rows), parts = paged_max_parts(block);
  const size_t bytes = static_cast<size_t>(2 * parts) * block * (D * 4 + 8) + parts * 8;
  return (bytes + 255) / 256 * 256;
}
cudaError_t launch_page_select(const SelectLaunch& a);

}  // namespace fa
