// Host-side launch interface between the C ABI of the paged cache
// (fa_paged_api.cu) and its kernels' units. Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include "fa_paged.cuh"

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
  int Hq, Tq, causal, window;
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
cudaError_t launch_paged_fwd(const PagedFwdLaunch& a);
cudaError_t launch_page_select(const SelectLaunch& a);

}  // namespace fa
