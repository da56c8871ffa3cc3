// C ABI of the paged cache: argument checks and launch set-up. As in fa_api.cu,
// everything the host can see is checked before anything is launched; what
// lives on the device (page table, lengths, selections) the kernels check.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_launch.h"
#include "fa_paged_launch.h"

using namespace fa;

namespace {

constexpr int kMaxTokens = 1 << 22;
constexpr int64_t kMaxUnits = 1 << 24;     // B * heads
constexpr int64_t kMaxPool = 1 << 30;      // num_pages * Hkv, and positions of a sequence
constexpr int kMaxSelected = 1 << 20;
constexpr int kMaxHeads = 1 << 14;         // of one token of fa_kv_append

fa_status check_cache(const fa_paged_kv* kv, bool need_bounds) {
  if (!kv) return FA_ERR_INVALID_ARG;
  if (kv->B < 1 || kv->Hkv < 1 || kv->num_pages < 1 || kv->max_pages < 1) return FA_ERR_INVALID_ARG;
  const int ps = kv->page_size;
  if (!(ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256)) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kv->B) * kv->Hkv > kMaxUnits) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kv->num_pages) * kv->Hkv > kMaxPool) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kv->max_pages) * ps > kMaxPool) return FA_ERR_INVALID_ARG;
  const int D = kv->D;
  if (!(D == 64 || D == 96 || D == 128 || D == 256)) return FA_ERR_UNSUPPORTED_HEAD_DIM;
  if (kv->dt != FA_FP16 && kv->dt != FA_BF16) return FA_ERR_UNSUPPORTED_DTYPE;
  if (!kv->k || !kv->v || !kv->page_table || !kv->kv_lens) return FA_ERR_INVALID_ARG;
  if (need_bounds && !kv->k_bounds) return FA_ERR_INVALID_ARG;
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->k_bounds)) return FA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(kv->page_table) | reinterpret_cast<uintptr_t>(kv->kv_lens)) & 3u)
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

size_t pool_bytes(const fa_paged_kv* kv) {
  return static_cast<size_t>(kv->num_pages) * kv->Hkv * kv->page_size * kv->D * 2;
}
size_t bounds_bytes(const fa_paged_kv* kv) {
  return kv->k_bounds ? static_cast<size_t>(kv->num_pages) * kv->Hkv * 2 * kv->D * 2 : 0;
}
size_t table_bytes(const fa_paged_kv* kv) { return static_cast<size_t>(kv->B) * kv->max_pages * 4; }

// Byte ranges of a call, with the rule that an output meets nothing else.
struct Ranges {
  const void* p[16];
  size_t n[16];
  int count = 0, outs = 0;
  void out(const void* q, size_t bytes) { add(q, bytes), outs = count; }
  void in(const void* q, size_t bytes) { add(q, bytes); }
  void add(const void* q, size_t bytes) {
    if (!q || bytes == 0) return;
    p[count] = q;
    n[count++] = bytes;
  }
  bool clash() const {
    for (int i = 0; i < outs; ++i)
      for (int j = i + 1; j < count; ++j)
        if (overlap(p[i], n[i], p[j], n[j])) return true;
    return false;
  }
};

PagedView make_view(const fa_paged_kv* kv, uint32_t* status) {
  PagedView c;
  c.k = static_cast<uint16_t*>(kv->k);
  c.v = static_cast<uint16_t*>(kv->v);
  c.bounds = static_cast<uint16_t*>(kv->k_bounds);
  c.table = kv->page_table;
  c.lens = kv->kv_lens;
  c.B = kv->B; c.Hkv = kv->Hkv; c.D = kv->D;
  c.num_pages = kv->num_pages; c.max_pages = kv->max_pages;
  c.page_shift = 0;
  while ((1 << c.page_shift) < kv->page_size) ++c.page_shift;
  c.status = status;
  return c;
}

// Strides of a [B, H, T, D] view: whole 16-byte chunks, not negative, at most 2^38
// elements (so the extent in bytes stays in 64 bits). Returns the elements from the
// first to behind the last one read, or -1.
int64_t view_extent(const int64_t* s, int64_t B, int64_t H, int64_t T, int64_t D) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] % 8 != 0 || s[i] > (int64_t(1) << 38)) return -1;
  return (B - 1) * s[0] + (H - 1) * s[1] + (T - 1) * s[2] + D;
}

}  // namespace

extern "C" {

fa_status fa_kv_append(const fa_paged_kv* kv, const void* k_new, const int64_t* k_strides,
                       const void* v_new, const int64_t* v_strides, const void* q,
                       const int64_t* q_strides, void* q_out, int Hq, int T, const int* new_lens,
                       const float* cos_table, const float* sin_table, int rope_len, int rot_dim,
                       int interleaved, cudaStream_t stream) {
  fa_status st = check_cache(kv, false);
  if (st != FA_OK) return st;
  if (T < 1 || T > kMaxTokens || static_cast<int64_t>(kv->B) * T > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (!k_new || !v_new || !k_strides || !v_strides) return FA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (q && (!q_strides || Hq < 1 || Hq % kv->Hkv != 0 || static_cast<int64_t>(kv->B) * Hq > kMaxUnits ||
            Hq > kMaxHeads))
    return FA_ERR_INVALID_ARG;
  if (kv->Hkv > kMaxHeads) return FA_ERR_INVALID_ARG;
  if ((cos_table == nullptr) != (sin_table == nullptr)) return FA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (cos_table ? (rot_dim < 16 || rot_dim > kv->D || rot_dim % 16 != 0 || rope_len < 1) : rot_dim != 0)
    return FA_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(q) || !aligned16(q_out) ||
      !aligned16(cos_table) || !aligned16(sin_table) || misaligned4(new_lens))
    return FA_ERR_MISALIGNED;
  const int64_t nk = view_extent(k_strides, kv->B, kv->Hkv, T, kv->D);
  const int64_t nv = view_extent(v_strides, kv->B, kv->Hkv, T, kv->D);
  const int64_t nq = q ? view_extent(q_strides, kv->B, Hq, T, kv->D) : 0;
  if (nk < 0 || nv < 0 || nq < 0) return FA_ERR_INVALID_ARG;
  const size_t angles = static_cast<size_t>(rope_len > 0 ? rope_len : 0) * (rot_dim / 2) * 4;
  Ranges r;
  r.out(kv->k, pool_bytes(kv));
  r.out(kv->v, pool_bytes(kv));
  r.out(kv->k_bounds, bounds_bytes(kv));
  if (q) r.out(q_out, static_cast<size_t>(kv->B) * Hq * T * kv->D * 2);
  r.in(k_new, static_cast<size_t>(nk) * 2);
  r.in(v_new, static_cast<size_t>(nv) * 2);
  r.in(q, static_cast<size_t>(nq) * 2);
  r.in(cos_table, angles);
  r.in(sin_table, angles);
  r.in(kv->page_table, table_bytes(kv));
  r.in(kv->kv_lens, static_cast<size_t>(kv->B) * 4);
  r.in(new_lens, static_cast<size_t>(kv->B) * 4);
  if (r.clash()) return FA_ERR_INVALID_ARG;
  WaitCfg wc;
  if (!launch_waits(&wc)) return FA_ERR_LAUNCH;
  AppendLaunch a;
  a.c = make_view(kv, wc.status);
  a.k = static_cast<const uint16_t*>(k_new);
  a.v = static_cast<const uint16_t*>(v_new);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.ks = {k_strides[0], k_strides[1], k_strides[2]};
  a.vs = {v_strides[0], v_strides[1], v_strides[2]};
  a.qs = {0, 0, 0};
  if (q) a.qs = {q_strides[0], q_strides[1], q_strides[2]};
  a.Hq = q ? Hq : 0;
  a.T = T;
  a.new_lens = new_lens;
  a.cos_table = cos_table;
  a.sin_table = sin_table;
  a.rope_len = rope_len;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.bf16 = kv->dt == FA_BF16;
  a.stream = stream;
  return launch_kv_append(a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_paged_workspace_size(int Hq, int Hkv, int Tq, int D) {
  if (Hq < 1 || Hq > kMaxUnits || Hkv < 1 || Hq % Hkv != 0 || Tq < 1 || Tq > kDecodeMaxTq) return 0;
  if (!(D == 64 || D == 96 || D == 128 || D == 256)) return 0;
  return paged_fwd_workspace(Hq / Hkv * Tq, D);
}

fa_status fa_paged_fwd(const fa_paged_kv* kv, const void* q, void* o, float* lse, int Hq, int Tq,
                       float scale, int causal, int window, const int* new_lens, const int* sel,
                       const int* sel_lens, int n_sel, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  fa_status st = check_cache(kv, false);
  if (st != FA_OK) return st;
  if (Tq < 1 || Tq > kDecodeMaxTq || Hq < 1 || Hq % kv->Hkv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kv->B) * Hq > kMaxUnits) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0) return FA_ERR_INVALID_ARG;
  if (!q || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
  if ((sel == nullptr) != (sel_lens == nullptr)) return FA_ERR_INVALID_ARG;
  if (sel && (n_sel < 1 || n_sel > kMaxSelected)) return FA_ERR_INVALID_ARG;
  // tiles are counted in 32 bits
  const int block = paged_block_rows(Hq / kv->Hkv * Tq, kv->D);
  const int64_t all_units = static_cast<int64_t>(kv->B) * kv->Hkv * ((Hq / kv->Hkv * Tq + block - 1) / block);
  if (paged_tiles(all_units, static_cast<int64_t>(sel ? n_sel : kv->max_pages) * kv->page_size) > INT32_MAX)
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_paged_workspace_size(Hq, kv->Hkv, Tq, kv->D);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned16(workspace) ||
      misaligned4(new_lens) || misaligned4(sel) || misaligned4(sel_lens))
    return FA_ERR_MISALIGNED;
  const size_t rows = static_cast<size_t>(kv->B) * Hq * Tq;
  const size_t units = static_cast<size_t>(kv->B) * kv->Hkv;
  Ranges r;
  r.out(o, rows * kv->D * 2);
  r.out(lse, rows * 4);
  r.out(workspace, workspace_bytes);
  r.in(q, rows * kv->D * 2);
  r.in(kv->k, pool_bytes(kv));
  r.in(kv->v, pool_bytes(kv));
  r.in(kv->k_bounds, bounds_bytes(kv));
  r.in(kv->page_table, table_bytes(kv));
  r.in(kv->kv_lens, static_cast<size_t>(kv->B) * 4);
  r.in(new_lens, static_cast<size_t>(kv->B) * 4);
  r.in(sel, units * (sel ? n_sel : 0) * 4);
  r.in(sel_lens, units * 4);
  if (r.clash()) return FA_ERR_INVALID_ARG;
  PagedFwdLaunch a;
  if (!launch_waits(&a.wc)) return FA_ERR_LAUNCH;
  a.c = make_view(kv, a.wc.status);
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.Hq = Hq; a.Tq = Tq; a.causal = causal; a.window = window;
  a.scale_log2 = scale * kLog2e;
  a.new_lens = new_lens;
  a.sel = sel; a.sel_lens = sel_lens; a.n_sel = n_sel;
  a.ws = static_cast<float*>(workspace);
  a.bf16 = kv->dt == FA_BF16;
  a.stream = stream;
  cudaError_t e;
  switch (kv->D) {
    case 64: e = launch_paged_fwd_d64(a); break;
    case 96: e = launch_paged_fwd_d96(a); break;
    case 128: e = launch_paged_fwd_d128(a); break;
    default: e = launch_paged_fwd_d256(a); break;
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_page_select_workspace_size(int B, int Hkv, int max_pages) {
  if (B < 1 || Hkv < 1 || max_pages < 1 || max_pages > kMaxPool || static_cast<int64_t>(B) * Hkv > kMaxUnits) return 0;
  const size_t bytes = static_cast<size_t>(B) * Hkv * max_pages * 12;  // scores in 32 and in 64 bits
  return (bytes + 255) / 256 * 256;
}

fa_status fa_page_select(const fa_paged_kv* kv, const void* q, int Hq, int n_sel, int keep_first,
                         int keep_last, int* sel, int* sel_lens, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
  fa_status st = check_cache(kv, true);
  if (st != FA_OK) return st;
  if (Hq < 1 || Hq % kv->Hkv != 0 || static_cast<int64_t>(kv->B) * Hq > kMaxUnits) return FA_ERR_INVALID_ARG;
  if (n_sel < 1 || n_sel > kMaxSelected || keep_first < 0 || keep_last < 0 ||
      static_cast<int64_t>(keep_first) + keep_last > n_sel)
    return FA_ERR_INVALID_ARG;
  if (!q || !sel || !sel_lens || !workspace) return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_page_select_workspace_size(kv->B, kv->Hkv, kv->max_pages))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(workspace) || misaligned4(sel) || misaligned4(sel_lens))
    return FA_ERR_MISALIGNED;
  const size_t units = static_cast<size_t>(kv->B) * kv->Hkv;
  Ranges r;
  r.out(sel, units * n_sel * 4);
  r.out(sel_lens, units * 4);
  r.out(workspace, workspace_bytes);
  r.in(q, static_cast<size_t>(kv->B) * Hq * kv->D * 2);
  r.in(kv->k_bounds, bounds_bytes(kv));
  r.in(kv->k, pool_bytes(kv));
  r.in(kv->v, pool_bytes(kv));
  r.in(kv->page_table, table_bytes(kv));
  r.in(kv->kv_lens, static_cast<size_t>(kv->B) * 4);
  if (r.clash()) return FA_ERR_INVALID_ARG;
  WaitCfg wc;
  if (!launch_waits(&wc)) return FA_ERR_LAUNCH;
  SelectLaunch a;
  a.c = make_view(kv, wc.status);
  a.q = static_cast<const uint16_t*>(q);
  a.Hq = Hq; a.n_sel = n_sel; a.keep_first = keep_first; a.keep_last = keep_last;
  a.sel = sel; a.sel_lens = sel_lens;
  a.ws = workspace;
  a.bf16 = kv->dt == FA_BF16;
  a.stream = stream;
  return launch_page_select(a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
