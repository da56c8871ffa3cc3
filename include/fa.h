/*
 * fa.h — exact scaled-dot-product attention on sm_103a (GB300), for training and
 * for serving from a paged key/value cache.
 *
 * C ABI of libfa_gb300.so: a forward pass that caches the per-row log-sum-exp
 * (LSE), and its vector-Jacobian product (VJP) split into a D-vector
 * preprocess, a dK/dV kernel and a dQ kernel that recompute P per tile from
 * the cached LSE; and, further down, the calls of the paged cache.
 *
 * The operation (page "mlx-bun 0.0.4: package/src/model/flash-attention.ts",
 * forward shader and backward passes 1-3; page "[Metal] Add Flash Attention
 * VJP for training", Implementation Notes):
 *
 *   S[i,j] = scale * Q[b,h,i,:] . K[b,g,j,:]          g = h / (Hq / Hkv)
 *   a key j is hidden from query i when
 *       (causal && j > i)  or  (window > 0 && i >= j && i - j >= window)
 *   LSE[i] = ln sum_{j visible} exp(S[i,j]);   P[i,j] = exp(S[i,j] - LSE[i])
 *   O[i,:] = sum_j P[i,j] V[b,g,j,:]
 *   D[i]   = sum_d dO[i,d] O[i,d]
 *   dS     = P o (dO V^T - D)
 *   dQ = scale * dS K;  dK = scale * sum_{h in group} dS^T Q;  dV = sum_{h in group} P^T dO
 *
 * Conventions shared by every entry point:
 *  - Q, O, dO, dQ are [B, Hq, Tq, D]; K, V, dK, dV are [B, Hkv, Tkv, D];
 *    LSE is [B, Hq, Tq]. All are dense row-major (innermost index last) device
 *    buffers in HBM, owned by the caller, 16-byte aligned.
 *  - Element type: fp16 or bf16 (fa_dtype) for Q, K, V, O, dO, dQ, dK, dV;
 *    LSE is fp32 in natural log. Arithmetic: fp32 accumulation on the tensor
 *    cores, fp32 softmax statistics, round-to-nearest-even on every store.
 *  - Grouped-query attention: Hq must be a multiple of Hkv; consecutive query
 *    heads share a KV head (g = h / (Hq / Hkv)).
 *  - causal is 0 or 1; with Tq != Tkv the causal mask is aligned at the top
 *    left (query i sees keys 0..i), as in page "R/ag_flash_attn.R" (ggmlR),
 *    mask builder. window >= 0 (0 = no window): the window hides only past
 *    keys, so a query sees `window` keys of its past including its own
 *    position; without causal, future keys stay visible.
 *  - A query row that sees no key at all (only possible with a window and
 *    Tq > Tkv) gets O = 0, LSE = -inf, dQ = 0 and adds nothing to dK/dV.
 *  - head_dim D is one of 64, 96, 128, 256. scale must be finite and > 0.
 *  - Outputs are fully overwritten; the caller need not zero them. Outputs
 *    must not overlap inputs or each other.
 *  - The library never allocates or frees memory. Calls are asynchronous on
 *    `stream` (0 = the legacy default stream); results are ready when the
 *    stream reaches the point after the call.
 *  - Arguments are validated before anything is launched; a bad argument
 *    returns an error code and launches nothing. A launch failure returns
 *    FA_ERR_LAUNCH. Errors never abort the process.
 *  - Every wait inside the kernels is bounded (default 4 s, environment
 *    variable FA_WAIT_TIMEOUT_MS overrides). A wait that gives up sets a bit
 *    in a device status word, the kernel runs to its exit without further
 *    waiting, and fa_device_status() reports FA_ERR_TIMEOUT.
 */
#ifndef FA_GB300_H_
#define FA_GB300_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,          /* null pointer, bad size, overlap, bad scale/mask */
  FA_ERR_UNSUPPORTED_HEAD_DIM = 2, /* D not in {64, 96, 128, 256} */
  FA_ERR_UNSUPPORTED_DTYPE = 3,    /* dtype not FA_FP16 / FA_BF16 */
  FA_ERR_MISALIGNED = 4,           /* a buffer is not 16-byte aligned */
  FA_ERR_LAUNCH = 5,               /* a CUDA launch or driver call failed */
  FA_ERR_TIMEOUT = 6,              /* a bounded device wait gave up */
  FA_ERR_BAD_INDEX = 7             /* a kernel met a page, length or position out of range */
} fa_status;

typedef enum { FA_FP16 = 0, FA_BF16 = 1 } fa_dtype;

/* Forward pass (page "mlx-bun 0.0.4: package/src/model/flash-attention.ts",
 * forward shader; online softmax that never materialises S).
 *   q [B,Hq,Tq,D], k/v [B,Hkv,Tkv,D]   inputs, dtype `dt`
 *   o [B,Hq,Tq,D]                      output, dtype `dt`
 *   lse [B,Hq,Tq]                      output, fp32 natural-log LSE (kept for fa_bwd)
 * Sizes: B, Hq, Hkv, Tq, Tkv >= 1; Tq, Tkv <= 2^22; B * Hq <= 2^24.
 * One kernel launch. Tq <= 8 (decode-shaped calls) runs a split-key kernel
 * that launches thread-block clusters of up to 8 CTAs; longer query blocks run
 * the tensor-core tile kernel. Both compute the same result; which one runs
 * changes only the rounding of the fp32 sums.
 * The kernel is launched with programmatic stream serialisation: its launch
 * and set-up overlap the end of the previous kernel in `stream`, and it
 * waits for that kernel to complete before it reads or writes global memory.
 * So stream order is what the caller sees.
 * Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                 int causal, int window, fa_dtype dt, cudaStream_t stream);

/* Bytes of device workspace fa_bwd needs: the fp32 D-vector [B,Hq,Tq]
 * rounded up to 256 bytes. Returns 0 for non-positive sizes. */
size_t fa_bwd_workspace_size(int B, int Hq, int Tq);

/* Backward pass / VJP (page "mlx-bun 0.0.4: package/src/model/
 * flash-attention.ts", backward passes 1-3; page "[Metal] Add Flash Attention
 * VJP for training", Implementation Notes: two kernels, KV-row ownership so
 * grouped heads reduce without atomics). Launches, in order on `stream`:
 *   1. D-vector preprocess  D = rowsum(dO o O)   (from the stored O)
 *   2. dK/dV kernel (one CTA, or a cluster of CTAs sharing the tiles, owns a
 *      block of KV rows and loops over every query head of its group and
 *      every query tile that can see it; Tq <= 8: a kernel that sums over
 *      every query row of the group in fp32 per key row, any mask)
 *   3. dQ kernel (one CTA owns a block of query rows, loops over KV tiles;
 *      Tq <= 8: a split-key kernel over thread-block clusters of up to 8 CTAs)
 * Which kernels run changes only the rounding order of the fp32 sums.
 * Ordering: as for fa_fwd, each kernel is launched to overlap the end of the
 * previous kernel in `stream` (programmatic stream serialisation). It waits
 * for that kernel before it reads or writes global memory, so stream order
 * holds for the caller. On causal, windowed and Tq <= 8 calls, the dQ kernel
 * starts without waiting for the dK/dV kernel: it needs only the D-vector.
 * It waits for dK/dV before it completes, so work queued after fa_bwd on
 * `stream` still sees all three outputs written.
 *   q, k, v, o, dO, lse       inputs (o and lse as written by fa_fwd)
 *   dq [B,Hq,Tq,D], dk/dv [B,Hkv,Tkv,D]  outputs, dtype `dt`
 *   workspace                 caller-owned device scratch of at least
 *                             fa_bwd_workspace_size(B,Hq,Tq) bytes, 16-byte
 *                             aligned; its contents are overwritten.
 * The gradient with respect to LSE is not an input: it is taken as zero.
 * Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv,
                 int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                 int causal, int window, fa_dtype dt, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream);

/* The three launches of fa_bwd as separate calls, for callers that schedule
 * them themselves (e.g. dK/dV and dQ on two streams once the D-vector is
 * ready) or time them one by one. `dvec` is the D-vector workspace:
 * [B,Hq,Tq] fp32, 16-byte aligned, at least fa_bwd_workspace_size bytes.
 * fa_bwd_preprocess (backward pass 1 of the mlx-bun flash-attention.ts page):
 *   dvec[i] = sum_d dO[i,d] O[i,d]   (fp32 accumulation of the stored O)
 * fa_bwd_dkv (backward pass 2): dk, dv from q, k, v, dO, lse, dvec.
 * fa_bwd_dq  (backward pass 3): dq from q, k, v, dO, lse, dvec.
 * Same argument rules and error behaviour as fa_bwd. */
fa_status fa_bwd_preprocess(const void* o, const void* dO, float* dvec, int B, int Hq, int Tq,
                            int D, fa_dtype dt, cudaStream_t stream);
fa_status fa_bwd_dkv(const void* q, const void* k, const void* v, const void* dO,
                     const float* lse, const float* dvec, void* dk, void* dv,
                     int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                     int causal, int window, fa_dtype dt, cudaStream_t stream);
fa_status fa_bwd_dq(const void* q, const void* k, const void* v, const void* dO,
                    const float* lse, const float* dvec, void* dq,
                    int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                    int causal, int window, fa_dtype dt, cudaStream_t stream);

/* fa_fwd and fa_bwd with first keys that the window does not hide: a key j is hidden from
 * query i when
 *     (causal && j > i)  or  (window > 0 && i >= j && i - j >= window && j >= sinks)
 * sinks >= 0; without a window it has no effect, and sinks = 0 is fa_fwd and fa_bwd.
 * Every other rule is theirs. The backward's workspace has
 * fa_bwd_sinks_workspace_size bytes (0 for sizes that it refuses): the D-vector and, where
 * the blocks of first keys, which every later query sees, are shared by several CTAs, the
 * fp32 sums of each, added in a fixed order by a last kernel. Calls that may overlap
 * need a workspace each. */
fa_status fa_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse,
                       int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                       int causal, int window, int sinks, fa_dtype dt, cudaStream_t stream);
size_t fa_bwd_sinks_workspace_size(int B, int Hq, int Hkv, int Tq, int Tkv, int D, int window, int sinks);
fa_status fa_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const void* dO,
                       const float* lse, void* dq, void* dk, void* dv,
                       int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                       int causal, int window, int sinks, fa_dtype dt, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/* fa_bwd without a workspace argument, for callers that cannot allocate any
 * device memory: a plug-in inside a host program that owns every device
 * allocation, or a loop that may not call the allocator (which can
 * synchronise the device) once it runs. The pages have no counterpart of
 * this call; it exists for such callers only.
 * The D-vector goes to a fixed 4 MiB array inside the library instead of a
 * caller buffer: B * Hq * Tq must not exceed fa_bwd_noalloc_max_rows()
 * (2^20), else FA_ERR_INVALID_ARG and nothing is launched. Every other
 * argument, layout and error rule is that of fa_bwd.
 * The array is one per device, shared by every call on that device and kept
 * until the process exits; it holds the last call's D-vector. Calls whose
 * launches overlap on the GPU (two streams, or two host threads) race on it:
 * keep them ordered on one stream. The first call on a device (with that
 * device current) looks up the array's device address, which is set-up work:
 * make that first call before any stream capture. The address belongs to the
 * device's CUDA context; after cudaDeviceReset() the next call finds a new
 * context and looks the address up again (so, after a reset, that call is
 * again a first call). Nothing in the array has to start at zero: each call
 * rewrites the part it uses before reading it. */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                         const void* dO, const float* lse, void* dq, void* dk, void* dv,
                         int B, int Hq, int Hkv, int Tq, int Tkv, int D, float scale,
                         int causal, int window, fa_dtype dt, cudaStream_t stream);

/* Largest B * Hq * Tq that fa_bwd_noalloc accepts. */
size_t fa_bwd_noalloc_max_rows(void);

/* ------------------------------------------------------------------------
 * Serving from a paged key/value cache. The pages of the sources describe
 * training only and have no counterpart of these calls; the operation inside
 * fa_paged_fwd is the forward above.
 *
 * The cache is a pool of pages: k and v are [num_pages, Hkv, page_size, D], so
 * one KV head's keys of a page are page_size consecutive rows. Sequence b
 * keeps key j in slot j % page_size of pool page page_table[b, j / page_size].
 * kv_lens[b] counts the keys of sequence b, the tokens of the current call
 * among them: with n_b new tokens (new_lens[b], or all T rows where new_lens
 * is null) token t < n_b has position kv_lens[b] - n_b + t. Rows t >= n_b of a
 * call are padding. One kv_lens array thus serves fa_kv_append and the
 * fa_paged_fwd that follows; the caller advances it between steps.
 *
 * k_bounds (may be null: then fa_kv_append keeps none and fa_page_select
 * refuses) is [num_pages, Hkv, 2, D]: the element-wise minimum and maximum of
 * the keys written to the page since its slot 0 was last written (a NaN is left
 * out where there is a number).
 *
 * page_table and kv_lens live on the device and are read by the kernels, so
 * calls can be captured into a graph and replayed with other lengths and
 * pages. Entries of page_table past a sequence's last page are not used. What
 * the host cannot check the kernels do: a page outside [0, num_pages), a length
 * outside [0, max_pages * page_size], a position outside the angle tables or a
 * new_lens[b] outside [0, T] raises a bit that fa_device_status() reports as
 * FA_ERR_BAD_INDEX. Lengths are clamped to their range; keys of a bad page are
 * neither written nor read (hidden from every query). These arrays must not be
 * written while a call that reads them runs (write them in the call's stream order);
 * the outputs of such a call are undefined, and it may report FA_ERR_TIMEOUT.
 *
 * Limits: B * Hkv <= 2^24, num_pages * Hkv <= 2^30, max_pages * page_size <= 2^30;
 * page_size is 16, 32, 64, 128 or 256. Pool offsets are 64-bit. */
typedef struct {
  void* k;               /* [num_pages, Hkv, page_size, D] */
  void* v;               /* [num_pages, Hkv, page_size, D] */
  void* k_bounds;        /* [num_pages, Hkv, 2, D] or null */
  const int* page_table; /* [B, max_pages] */
  const int* kv_lens;    /* [B] */
  int B, Hkv, D, num_pages, page_size, max_pages;
  fa_dtype dt;
} fa_paged_kv;

/* Append the keys and values of new tokens to the cache, rotating the keys by
 * their position on the way, and rotate the queries of the same tokens.
 *   k_new, v_new  [B, Hkv, T, D]; q [B, Hq, T, D] or null (then q_out is null
 *                 and Hq is not used). Each is read through its strides
 *                 (elements) of the batch, head and token index; the innermost
 *                 index is contiguous. Bases are 16-byte aligned and strides
 *                 multiples of 8 (at most 2^38), so slices of a fused projection
 *                 [B, T, (Hq + 2 Hkv) * D] are read in place.
 *   q_out         [B, Hq, T, D] dense; padding rows are set to zero.
 *   cos_table, sin_table  fp32 [rope_len, rot_dim / 2], row p for position p;
 *                 both null for no rotation (rot_dim = 0).
 * Dimensions i < rot_dim are rotated in pairs (i, i + rot_dim / 2), or, with
 * interleaved = 1, (2i, 2i + 1): (a, b) -> (a cos - b sin, b cos + a sin) in
 * fp32, rounded once; the rest is copied. rot_dim is a multiple of 16, at most
 * D. Token t of sequence b is written to its slot; nothing else of the pools is
 * touched. With k_bounds the bounds of every page that receives a token are
 * updated: started afresh where the page's slot 0 is among the new tokens, else
 * widened (so after tokens were taken back they may be wider than needed).
 * 1 <= T <= 2^22, B * T < 2^31, Hq and Hkv <= 2^14. Two sequences of one call
 * must not append to the same page, nor one sequence to a page that its table
 * holds twice.
 * One kernel launch. Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_kv_append(const fa_paged_kv* kv, const void* k_new, const int64_t* k_strides,
                       const void* v_new, const int64_t* v_strides, const void* q,
                       const int64_t* q_strides, void* q_out, int Hq, int T, const int* new_lens,
                       const float* cos_table, const float* sin_table, int rope_len, int rot_dim,
                       int interleaved, cudaStream_t stream);

/* Bytes of device workspace fa_paged_fwd needs for Hq query heads over Hkv KV
 * heads, Tq tokens per sequence and head dim D; independent of batch, lengths
 * and device. Returns 0 for sizes fa_paged_fwd refuses. */
size_t fa_paged_workspace_size(int Hq, int Hkv, int Tq, int D);

/* Attention of Tq <= 8 new tokens per sequence over the paged cache (the forward
 * of fa_fwd with keys and values read through the page table).
 *   q [B, Hq, Tq, D], o likewise, lse [B, Hq, Tq] fp32; dense.
 *   A key j < kv_lens[b] is hidden from the query at position p when
 *     (causal && j > p)  or  (window > 0 && p >= j && p - j >= window)
 *   so with causal = 1 the new tokens see the cache and each other causally
 *   (the mask is aligned at the end of the cache, not at the top left).
 *   sel, sel_lens  both null, or int32 [B, Hkv, n_sel] and [B, Hkv]: query heads
 *     of KV head g then see only the keys of the sequence's pages sel[b, g, 0 ..
 *     sel_lens[b, g] - 1] (page numbers within the sequence, distinct, any
 *     order). An entry outside the sequence's pages, or sel_lens outside
 *     [0, n_sel], is a bad index.
 * Limit: B * Hkv * ceil(rows / 64) * ceil(keys / 64) < 2^31, rows = (Hq / Hkv) * Tq
 * (D = 256: / 32), keys = max_pages * page_size, with sel n_sel * page_size; over a cache
 * of 8 bits with rows <= 16: B * Hkv * (ceil(keys / 64) + 2) < 2^31.
 * A row that sees no key (or whose every score is -inf), and every padding row,
 * gets O = 0 and LSE = -inf.
 * Scores are held in fp32 in units of ln 2: |scale q.k| above 2.3e38 counts as
 * infinite.
 * Values of keys that no row sees never reach a result, whatever they hold. A
 * key that is visible to one row and hidden from another adds exactly nothing to
 * the latter as well. A NaN in a row's query or in a key that the row sees makes
 * that row's O and LSE NaN; an infinite value of V that it sees makes O infinite or
 * NaN there.
 *   workspace  fa_paged_workspace_size bytes, 16-byte aligned; contents
 *     undefined before and after. Calls that may overlap need one each.
 * The result does not depend on what else runs and is the same on every run.
 * Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_paged_fwd(const fa_paged_kv* kv, const void* q, void* o, float* lse, int Hq, int Tq,
                       float scale, int causal, int window, const int* new_lens, const int* sel,
                       const int* sel_lens, int n_sel, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream);

/* fa_paged_fwd with first keys that the window does not hide: a key j is hidden
 * from the query at position p when
 *     (causal && j > p)  or  (window > 0 && p >= j && p - j >= window && j >= sinks)
 * sinks >= 0; without a window it has no effect. Only pages that hold a key which
 * the window or the first keys show are read (where no pages are selected), so the
 * table may hold -1 for the others, as where fa_page_assign has given them back.
 * sinks = 0 is fa_paged_fwd. */
fa_status fa_paged_fwd_sinks(const fa_paged_kv* kv, const void* q, void* o, float* lse, int Hq, int Tq,
                             float scale, int causal, int window, int sinks, const int* new_lens,
                             const int* sel, const int* sel_lens, int n_sel, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* The cache held in 8 bits: e4m3 (4 exponent and 3 mantissa bits, no infinities, largest
 * number 448). k and v are [num_pages, Hkv, page_size, D] bytes; k_scales and
 * v_scales are fp32 [num_pages, Hkv]: a held value stands for itself times its page's and
 * head's scale, a power of two from 2^-126 on. Everything else is as in fa_paged_kv. */
typedef struct {
  void* k;               /* [num_pages, Hkv, page_size, D] e4m3 */
  void* v;               /* [num_pages, Hkv, page_size, D] e4m3 */
  float* k_scales;       /* [num_pages, Hkv] */
  float* v_scales;       /* [num_pages, Hkv] */
  const int* page_table; /* [B, max_pages] */
  const int* kv_lens;    /* [B] */
  int B, Hkv, D, num_pages, page_size, max_pages;
} fa_paged_kv8;

/* fa_kv_append into a cache of 8 bits: new keys, values and queries of type dt. For each
 * page that receives tokens, KV head, and keys and values apart:
 *   s = the least power of two, 2^-126 or above, with |x| <= 448 s for every finite
 *       element x of the call's new rows in the page (of keys: rotated, in fp32),
 *   and at least the page's old scale unless the page's slot 0 is among the new rows.
 * New rows are held as x / s, rounded once; a NaN or an infinity is held as NaN. Where s is
 * more than the old scale, the page's rows below the first new one are held anew, their
 * values as before but for those below 2^-6 s, which are rounded to multiples of 2^-9 s.
 * Nothing else of the pools and scales is touched. Argument rules of fa_kv_append. */
fa_status fa_kv_append8(const fa_paged_kv8* kv, const void* k_new, const int64_t* k_strides,
                        const void* v_new, const int64_t* v_strides, const void* q,
                        const int64_t* q_strides, void* q_out, int Hq, int T, const int* new_lens,
                        const float* cos_table, const float* sin_table, int rope_len, int rot_dim,
                        int interleaved, fa_dtype dt, cudaStream_t stream);

/* fa_paged_fwd_sinks over a cache of 8 bits: q and o of type dt; keys and values are the
 * numbers that the cache stands for. Weights p of the values are rounded to fp16 numbers for
 * bf16 outputs, so that O is off by up to 2^-11 sum p |v| / sum p beside its own rounding, and
 * held to 2^-22 of themselves for fp16 outputs; and each key's p v is off by up to 2^-32 of the
 * row's largest p times 448 times its sequence's largest scale of values. Workspace and rules of fa_paged_fwd; a scale that
 * fa_kv_append8 would not write (0, negative, no power of two, infinite or NaN) gives
 * undefined rows. */
fa_status fa_paged_fwd8(const fa_paged_kv8* kv, const void* q, void* o, float* lse, int Hq, int Tq,
                        float scale, int causal, int window, int sinks, const int* new_lens,
                        const int* sel, const int* sel_lens, int n_sel, fa_dtype dt, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);

/* Page tables of a batch from its lengths: the step's new tokens get pool pages, and pages
 * that no query of this step or a later one sees go back to the pool.
 *   page_table [B, max_pages], written: entries that get a page, and -1 where one is
 *     given back or none was left; others keep what they hold.
 *   kv_lens [B]: keys of each sequence, the step's new tokens (new_lens[b], or T) among them.
 *   held [B, 3]: per sequence (head, first, end): it holds a pool page for its pages
 *     [0, head) and [first, end), 0 <= head <= first <= end <= max_pages. Kept from
 *     call to call; zeros for a sequence that holds none.
 *   free_pages [num_pages], free_count [2]: a stack of the free pool pages, the first
 *     free_count[0] entries. free_count[1] is written: how many pages were wanted and
 *     not there.
 *   slots [B, T] int64 or null: for each new token the place of its row among those of the
 *     pool seen as [num_pages * page_size] rows, page_table entry * page_size + slot, or -1
 *     for padding and where there is no page.
 * A sequence wants its pages [0, end), end = ceil(kv_lens / page_size); with a window only
 * those of the first `sinks` keys and those from the page of the first key on that the
 * window shows to its first new token (position kv_lens - n), max(0, kv_lens - n - window + 1).
 * What was given back does not come again (while held has a gap between head and
 * first, neither grows into it). Pages held but not wanted are pushed to the stack,
 * sequence by sequence in ascending order; then wanted pages not held are popped from
 * it in the same order. Where it runs out the rest get none: those sequences hold the
 * lowest of what they want, and ask again in the next call.
 * To end a sequence give it kv_lens[b] = 0 for one call, which returns all its pages.
 * Lengths, counts and states out of range raise FA_ERR_BAD_INDEX's bit and are clamped; so
 * does a table entry given back that is no pool page, which goes to the stack as -1.
 * B <= 65536, num_pages <= 2^30, max_pages * page_size <= 2^30, 1 <= T <= 2^22,
 * B * T < 2^31, B * max_pages < 2^31; slots 8-byte aligned, the others 4-byte aligned; outputs
 * meet nothing else. The result does not depend on what else runs.
 * One or two kernel launches. Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_page_assign(int* page_table, const int* kv_lens, int* held, int* free_pages, int* free_count,
                         int B, int num_pages, int page_size, int max_pages, int T, const int* new_lens,
                         int window, int sinks, int64_t* slots, cudaStream_t stream);

/* Bytes of device workspace fa_page_select needs. Returns 0 for sizes it
 * refuses. */
size_t fa_page_select_workspace_size(int B, int Hkv, int max_pages);

/* Choose, for one new token per sequence, the pages its attention reads: per
 * sequence and KV head the n_sel pages with the highest score
 *   score(page) = max over the group's query heads h of
 *                 sum_d max(q[h,d] min[page,d], q[h,d] max[page,d]),
 * an upper bound of q . k over the page's keys, from k_bounds alone.
 *   q [B, Hq, 1, D]; n_sel >= 1; the first keep_first and the last keep_last
 *   pages of the sequence are always chosen (keep_first + keep_last <= n_sel).
 *   sel [B, Hkv, n_sel] int32: the chosen page numbers within the sequence,
 *   ascending, then -1; sel_lens [B, Hkv] int32: how many. A sequence of at most
 *   n_sel pages gets all of them.
 * The choice is the one that scores computed in 64 bits give, ties going to the
 * lower page; a NaN score counts as the highest. A bad page (see above) scores
 * lowest. 1 <= n_sel <= 2^20. Workspace: fa_page_select_workspace_size(B,
 * Hkv, max_pages) bytes, 16-byte aligned; as for fa_paged_fwd.
 * Returns FA_OK or an error code (nothing launched on error). */
fa_status fa_page_select(const fa_paged_kv* kv, const void* q, int Hq, int n_sel, int keep_first,
                         int keep_last, int* sel, int* sel_lens, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* Human-readable name of a status code (static storage; never NULL). */
const char* fa_status_string(fa_status s);

/* Read the device status word on the current device after synchronising
 * `stream`. *bits receives the raw word (bit 0: a bounded wait gave up; bit 2: a
 * kernel of the paged cache met an index out of range); when `clear` is
 * non-zero the word is reset to 0 afterwards. Returns FA_OK when the word is 0,
 * FA_ERR_BAD_INDEX when only bit 2 is set, FA_ERR_TIMEOUT for any other bit,
 * FA_ERR_LAUNCH when the read itself failed. */
fa_status fa_device_status(unsigned int* bits, int clear, cudaStream_t stream);

/* Self-test of the bounded waits (a library check; the pages have no
 * counterpart). Launches one small kernel on `stream` in which one warp waits
 * on an mbarrier that can never complete, with a limit of `timeout_ms`
 * milliseconds, and a second warp waits on another such barrier with four
 * times that limit. The first wait gives up, sets FA_ERR_TIMEOUT's bit in the
 * device status word and raises the kernel's abort flag, which lets the second
 * warp leave at once; the kernel then exits normally and the context stays
 * usable. Read the result with fa_device_status(). Returns FA_OK once the
 * kernel is launched, FA_ERR_INVALID_ARG for timeout_ms outside 1..10000,
 * FA_ERR_LAUNCH on a launch failure. */
fa_status fa_selftest_wait_timeout(unsigned int timeout_ms, cudaStream_t stream);

/* Bound, in SM clock cycles, of the ordinary waits of every kernel launched
 * after this call by any host thread of the process (a library diagnostic for
 * tests of the give-up path; the pages have no counterpart). 0 restores the
 * default (FA_WAIT_TIMEOUT_MS, else 4 s). With a bound of a few cycles the
 * first wait of each kernel gives up: the kernel sets FA_ERR_TIMEOUT's bit in
 * the device status word and runs to its exit. The waits at exit that let
 * copies and MMAs already in flight finish keep the default bound, so no CTA
 * leaves with work outstanding; outputs of such a call are undefined. Calls
 * made after restoring the default compute normally. Always returns FA_OK. */
fa_status fa_set_wait_limit_cycles(unsigned long long cycles);

/* Version of this ABI (major * 100 + minor). */
int fa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H_ */
