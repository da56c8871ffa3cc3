// Attention over the paged cache where a KV head has many query rows (drafted
// tokens times a group of heads): the split list of fa_paged_fwd.cuh with its
// products on tcgen05.
//
// With R rows per KV head every key takes 6 R D flops for 4 D bytes (the product
// with V twice, see below): at 64 rows 96 flops per byte, 650 TFLOP/s at the copy
// rate. Warp-level products do not get there: their fragments go through registers
// and two warps per scheduler wait for each other's chains.
//
// The 128 rows of an MMA are TMEM lanes, and a warp can read 32 of them only. So a
// block of 32 or 64 rows is there four times or twice: copy k of a row takes keys
// [64 k / copies, ...) of each tile, with a running maximum, a sum and an
// accumulator of its own, and the copies are joined at the end of the segment, as
// the warps' keys are in the other kernel. Every thread of the softmax warps then
// has one row and 16, 32 or 64 keys of a tile, whatever the number of rows. What a
// copy does not take has P = 0, written once: the columns of the other copies are
// never touched.
//
// Roles: two warpgroups of softmax (D 256: one; thread = TMEM lane = row), which take
// tiles in turn, each with its own buffers, maxima, sums and accumulator: a tile is a
// chain of waits and TMEM round trips of over 1100 cycles, more than its bytes take.
// One or two warps look pages up and load by TMA (one takes 1000 cycles a tile and
// more). One warp issues S(t) = Q K(t)^T; the softmax reads it (then S(t + 2) may
// overwrite it) and writes P(t) = 2^(S - m) in two words of the cache's type, P_hi +
// P_lo; another warp issues O += P_hi V + P_lo V. (One warp for both takes 1500 cycles
// a tile, a hundred and more in each wait.) O is rescaled in TMEM when a maximum grows
// by more than 2^8. At the end of a segment both warpgroups read both accumulators,
// half of the columns each.
//
// Measured (269 MB of bf16 keys and values, 16 units, no window, start and join of some 10 us
// included; warp-level products in brackets): D 128, 32 rows 57 us (64), 64 rows 59
// (111), 128 rows 67 (190); D 96, 52 and 65 us for 64 and 128 rows of 201 MB; D 64, 32
// rows 58 (80), 64 rows 65 (128), 128 rows 88 (233); D 256, 32 rows 66 (65), 64 rows 72
// (106), 128 rows 83 (190). At D 128 the loads bound it up to 64 rows (537 MB 93 to 96
// us, 83 to 85% of the copy rate), at D 64, with half the bytes per tile, the softmax's
// chain, at D 256 the two stages that fit.
// Rings of their own for K and V (D 256 62 us with 32 rows, but D 64 67 and five drafts
// of short lists 8% slower) add waits and commits where D 64 has no time for them.
#pragma once

namespace fa {

// RG: groups of 32 rows. E8: the cache is held in e4m3 with scales. Its tiles come into a ring
// of their own (Raw), a warpgroup converts them to fp16 into the ring that the MMAs read, and
// the scales go to the scores and, as parts of the largest one so far, to the weights.
// Measured (134 MB of e4m3, bf16 queries, 16 units of 32768 keys, start and join included): D 128, 32
// rows 58 us, 64 rows 67, 128 rows 86; D 64 with 65536 keys 64 rows 83: bound by the softmax's chain,
// 3300 to 5100 cycles for a warpgroup's tile, two of them in turn (D 128, 64 rows: score load 680,
// scales and mask 400, exponentials 550, waits for scores and products 800). Warp-level products,
// with the same tiles and shares: 64 rows 102, 128 rows 180. D 256 keeps those (64 rows of 16384
// keys 93 us): fp16 tiles of 64 KB beside their raw ones leave one stage.
template <int D_, int RG_, bool BF16_, bool E8_, int MASK_>
struct PagedTcCfg {
  static constexpr int D = D_, RG = RG_;
  static constexpr bool BF16 = BF16_, E8 = E8_, WINDOW = MASK_ >= kWindow, SINKS = MASK_ == kWindowSinks;
  static constexpr bool MMA_BF16 = BF16 && !E8;   // type of the products' operands
  static constexpr bool TWO_WORDS = !(E8 && BF16);  // of weights: one fp16 word for a bf16 output (fa_paged8.cuh)
  static constexpr int ROWS = 32 * RG;           // rows of a block
  static constexpr int COPIES = 4 / RG;          // of each row
  static constexpr int KEYS = kPagedTile / COPIES;  // of a tile that a copy takes
  // (128 rows, where the softmax bounds the kernel, D 128: 68.8 us with one producer,
  // 75.2 with two; 64 rows, D 64 in pages of 16: 92.9 and 72.5)
  static constexpr int PRODUCERS = (RG == 4 && !E8) || D == 256 ? 1 : 2;
  // D = 256: one accumulator is all that TMEM holds beside the scores and weights, and a
  // tile's bytes take longer than the softmax's chain
  static constexpr int WGS = D == 256 ? 1 : 2;
  // (E8: whole warpgroups, which share the registers unevenly: producers and issuers, converters)
  static constexpr int SOFT = 128 * WGS, SCORE_WARP = 4 * WGS + PRODUCERS, CONVERT_WARP = 4 * WGS + 4;
  static_assert(!E8 || SCORE_WARP + 2 == CONVERT_WARP, "every warp has a role: the window moves on with all of them");
  static constexpr int THREADS = E8 ? SOFT + 256 : SOFT + 32 * PRODUCERS + 64;
  static constexpr int REG_SOFT = 168, REG_REST = 88;
  static constexpr int REG_NEEDED = E8 ? SOFT * REG_SOFT + 256 * REG_REST : 0;
  static constexpr int COLS = 64, KREG = (D + 63) / 64, REGION = kPagedTile * 128, TILE = KREG * REGION;
  static constexpr int QREGION = 128 * 128;
  static constexpr int STAGES = E8 ? (D == 64 ? 6 : 4) : D == 256 ? 2 : D == 64 ? 8 : 5;
  struct Raw {  // tiles as they are held
    static constexpr bool E8 = true, WINDOW = true, SINKS = true;
    static constexpr int COLS = 128, KREG = (D_ + 127) / 128, REGION = kPagedTile * 128, TILE = KREG * REGION;
    static constexpr int STAGES = D_ == 64 ? 5 : 3, PRODUCERS = PagedTcCfg::PRODUCERS;
  };
  static constexpr int MC = D == 96 ? 48 : 64;   // columns merged at a time (all at once would cost a stage)
  static constexpr int OP = MC + 4;              // row pitch of the merge buffer (floats)
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = OFF_KV + STAGES * 2 * TILE;
  // (E8: over the queries, which nobody reads then)
  static constexpr int Q_BYTES = KREG * QREGION, O_BYTES = COPIES > 1 ? ROWS * OP * 4 : 0;
  static constexpr int OFF_O = E8 ? OFF_Q : OFF_Q + Q_BYTES;
  static constexpr int OFF_ML = E8 ? OFF_Q + (Q_BYTES > O_BYTES ? Q_BYTES : O_BYTES) : OFF_O + O_BYTES;  // [warpgroup][copies][rows]
  static constexpr int OFF_RAW = (OFF_ML + SOFT * 8 + 1023) / 1024 * 1024;
  static constexpr int SMEM_BYTES = (E8 ? OFF_RAW + Raw::STAGES * 2 * Raw::TILE : OFF_ML + SOFT * 8) + 1024;
  // fp16 weights are up to 2^8 (E8: times parts of scales, at most 1); times this they stay
  // within fp16, and small ones beside a dominating key keep their digits (E8: what a small
  // part leaves of them is 2^-31 of the largest scale)
  static constexpr int LIFT_LOG2 = MMA_BF16 ? 0 : 7;
  static constexpr float LIFT = MMA_BF16 ? 1.f : 128.f;
  static_assert(SMEM_BYTES <= 229000, "shared memory");
  // TMEM columns
  __host__ __device__ static constexpr int S_COL(int b) { return kPagedTile * b; }
  __host__ __device__ static constexpr int P_COL(int b) { return 2 * kPagedTile + kPagedTile * b; }  // P_hi, then P_lo
  static constexpr int P_LO = kPagedTile / 2;
  __host__ __device__ static constexpr int O_COL(int b) { return 4 * kPagedTile + KREG * 64 * b; }
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(4 * kPagedTile + WGS * KREG * 64 <= 512, "TMEM");
};

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(taddr, r);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_ld32(taddr + i, *reinterpret_cast<uint32_t(*)[32]>(&r[i]));
  }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 8)
    tmem_st8(taddr, r);
  else if constexpr (N == 16)
    tmem_st16(taddr, r);
  else
    tmem_st32(taddr, r);
}

// Two fp32 values side by side: both + c, times f.
__device__ __forceinline__ uint64_t pair_of(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(uint32_t a, uint32_t b, uint64_t f, uint64_t c, uint64_t g, uint64_t d) {  // ((a, b) f + c) g + d
  float2 r;
  asm("{\n .reg .b64 x;\n"
      " mov.b64 x, {%2, %3};\n fma.rn.f32x2 x, x, %4, %5;\n fma.rn.f32x2 x, x, %6, %7;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b), "l"(f), "l"(c), "l"(g), "l"(d));
  return r;
}
__device__ __forceinline__ float2 add_fma2(uint32_t a, uint32_t b, uint64_t c, uint64_t f, uint64_t d) {  // ((a, b) + c) f + d
  float2 r;
  asm("{\n .reg .b64 x;\n"
      " mov.b64 x, {%2, %3};\n add.rn.f32x2 x, x, %4;\n fma.rn.f32x2 x, x, %5, %6;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b), "l"(c), "l"(f), "l"(d));
  return r;
}
__device__ __forceinline__ float2 add_mul2(uint32_t a, uint32_t b, uint64_t c, uint64_t f) {
  float2 r;
  asm("{\n .reg .b64 x;\n"
      " mov.b64 x, {%2, %3};\n add.rn.f32x2 x, x, %4;\n mul.rn.f32x2 x, x, %5;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b), "l"(c), "l"(f));
  return r;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
fa_paged_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const PagedFwdArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[C::STAGES], empty[C::STAGES], s_full[2], s_free[2], p_full[2], o_ready[2],
      q_ready, s_drained, o_drained, meet[2];
  __shared__ __align__(16) int key_pos[C::STAGES][kPagedKeyWarps];
  __shared__ int odd_flags[2][2][4];
  __shared__ ItemLens item_lens[kItemWindow];
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_slot;
  // E8: the ring of tiles as they are held, scales of a stage's 16 keys, of query rows, and the
  // accumulators' units
  using Raw = typename C::Raw;
  constexpr int RAW = C::E8 ? Raw::STAGES : 1;
  __shared__ __align__(8) uint64_t raw_full[RAW], raw_empty[RAW];
  __shared__ int raw_pos[RAW][kPagedKeyWarps];
  __shared__ float2 raw_scale[RAW][kPagedKeyWarps], kv_scale[C::E8 ? C::STAGES : 1][kPagedKeyWarps];
  __shared__ bool seen[C::E8 ? C::STAGES : 1];  // all keys of the stage, by every row
  __shared__ float row_scale[C::E8 ? C::ROWS : 1], units[C::E8 ? C::SOFT : 1];
  constexpr int D = C::D;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x, parts = gridDim.x;
  const uint64_t tmo = p.wc.timeout_cycles;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), C::E8 ? 4 : 1);  // the converters' warps
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < RAW; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1 + kPagedKeyWarps);  // the tile, and the scales of each 16 keys
      mbar_init(smem_u32(&raw_empty[i]), 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&s_free[b]), 4);   // one per warp of a warpgroup
      mbar_init(smem_u32(&p_full[b]), 4);
      mbar_init(smem_u32(&o_ready[b]), 1);
      mbar_init(smem_u32(&meet[b]), 4);
    }
    mbar_init(smem_u32(&q_ready), 4 * C::WGS);
    mbar_init(smem_u32(&s_drained), 1);
    mbar_init(smem_u32(&o_drained), 1);
    fence_mbar_init();
  }
  if (warp == C::SCORE_WARP) {
    tmem_alloc(smem_u32(&tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == C::SOFT) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  grid_wait_prior();
  grid_release_next();
  prefetch_inputs<C>(p, part);
  tc_fence_before();
  const ListShape list = list_shape<C>(p);
  ItemWindow<C::THREADS> window{p, item_lens, list.items, 0};
  const Share share = find_share<C::THREADS>(p, list, part, parts, window);  // barriers inside
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Every warp walks the share to its end, whether or not its waits gave up: the window
  // moves on with all of them.

  if (C::E8 && warp >= 4 * C::WGS) regs_release<C::REG_REST>();
  if (C::E8 && warp >= C::CONVERT_WARP) {
    // --------------------------------------------------------------- converters
    // A thread takes a row's 64 columns (D 64: 32), 16 at a time; threads of one row in another
    // order, so that neither reads nor writes meet in a bank.
    bool ok = true;
    const int ct = threadIdx.x - 32 * C::CONVERT_WARP, row = ct >> 1, half = ct & 1;
    constexpr int CHUNKS = D / 32;  // of 16 columns, per thread
    int gi = 0;
    Walk w;
    for (bool more = w.start(list, share, window); more; more = w.next(list, window)) {
      for (int t = w.t0; t < w.t1 && ok; ++t, ++gi) {
        const int from = gi % RAW, to = gi % C::STAGES;
        const uint32_t bar_raw = smem_u32(&raw_full[from]), bar_to = smem_u32(&empty[to]);
        const bool there = mbar_test_wait(bar_raw, (gi / RAW) & 1);
        const bool room = gi < C::STAGES || mbar_test_wait(bar_to, (gi / C::STAGES - 1) & 1);
        if (!__all_sync(0xffffffffu, there && room)) {
          ok = mbar_wait(bar_raw, (gi / RAW) & 1, tmo, &abort_flag, p.wc.status) &&
               (gi < C::STAGES || mbar_wait(bar_to, (gi / C::STAGES - 1) & 1, tmo, &abort_flag, p.wc.status));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (ct < kPagedKeyWarps) {
          const int j0 = raw_pos[from][ct];
          const bool every = __all_sync(0xfu, (j0 & kSeenByAll) != 0);
          if (ct == 0) seen[to] = every;
          key_pos[to][ct] = j0 & ~kSeenByAll;
          // (keys that were not loaded have no scale)
          kv_scale[to][ct] = j0 == kNoPosition ? make_float2(1.f, 0.f) : raw_scale[from][ct];
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {  // keys, values
          const uint8_t* src = smem + C::OFF_RAW + (2 * from + v) * Raw::TILE;
          uint8_t* dst = smem + C::OFF_KV + (2 * to + v) * C::TILE;
          uint4 x[CHUNKS];
          auto chunk = [&](int j) { return half * CHUNKS + (half && CHUNKS == 4 ? j ^ 2 : j); };
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) x[j] = *reinterpret_cast<const uint4*>(src + sw128_offset(row, chunk(j)));
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) {
            uint32_t y[8];
            const uint32_t words[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) f16_of(words[e], y[2 * e], y[2 * e + 1]);
            const int ch = 2 * chunk(j);  // of 8 columns
            uint8_t* at = dst + (ch >> 3) * C::REGION;
            *reinterpret_cast<uint4*>(at + sw128_offset(row, ch & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(at + sw128_offset(row, (ch + 1) & 7)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&full[to]));
          mbar_arrive(smem_u32(&raw_empty[from]));
        }
      }
    }
  } else if (warp >= 4 * C::WGS && warp < C::SCORE_WARP) {
    // ----------------------------------------------------------- producer warps
    if constexpr (C::E8) {
      TileRing<Raw> ring(p, map_k, map_v, sbase + C::OFF_RAW, raw_full, raw_empty, raw_pos, &abort_flag, warp - 4 * C::WGS,
                         raw_scale);
      produce_share<Raw>(p, list, share, window, ring);
      ring.drain();
    } else {
      TileRing<C> ring(p, map_k, map_v, sbase + C::OFF_KV, full, empty, key_pos, &abort_flag, warp - 4 * C::WGS);
      produce_share<C>(p, list, share, window, ring);
      ring.drain();
    }
  } else if (warp >= C::SCORE_WARP) {
    // -------------------------------------------------------------- MMA issuers
    // (all lanes compute the descriptors and one issues)
    const bool leader = elect_one_sync(), scores = warp == C::SCORE_WARP;
    constexpr uint32_t idesc_s = make_idesc_f16(128, kPagedTile, C::MMA_BF16 ? 1 : 0, 0, 0);
    constexpr uint32_t idesc_o = make_idesc_f16(128, D, C::MMA_BF16 ? 1 : 0, 0, 1);
    bool ok = true;
    auto wait = [&](uint64_t& bar, int parity) {
      ok = ok && mbar_wait_poll(smem_u32(&bar), parity & 1, tmo, &abort_flag, p.wc.status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) tc_fence_after();
    };
    int gi = 0, seg = 0;
    Walk w;
    for (bool more = w.start(list, share, window); more; more = w.next(list, window), ++seg) {
      if (!ok) continue;
      const int first = gi, end = gi + w.t1 - w.t0;
      if (scores) wait(q_ready, seg);
      for (; gi < end && ok; ++gi) {
        const int slot = gi % C::STAGES, b = gi & 1;
        const uint32_t kv = sbase + C::OFF_KV + slot * 2 * C::TILE;
        if (scores) {
          // (scores of the segment before: read at its end)
          const bool there = mbar_test_wait(smem_u32(&full[slot]), gi / C::STAGES & 1);
          const bool read = gi - 2 < first || mbar_test_wait(smem_u32(&s_free[b]), ((gi - 2) >> 1) & 1);
          if (__all_sync(0xffffffffu, there && read)) {
            tc_fence_after();
          } else {
            wait(full[slot], gi / C::STAGES);
            if (gi - 2 >= first) wait(s_free[b], (gi - 2) >> 1);
            if (!ok) break;
          }
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk & 3) * 32;  // 16 elements along K
            const uint64_t qd = make_sdesc(sbase + C::OFF_Q + (kk >> 2) * C::QREGION + off, 16, 1024, 2);
            const uint64_t kd = make_sdesc(kv + (kk >> 2) * C::REGION + off, 16, 1024, 2);
            if (leader) mma_ss(tmem + C::S_COL(b), qd, kd, idesc_s, kk > 0);
          }
          if (leader) mma_commit(smem_u32(&s_full[b]));
        } else {
          wait(p_full[b], gi >> 1);
          if (!ok) break;
#pragma unroll
          for (int kk = 0; kk < kPagedTile / 16; ++kk) {
            const uint64_t vd = make_sdesc(kv + C::TILE + kk * 16 * 128, C::REGION, 1024, 2);
            const uint32_t pc = tmem + C::P_COL(b) + kk * 8;
            if (leader) mma_ts(tmem + C::O_COL(C::WGS > 1 ? b : 0), pc, vd, idesc_o, 1);
            if (C::TWO_WORDS && leader) mma_ts(tmem + C::O_COL(C::WGS > 1 ? b : 0), pc + C::P_LO, vd, idesc_o, 1);
          }
          if (leader) mma_commit(smem_u32(&o_ready[b]));
          if (leader) mma_commit(smem_u32(&empty[slot]));
        }
      }
    }
    // nothing is in flight when TMEM is released
    uint64_t& drained = scores ? s_drained : o_drained;
    if (leader) mma_commit(smem_u32(&drained));
    mbar_wait(smem_u32(&drained), 0, p.wc.drain_cycles, nullptr, p.wc.status);
  } else {
    // ------------------------------------------------------------------ softmax
    if constexpr (C::E8) regs_claim<C::REG_SOFT>();
    const int tid = threadIdx.x, wg = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const int copy = quarter / C::RG, row = tid % C::ROWS;
    float* om = reinterpret_cast<float*>(smem + C::OFF_O);
    float2* mls = reinterpret_cast<float2*>(smem + C::OFF_ML);
    auto sync_rows = [&] { named_bar_sync(1, C::SOFT); };
    if (tid == 0 && !p.by_unit) p.joins[part] = make_int2(-1, 0);
    {  // P = 0 where this warp's copy takes no keys
      const uint32_t zero[32] = {};
      for (int b = wg; b < 2; b += C::WGS)
        for (int col = 0; col < kPagedTile; col += 32) tmem_store(lanes + C::P_COL(b) + col, zero);
    }
    int begin = 0, meets = 0;  // tiles of the segments before
    bool ok = true;
    // all four warps of the warpgroup are here (bounded: a warp that gave up does not come)
    auto meet_warps = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&meet[wg]));
      ok = ok && mbar_wait(smem_u32(&meet[wg]), meets & 1, tmo, &abort_flag, p.wc.status);
      ok = __all_sync(0xffffffffu, ok);
      ++meets;
    };
    Walk w;
    for (bool more = w.start(list, share, window); more; more = w.next(list, window)) {
      const int g = kv_head(p, w), rb = row_block(p, w);
      const int rows = min(C::ROWS, p.rows - rb * C::ROWS);
      const int64_t row0 = block_row0(p, item_seq(p, w.item), g, rb, C::ROWS);
      const int len = w.it.len, n = w.it.n;
      const int p_lo = len - n, p_hi = len - 1;  // positions of the new tokens
      const int tok = (rb * C::ROWS + row) % p.Tq, pos = p_lo + tok;
      // queries, every copy; rows behind the last one zero
      constexpr int CHUNKS = C::ROWS * (D / 8), LOADS = (CHUNKS + C::SOFT - 1) / C::SOFT;
      constexpr int WARP_ROWS = C::ROWS / (4 * C::WGS);  // E8: whole rows to a warp
      uint4 x[C::E8 ? WARP_ROWS : LOADS];
      if constexpr (C::E8) {
#pragma unroll
        for (int i = 0; i < WARP_ROWS; ++i) {
          const int r = warp + i * 4 * C::WGS;
          x[i] = make_uint4(0, 0, 0, 0);
          if (r < rows && lane < D / 8) x[i] = reinterpret_cast<const uint4*>(p.q + (row0 + r) * D)[lane];
        }
      } else {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {  // all under way at once
          const int at = tid + i * C::SOFT, r = at / (D / 8);
          x[i] = make_uint4(0, 0, 0, 0);
          if (r < rows) x[i] = reinterpret_cast<const uint4*>(p.q + row0 * D)[at];
        }
      }
      {
        const uint32_t zero[32] = {};
#pragma unroll
        for (int col = 0; col < D; col += 32) tmem_store(lanes + C::O_COL(wg) + col, zero);
      }
      if constexpr (C::E8) {
#pragma unroll
        for (int i = 0; i < WARP_ROWS; ++i) {
          const int r = warp + i * 4 * C::WGS;
          const float undo = row_f16<C::BF16>(x[i]);
          if (lane == 0) row_scale[r] = undo;
          if (lane < D / 8) {
#pragma unroll
            for (int k = 0; k < C::COPIES; ++k)
              *reinterpret_cast<uint4*>(smem + C::OFF_Q + (lane >> 3) * C::QREGION + sw128_offset(k * C::ROWS + r, lane & 7)) = x[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int at = tid + i * C::SOFT, r = at / (D / 8), ch = at - r * (D / 8);
          if (at >= CHUNKS) break;
#pragma unroll
          for (int k = 0; k < C::COPIES; ++k)
            *reinterpret_cast<uint4*>(smem + C::OFF_Q + (ch >> 3) * C::QREGION + sw128_offset(k * C::ROWS + r, ch & 7)) = x[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_ready));
      float own_scale = 1.f, unit = 0.f;  // E8: of this row; what its sums are in units of, less LIFT
      if constexpr (C::E8) {
        sync_rows();  // other warps have staged this row
        own_scale = row_scale[row];
      }
      // The row's running maximum among unscaled scores. An exponent is (s - top) scale: the
      // difference of near scores is exact, so that it is 0 for the maximum, however large
      // (s scale - m in one rounding is not, where the steps of m are large).
      float top = kNoMax, l = 0.f;
      const uint64_t scale2 = pair_of(p.scale_log2);
      const int end = begin + w.t1 - w.t0;
      // the products of tile t (of segments before: waited for at their ends)
      auto wait_products = [&](int t) {
        if (t < begin) return;
        ok = ok && mbar_wait(smem_u32(&o_ready[t & 1]), (t >> 1) & 1, tmo, &abort_flag, p.wc.status);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) tc_fence_after();
      };
      for (int gi = begin + (C::WGS > 1 ? (begin ^ wg) & 1 : 0); gi < end; gi += C::WGS) {
        const int slot = gi % C::STAGES, b = gi & 1;
        // a wait that finds its phase complete still takes a hundred cycles and more: all
        // three are tried at once
        const uint32_t bar_kv = smem_u32(&full[slot]), bar_s = smem_u32(&s_full[b]);
        const bool there = mbar_test_wait(bar_kv, (gi / C::STAGES) & 1), scored = mbar_test_wait(bar_s, (gi >> 1) & 1);
        const bool added = gi - 2 < begin || mbar_test_wait(smem_u32(&o_ready[b]), ((gi - 2) >> 1) & 1);
        const bool p_idle = __all_sync(0xffffffffu, added);
        if (!__all_sync(0xffffffffu, there && scored)) {
          ok = ok && mbar_wait(bar_kv, (gi / C::STAGES) & 1, tmo, &abort_flag, p.wc.status) &&
               mbar_wait(bar_s, (gi >> 1) & 1, tmo, &abort_flag, p.wc.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_after();
        uint32_t sv[C::KEYS];
        tmem_load(lanes + C::S_COL(b) + copy * C::KEYS, sv);
        const int4 kp = *reinterpret_cast<const int4*>(key_pos[slot]);
        const int j0s[4] = {kp.x, kp.y, kp.z, kp.w};
        // does every row see all keys of a group; does some group hide keys from some
        // rows only
        bool all_seen = true, differ = false;
        if (!C::E8 || !seen[slot]) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j0 = j0s[q];
            all_seen &= j0 + 15 < len && !(p.causal && j0 + 15 > p_lo) &&
                        !(windowed<C>(p) && j0 <= p_hi - p.window && past_sinks<C>(p, j0 + 15));
            differ |= n > 1 && j0 < len &&
                      ((p.causal && j0 + 15 > p_lo) ||
                       (windowed<C>(p) && j0 <= p_hi - p.window && j0 + 15 > p_lo - p.window));
          }
        }
        // E8, of each 16 keys: what their scores are to be multiplied by, and the power of two
        // that takes their weights to `unit` (with LIFT). `lower`: what the sums so far are to
        // be multiplied by.
        constexpr int GROUPS = C::E8 ? C::RG : 1;
        float key_scale[GROUPS], factor[GROUPS], power[GROUPS], lower = 1.f;
        if constexpr (C::E8) {
          float most = 0.f, value_scale[GROUPS];
#pragma unroll
          for (int q = 0; q < C::RG; ++q) {
            const float2 sc = kv_scale[slot][copy * C::RG + q];
            key_scale[q] = sc.x;
            value_scale[q] = sc.y;
            factor[q] = own_scale * sc.x;
            most = fmaxf(most, sc.y);
          }
          if (most > unit) {
            lower = unit * inverse_power(most);
            unit = most;
          }
#pragma unroll
          for (int q = 0; q < C::RG; ++q)
            power[q] = static_cast<float>((__float_as_int(value_scale[q]) >> 23) - (__float_as_int(unit) >> 23) + C::LIFT_LOG2);
        }
        tmem_ld_wait();
        auto free_scores = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_free[b]));
        };
        if (!differ) free_scores();  // (else they may be read again below)
        if constexpr (C::E8) {
#pragma unroll
          for (int q = 0; q < C::RG; ++q)
            if (!(factor[q] > 1e-36f && factor[q] < 1e36f)) {
              // the smaller one first, so that it is only the score that can leave the range
              const float f0 = fminf(own_scale, key_scale[q]), f1 = fmaxf(own_scale, key_scale[q]);
#pragma unroll
              for (int e = 0; e < 16; ++e) sv[16 * q + e] = __float_as_uint(__uint_as_float(sv[16 * q + e]) * f0 * f1);
              factor[q] = 1.f;
            }
        }
        if (!all_seen) {
#pragma unroll
          for (int q = 0; q < C::RG; ++q) {
            const int j0 = key_pos[slot][copy * C::RG + q];
            const int lo = windowed<C>(p) ? pos - p.window + 1 - j0 : -j0;
            const int hi = (p.causal ? min(len, pos + 1) : len) - j0;
            const unsigned span = static_cast<unsigned>(max(hi - lo, 0));
            const int keep = C::SINKS ? min(p.sinks - j0, hi) : 0;  // first keys that the window leaves
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (static_cast<unsigned>(e - lo) >= span && (!C::SINKS || e >= keep)) sv[16 * q + e] = __float_as_uint(-INFINITY);
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if constexpr (C::E8) {
#pragma unroll
          for (int q = 0; q < C::RG; ++q) {
            float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 16; ++e) m2[e & 1] = fmaxf(m2[e & 1], __uint_as_float(sv[16 * q + e]));
            m4[q] = fmaxf(m2[0], m2[1]) * factor[q];
          }
        } else {
#pragma unroll
          for (int e = 0; e < C::KEYS; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(sv[e]));
        }
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), rise = (mx - top) * p.scale_log2;
        const bool rises = rise > kPagedSlack, grow = rises || (C::E8 && lower != 1.f);
        float alpha = 1.f;
        if (rises) {
          alpha = ex2(-rise);
          top = mx;
          l *= alpha;
        }
        if constexpr (C::E8) alpha *= lower;
        const uint64_t top2 = pair_of(-top);
        // weights in two words of the cache's type (see the other kernel)
        uint32_t hi[C::KEYS / 2], lo[C::KEYS / 2];
        float sum[2] = {0.f, 0.f}, own[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < C::KEYS / 2; ++e) {
          // E8: the power goes into the exponent, and out of the sum of these 16 weights. (Below
          // 2^-40 a weight, at most 2^8, is 0 in fp16 anyway: the sum is taken by itself.)
          const int q = C::E8 ? e / 8 : 0;
          float2 x;
          if constexpr (C::E8)
            x = fma2(sv[2 * e], sv[2 * e + 1], pair_of(factor[q]), top2, scale2, pair_of(power[q] < -40.f ? 0.f : power[q]));
          else if constexpr (C::LIFT_LOG2 > 0)
            x = add_fma2(sv[2 * e], sv[2 * e + 1], top2, scale2, pair_of(C::LIFT_LOG2));
          else
            x = add_mul2(sv[2 * e], sv[2 * e + 1], top2, scale2);
          const float p0 = ex2(x.x), p1 = ex2(x.y);
          if constexpr (C::E8) {
            own[0] = e % 8 ? own[0] + p0 : p0;
            own[1] = e % 8 ? own[1] + p1 : p1;
            if (e % 8 == 7) {
              const float undo = power[q] < -40.f ? 1.f : __int_as_float((127 - static_cast<int>(power[q])) << 23);
              sum[0] = fmaf(own[0] + own[1], undo, sum[0]);
            }
          } else {
            sum[0] += p0;
            sum[1] += p1;
          }
          hi[e] = pack2<C::MMA_BF16>(p0, p1);
          if constexpr (C::TWO_WORDS) {
            const float2 f = unpack2<C::MMA_BF16>(hi[e]);
            lo[e] = pack2<C::MMA_BF16>(p0 - f.x, p1 - f.y);
          }
        }
        l += sum[0] + sum[1];
        if constexpr (C::E8) {
#pragma unroll
          for (int q = 0; q < C::RG; ++q)
            if (power[q] < -40.f) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                hi[8 * q + e] = 0;
                if constexpr (C::TWO_WORDS) lo[8 * q + e] = 0;
              }
            }
        }
        if (!p_idle) wait_products(gi - 2);  // they read this buffer's last P
        if (!ok) break;
        tmem_store(lanes + C::P_COL(b) + copy * (C::KEYS / 2), hi);
        if constexpr (C::TWO_WORDS) tmem_store(lanes + C::P_COL(b) + C::P_LO + copy * (C::KEYS / 2), lo);
        if (gi - C::WGS >= begin && __any_sync(0xffffffffu, grow)) {
          if (C::WGS == 1) wait_products(gi - 1);  // they add to O
          if (!ok) break;
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            uint32_t o[32];
            tmem_load(lanes + C::O_COL(wg) + col, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_store(lanes + C::O_COL(wg) + col, o);
          }
        }
        if (!all_seen) {
          // A key that no row sees gets V = 0 (its slot may hold anything, and 0 * NaN is
          // not 0); warp w of the four looks after keys 16 w on. Where rows differ in what they see
          // and some of these values are no finite numbers, those keys are added row by
          // row and get V = 0 as well.
          const uint32_t vs = sbase + C::OFF_KV + slot * 2 * C::TILE + C::TILE;
          uint8_t* v_rows = smem + (vs - sbase);
          auto kept = [&](int j) { return j < len && !(windowed<C>(p) && j <= p_lo - p.window && past_sinks<C>(p, j)); };
          auto partial = [&](int j) {
            return kept(j) && ((p.causal && j > p_lo) || (windowed<C>(p) && j <= p_hi - p.window && past_sinks<C>(p, j)));
          };
          const int own = key_pos[slot][quarter];
          constexpr int ROW = D / 8;
          auto chunk = [&](int i) {  // 16 bytes of this warp's keys
            const int e = i / ROW, x = i - e * ROW;
            return v_rows + (x >> 3) * C::REGION + sw128_offset(16 * quarter + e, x & 7);
          };
          bool apart = false;
          if (differ) {
            uint32_t odd = 0;
            for (int i = lane; i < 16 * ROW; i += 32) {
              if (!partial(own + i / ROW)) continue;
              const uint4 x = *reinterpret_cast<const uint4*>(chunk(i));
              odd |= not_finite2<C::MMA_BF16>(x.x) | not_finite2<C::MMA_BF16>(x.y) | not_finite2<C::MMA_BF16>(x.z) |
                     not_finite2<C::MMA_BF16>(x.w);
            }
            odd = __any_sync(0xffffffffu, odd != 0);
            int* flags = odd_flags[wg][meets & 1];
            if (lane == 0) flags[quarter] = static_cast<int>(odd);
            meet_warps();
            if (!ok) break;
            apart = (flags[0] | flags[1] | flags[2] | flags[3]) != 0;
            if (apart) {
              if (C::WGS == 1) wait_products(gi - 1);
              if (!ok) break;
              tmem_st_wait();
              for (int e = 0; e < C::KEYS; ++e) {
                const int key = copy * C::KEYS + e, j = key_pos[slot][key >> 4] + (key & 15);
                if (!partial(j)) continue;
                float s = __uint_as_float(tmem_ld1(lanes + C::S_COL(b) + key));
                tmem_ld_wait();
                float share = C::LIFT;
                if constexpr (C::E8) {
                  const float2 sc = kv_scale[slot][key >> 4];
                  s = s * fminf(own_scale, sc.x) * fmaxf(own_scale, sc.x);
                  share = sc.y * inverse_power(unit) * C::LIFT;
                }
                const bool seen = !(p.causal && j > pos) && !(windowed<C>(p) && j <= pos - p.window && past_sinks<C>(p, j));
                const float x = ex2((s - top) * p.scale_log2) * share;
#pragma unroll 1
                for (int col = 0; col < D; col += 32) {
                  uint32_t o[32];
                  tmem_load(lanes + C::O_COL(wg) + col, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 32; i += 2) {
                    const int at = col + i;
                    const float2 v = unpack2<C::MMA_BF16>(*reinterpret_cast<const uint32_t*>(
                        v_rows + (at >> 6) * C::REGION + sw128_offset(key, (at & 63) >> 3) + (at & 7) * 2));
                    if (seen) {
                      o[i] = __float_as_uint(fmaf(x, v.x, __uint_as_float(o[i])));
                      o[i + 1] = __float_as_uint(fmaf(x, v.y, __uint_as_float(o[i + 1])));
                    }
                  }
                  tmem_store(lanes + C::O_COL(wg) + col, o);
                  tmem_st_wait();
                }
              }
              meet_warps();  // before anybody overwrites what others read
              if (!ok) break;
            }
            free_scores();
          }
          for (int i = lane; i < 16 * ROW; i += 32) {
            const int j = own + i / ROW;
            if (!kept(j) || (apart && partial(j))) *reinterpret_cast<uint4*>(chunk(i)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[b]));
      }

      // ------------------------------------------------------ end of a segment
      // The last products of both warpgroups. (Nobody starts the next segment, whose
      // products would move these barriers on, before all have come to sync_rows.)
      for (int gi = max(begin, end - 2); gi < end; ++gi) {
        ok = ok && mbar_wait(smem_u32(&o_ready[gi & 1]), (gi >> 1) & 1, tmo, &abort_flag, p.wc.status);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) tc_fence_after();
      }
      begin = end;
      // padding rows (tokens the sequence does not have) see nothing; a row that has
      // met nothing but NaN keeps it
      float m = top * p.scale_log2;
      if (tok >= n || (top == kNoMax && l == 0.f)) {
        m = -INFINITY;
        l = 0.f;
      }
      const bool begins = w.t0 == 0, ends = w.t1 == w.it.tiles;
      const int part_slot = 2 * part + (begins ? 1 : 0);
      constexpr float DROP = C::E8 ? 1.f : 1.f / C::LIFT;  // (E8: the units have it, and l is without)
      mls[tid] = make_float2(m, l * DROP);  // [warpgroup][copy][row]
      if constexpr (C::E8) units[tid] = unit / C::LIFT;
      sync_rows();
      const float2 ml0 = mls[tid & 127], ml1 = mls[128 * (C::WGS - 1) + (tid & 127)];
      float mt = -INFINITY;
#pragma unroll
      for (int k = 0; k < C::WGS * C::COPIES; ++k) mt = fmaxf(mt, mls[k * C::ROWS + row].x);
      float f0 = exp2_rel(ml0.x, mt) * DROP, f1 = exp2_rel(ml1.x, mt) * DROP;
      if constexpr (C::E8) {
        f0 *= units[tid & 127];
        f1 *= units[128 * (C::WGS - 1) + (tid & 127)];
      }
      // columns [16 i, 16 i + 16) of this lane's row over the warpgroups
      auto sum16 = [&](int i, float4 (&x)[4]) {
        uint32_t o0[16], o1[16];
        tmem_load(lanes + C::O_COL(0) + 16 * i, o0);
        if constexpr (C::WGS > 1) tmem_load(lanes + C::O_COL(1) + 16 * i, o1);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          auto four = [&](const uint32_t (&o)[16]) {
            return make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]), __uint_as_float(o[4 * k + 2]),
                               __uint_as_float(o[4 * k + 3]));
          };
          if (ml0.x > -INFINITY) add4(x[k], four(o0), f0);  // nothing seen: not even 0 * inf
          if (C::WGS > 1 && ml1.x > -INFINITY) add4(x[k], four(o1), f1);
        }
        __syncwarp();
      };
      auto row_sum = [&](int r) {
        float2 ml = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < C::WGS * C::COPIES; ++k) ml.x = fmaxf(ml.x, mls[k * C::ROWS + r].x);
#pragma unroll
        for (int k = 0; k < C::WGS * C::COPIES; ++k) ml.y += mls[k * C::ROWS + r].y * exp2_rel(mls[k * C::ROWS + r].x, ml.x);
        return ml;
      };
      if constexpr (C::COPIES == 1) {
        const float2 ml = row_sum(row);
#pragma unroll 1
        for (int i = wg; i < D / 16; i += C::WGS) {
          float4 x[4];
          sum16(i, x);
          if (row < rows) {
            put_piece<C>(p, begins && ends, part_slot, row0, row, 2 * i, x[0], x[1], ml);
            put_piece<C>(p, begins && ends, part_slot, row0, row, 2 * i + 1, x[2], x[3], ml);
          }
          __syncwarp();
        }
      } else {
        // each share of the columns is summed by the copies in turn, half of it by each
        // of two warpgroups
        constexpr int SHARE = (C::MC / 16 + C::COPIES - 1) / C::COPIES;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += C::MC) {
          if (c0 > 0) sync_rows();  // the columns before are read
#pragma unroll 1
          for (int round = 0; round < C::COPIES; ++round) {
            const int first = (copy + round) % C::COPIES * SHARE;
#pragma unroll 1
            for (int i = first; i < min(first + SHARE, C::MC / 16); ++i) {
              if (C::WGS > 1 && (i & 1) != wg) continue;
              float4 x[4];
              sum16(c0 / 16 + i, x);
              float4* at = reinterpret_cast<float4*>(om + row * C::OP + 16 * i);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (round > 0) add4(x[k], at[k], 1.f);
                at[k] = x[k];
              }
            }
            sync_rows();
          }
          for (int i = tid; i < rows * (C::MC / 8); i += C::SOFT) {
            const int r = i / (C::MC / 8), ch = i - r * (C::MC / 8);
            const float4 x = *reinterpret_cast<const float4*>(om + r * C::OP + 8 * ch);
            const float4 y = *reinterpret_cast<const float4*>(om + r * C::OP + 8 * ch + 4);
            put_piece<C>(p, begins && ends, part_slot, row0, r, c0 / 8 + ch, x, y, row_sum(r));
          }
        }
      }
      tc_fence_before();
      sync_rows();  // accumulators, rows and sums are read
      tc_fence_after();
      if (tid == 0) record_unit(p, list, share, w, part);
    }
    write_empty_units<C>(p, list, part, parts, tid, C::SOFT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::SCORE_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace fa
