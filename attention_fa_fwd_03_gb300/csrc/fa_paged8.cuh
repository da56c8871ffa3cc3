// Attention over a cache held in 8 bits, up to 16 query rows per KV head: what differs from
// fa_paged_fwd.cuh (whose list, shares, parts and join it uses).
//
//   S = scale ks (q k8), O = sum p vs v8 / l      k8, v8 held; ks, vs their pages' scales
//
// A tile's bytes take half as long as with 16 bits, so instructions and what happens
// between tiles and segments count twice. e4m3 numbers are fp16 numbers: fragments are
// read as they are held and converted in registers, products are fp16 with fp32 sums, and
// the scales, one of each per 16 keys, go to factors that the scores and weights are
// multiplied by anyway.
#pragma once

namespace fa {

// ------------------------------------------------- products of held 8-bit values
// e4m3 values are fp16 numbers, so fragments are read as they are held, two columns to a
// 16-bit place, and converted in registers (64 pairs per clock and SM; with integer
// operations a third of that, and NaN would be lost).
__device__ __forceinline__ void f16_of(uint32_t four_e4m3, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(four_e4m3));
}
// Keys: a thread has columns 4 (lane % 4) to the third behind it of 16 of a key (x) and of
// the eighth behind it (y). Pairs of them make the fragment; its columns are thereby in another
// order, and so are the staged queries'.
__device__ __forceinline__ void keys_f16(uint32_t (&a)[4], uint32_t x, uint32_t y) {
  f16_of(x, a[0], a[2]);
  f16_of(y, a[1], a[3]);
}
// Values, read transposed: a place holds columns 2 (lane / 4) and the next of one key. The
// fragment's first eight rows are the even columns, the others the odd ones.
__device__ __forceinline__ void values_f16(uint32_t (&a)[4], uint32_t x, uint32_t y) {
  f16_of(__byte_perm(x, 0, 0x3120), a[0], a[1]);
  f16_of(__byte_perm(y, 0, 0x3120), a[2], a[3]);
}
// Column of element e of a thread's accumulator i.
template <class C>
__device__ __forceinline__ int acc_column(int i, int lane, int e) {
  return C::E8 ? 16 * i + 2 * (lane >> 2) + (e >> 1) : 16 * i + (lane >> 2) + 8 * (e >> 1);
}
// 1 / x of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float inverse_power(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }
// Not 0 where one of four e4m3 values is NaN.
__device__ __forceinline__ uint32_t nan4_e4m3(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// A query row in fp16, eight columns to a lane, and what it is to be multiplied by. A bf16 row
// is brought to a largest magnitude in [2^14, 2^15): its elements down to 2^-28 of that are
// exact, and the rest is off by at most 2^-40 of it.
template <bool BF16>
__device__ __forceinline__ float row_f16(uint4& x) {
  if constexpr (!BF16) return 1.f;
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<true>(w[i]);
    if (fabsf(f.x) < INFINITY) most = fmaxf(most, fabsf(f.x));
    if (fabsf(f.y) < INFINITY) most = fmaxf(most, fabsf(f.y));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  // 2^(e - 14) of a magnitude in [2^e, 2^(e + 1)), within normal numbers; of zeros 1
  const int field = most > 0.f ? min(max(static_cast<int>(__float_as_uint(most) >> 23) - 14, 1), 253) : 127;
  const float f = __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<true>(w[i]);
    w[i] = pack2<false>(v.x * f, v.y * f);
  }
  return __uint_as_float(static_cast<uint32_t>(field) << 23);
}

// A block's query rows in fp16, in the order of columns that keys_f16 gives, and their scales.
template <class C>
struct QueryRows {
  static constexpr int EACH = C::ROWS / C::WARPS, CHUNKS = C::D / 8;
  uint4 x[EACH];
  __device__ __forceinline__ void load(const PagedFwdArgs& p, int64_t row0, int rows, int warp, int lane) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) {  // all under way at once
      const int r = warp + k * C::WARPS;
      x[k] = make_uint4(0, 0, 0, 0);
      if (r < rows && lane < CHUNKS) x[k] = reinterpret_cast<const uint4*>(p.q + (row0 + r) * C::D)[lane];
    }
  }
  __device__ __forceinline__ void store(uint8_t* dst, float* scales, int warp, int lane);
};
template <class C>
__device__ __forceinline__ void QueryRows<C>::store(uint8_t* dst, float* scales, int warp, int lane) {
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int r = warp + k * C::WARPS;
    uint32_t* w = reinterpret_cast<uint32_t*>(&x[k]);
    const float undo = row_f16<C::BF16>(x[k]);
    if (lane == 0) scales[r] = undo;
    // pairs 0 2 4 6 of 16 columns to the first chunk, 1 3 5 7 to the second
    const bool odd = lane & 1;
    const uint32_t s0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), s1 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
    const uint4 y = odd ? make_uint4(s0, s1, w[1], w[3]) : make_uint4(w[0], w[2], s0, s1);
    if (lane < CHUNKS) *reinterpret_cast<uint4*>(dst + (lane >> 3) * C::QREGION + sw128_offset(r, lane & 7)) = y;
  }
}


// Weights go to their product as fp16 numbers times this: they are up to 2^8 (kPagedSlack) and
// parts of scales at most 1, so the products stay within fp16, and small ones keep their digits:
// as they are, a weight would lose digits from 2^-14 of the running maximum's on and be nothing
// below 2^-25, where one key dominates and many others share the rest the larger part of the row.
constexpr float kWeightLift = 128.f;

// One tile's 16 keys of a warp: their scores with the warp's query rows, weights, and the
// product with the values, added to the running maxima, sums and rows. `ks`, `vs`: shared
// addresses of the keys' and values' first rows, regions of 128 columns REGION bytes apart;
// `scale`: of the keys and of the values; `all`: every row sees every key. A row's element is
// as in fa_paged_fwd_kernel but for the columns of V (acc_column).
template <class C, int REGION, class Query>
__device__ __forceinline__ void step8(const PagedFwdArgs& p, uint32_t ks, uint32_t vs, int lane, float2 scale, int j0,
                                      bool all, int len, int n, uint64_t tokens, const Query& query,
                                      const float2 (&rs)[C::NT], float (&m)[C::NT][2], float (&l)[C::NT][2],
                                      float (&acc)[C::NT][C::D / 16][4], float& unit, bool& large) {
  constexpr int D = C::D, NT = C::NT;
  const int p_lo = len - n, p_hi = len - 1;
  auto token = [&](int nt, int e) { return static_cast<int>(tokens >> (8 * nt + 4 * e)) & 15; };
  float s[NT][4], s2[4];
  const int kr = lane & 15, kc = lane >> 4;
#pragma unroll
  for (int k2 = 0; k2 < D / 32; ++k2) {
    uint32_t x[4], a0[4], a1[4];
    ldsm4(x, ks + (k2 >> 2) * REGION + sw128_offset(kr, (2 * k2 + kc) & 7));
    keys_f16(a0, x[0], x[1]);
    keys_f16(a1, x[2], x[3]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t b[4];
      query(b, nt, k2);
      if (k2 == 0)
        mma16816_first<false>(s[nt], a0, b[0], b[1]);
      else
        mma16816<false>(s[nt], a0, b[0], b[1]);
      if (NT == 1 && k2 == 0)
        mma16816_first<false>(s2, a1, b[2], b[3]);
      else
        mma16816<false>(NT == 1 ? s2 : s[nt], a1, b[2], b[3]);
    }
  }
  if constexpr (NT == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][e] += s2[e];
  }
  // The values' scale goes to the weights, as a part of the largest one so far, `unit` (rows
  // are sums in units of unit / kWeightLift); where that would cost the weights digits (below
  // 1/16), to the products instead.
  if (scale.y > unit) {
    const float f = unit * inverse_power(scale.y);
    unit = scale.y;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][i][e] *= f;
  }
  const float part = scale.y * inverse_power(unit);
  const bool fold = part >= 0.0625f;
  // The keys' and the row's powers of two go to the factor that scores are multiplied by
  // anyway, where it stays a normal number; else to the scores, the smaller one first so
  // that it is only what the score is that can leave the range.
  float sf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float r = h ? rs[nt].y : rs[nt].x;
      sf[nt][h] = r * scale.x * p.scale_log2;
      if (!(sf[nt][h] > 1e-36f && sf[nt][h] < 1e36f)) {
        sf[nt][h] = p.scale_log2;
#pragma unroll
        for (int e = h; e < 4; e += 2) s[nt][e] = s[nt][e] * fminf(r, scale.x) * fmaxf(r, scale.x);
      }
    }
  uint32_t keep0 = ~0u, keep1 = ~0u;  // keys of this thread's V fragments that some row sees
  const int jv = j0 + 2 * (lane & 3);
  if (!all) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pos = p_lo + token(nt, h);
        const int lo = p.window > 0 ? pos - p.window + 1 - j0 : -j0;
        const int hi = (p.causal ? min(len, pos + 1) : len) - j0;
        const unsigned span = static_cast<unsigned>(max(hi - lo, 0)), j = (lane >> 2) - lo;
        const int keep = min(p.sinks - j0, hi);
        if (j >= span && (lane >> 2) >= keep) s[nt][h] = -INFINITY;
        if (j + 8 >= span && (lane >> 2) + 8 >= keep) s[nt][2 + h] = -INFINITY;
      }
    auto seen = [&](int j) { return j < len && !(p.window > 0 && j <= p_lo - p.window && j >= p.sinks); };
    keep0 = (seen(jv) ? 0xffffu : 0u) | (seen(jv + 1) ? 0xffff0000u : 0u);
    keep1 = (seen(jv + 8) ? 0xffffu : 0u) | (seen(jv + 9) ? 0xffff0000u : 0u);
  }
  // exponents against the running maxima, looked at across lanes only where one is above
  // the slack
  float x[NT][4];
  bool above = large;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[nt][e] = fmaf(s[nt][e], sf[nt][e & 1], -m[nt][e & 1]);
      above |= x[nt][e] > kPagedSlack;
    }
  if (__any_sync(0xffffffffu, above)) {
    bool any_large = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y = fmaxf(s[nt][h], s[nt][2 + h]);
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
        const float mn = fmaxf(m[nt][h], y * sf[nt][h]);
        alpha[h] = ex2(m[nt][h] - mn);
        m[nt][h] = mn;
        any_large |= large_max(mn);
        l[nt][h] *= alpha[h];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        acc[nt][i][0] *= alpha[0];
        acc[nt][i][1] *= alpha[1];
        acc[nt][i][2] *= alpha[0];
        acc[nt][i][3] *= alpha[1];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(s[nt][e], sf[nt][e & 1], -m[nt][e & 1]);
    }
    large = __any_sync(0xffffffffu, any_large);
    if (large) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = __fmul_rn(s[nt][e], sf[nt][e & 1]) - m[nt][e & 1];
    }
  }
  // Weights in fp16 (with all digits down to 2^-21 of the running maximum over `part`). For fp16
  // outputs in two words, to 2^-22 of themselves; for bf16 outputs in one, to 2^-11: O is off by
  // that times sum p |v| / l beside its own rounding by 2^-8 |O|, which is more unless values
  // cancel. A second word there: 131072 keys 55.1 us instead of 52.2, 64 ragged sequences 102.8
  // instead of 94.3, 16 units of 32768 keys with 128 rows (fa_paged_tc.cuh) 97 instead of 85.
  constexpr bool TWO_WORDS = !C::BF16;
  const float factor = fold ? part * kWeightLift : kWeightLift, rest = fold ? 1.f : part;
  uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[nt][h] = ex2(x[nt][h]);
      s[nt][2 + h] = ex2(x[nt][2 + h]);
      l[nt][h] += s[nt][h] + s[nt][2 + h];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] *= factor;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t hi = pack2<false>(s[nt][2 * h], s[nt][2 * h + 1]);
      pb[nt][h] = transpose8(hi);
      if constexpr (TWO_WORDS) {
        const float2 f = unpack2<false>(hi);
        pl[nt][h] = transpose8(pack2<false>(s[nt][2 * h] - f.x, s[nt][2 * h + 1] - f.y));
      }
    }
  }
  // O^T += V^T P^T. A key hidden from every row gets V = 0 (its slot may hold anything;
  // 0 * NaN would not be 0). Where rows differ in what they see and some of these values are
  // NaN, each token's product is taken with the keys it sees and only its rows are kept.
  const int vr = ((lane >> 4) << 3) + (lane & 7), vc = (lane >> 3) & 1;
  // two times 16 columns of V^T, from one read of the held values
  auto values_of = [&](uint32_t (&a)[2][4], int i2, uint32_t m0, uint32_t m1) {
    uint32_t v[4];
    ldsm4_trans(v, vs + (i2 >> 2) * REGION + sw128_offset(vr, (2 * i2 + vc) & 7));
    values_f16(a[0], v[0] & m0, v[2] & m1);
    values_f16(a[1], v[1] & m0, v[3] & m1);
  };
  if (all && fold) {
#pragma unroll
    for (int i2 = 0; i2 < D / 32; ++i2) {
      uint32_t a[2][4];
      values_of(a, i2, ~0u, ~0u);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816<false>(acc[nt][2 * i2 + h], a[h], pb[nt][0], pb[nt][1]);
      if constexpr (TWO_WORDS) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<false>(acc[nt][2 * i2 + h], a[h], pl[nt][0], pl[nt][1]);
      }
    }
    return;
  }
  const bool differ = !all && n > 1 &&
                      ((p.causal && j0 + 15 > p_lo && j0 <= p_hi) ||
                       (p.window > 0 && j0 <= p_hi - p.window && j0 + 15 > p_lo - p.window));
  bool apart = false;
  if (differ) {
    uint32_t odd = 0;
#pragma unroll
    for (int i2 = 0; i2 < D / 32; ++i2) {
      uint32_t v[4];
      ldsm4_trans(v, vs + (i2 >> 2) * REGION + sw128_offset(vr, (2 * i2 + vc) & 7));
      odd |= nan4_e4m3(v[0] & keep0) | nan4_e4m3(v[1] & keep0) | nan4_e4m3(v[2] & keep1) | nan4_e4m3(v[3] & keep1);
    }
    apart = __any_sync(0xffffffffu, odd != 0);
  }
#pragma unroll 1
  for (int tok = 0; tok < (apart ? n : 1); ++tok) {
    uint32_t k0 = keep0, k1 = keep1;
    if (apart) {
      const int pos = p_lo + tok;
      auto seen = [&](int j) {
        return j < len && !(p.causal && j > pos) && !(p.window > 0 && j <= pos - p.window && j >= p.sinks);
      };
      k0 = (seen(jv) ? 0xffffu : 0u) | (seen(jv + 1) ? 0xffff0000u : 0u);
      k1 = (seen(jv + 8) ? 0xffffu : 0u) | (seen(jv + 9) ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int i2 = 0; i2 < D / 32; ++i2) {
      uint32_t a[2][4];
      values_of(a, i2, k0, k1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4];
          mma16816_first<false>(y, a[h], pb[nt][0], pb[nt][1]);
          if constexpr (TWO_WORDS) mma16816<false>(y, a[h], pl[nt][0], pl[nt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!apart || token(nt, e & 1) == tok) acc[nt][2 * i2 + h][e] = fmaf(y[e], rest, acc[nt][2 * i2 + h][e]);
        }
    }
  }
}

// ---------------------------------------------------------------- split list
// One CTA per SM holds GROUPS of four consumer warps and a producer, each group with a share
// of the list, a ring and barriers of its own: twelve consumer warps are what it takes to
// keep up with the loads at D 128. (As CTAs of their own, five warps each, it happened that
// registers freed by other kernels' blocks left no place for the third one of an SM, which
// then ran a whole wave later: 64 sequences with one head per KV head 131 us, now 93.
// Four-warp CTAs in which every warp loads its own keys took 102 us for 64 ragged sequences,
// with 4 heads per KV head, against 93 here: the loads' instructions are in the way.)
//
// A group's warps leave their rows of a segment side by side and join them behind one
// barrier, while the next segment's queries are on their way.
//
// Measured (bf16, share of the copy rate): 131072 keys of one sequence, Hq32 Hkv8 D128, 51.8 us
// (77%; the kernel alone 45.8, its first 1.5 the shares, the join 5); 64 sequences of up to
// 8000 keys 93.4 (85%); D 256, 8 sequences of 8192 keys 53 (74%); D 64, of 16384 keys 37 (54%:
// half the bytes per tile, so instructions bound it).
template <int D_, int NT_, bool BF16_>
struct Paged8Cfg {
  static constexpr int D = D_, NT = NT_, RW = 1;
  static constexpr bool BF16 = BF16_, E8 = true, CLUSTER = false, WINDOW = true, SINKS = true;
  static constexpr int KW = kPagedKeyWarps, ROWS = 8 * NT;
  static constexpr int GROUPS = D == 256 ? (NT == 1 ? 2 : 1) : NT == 1 ? 3 : 2;
  static constexpr int WARPS = KW, GROUP_THREADS = 32 * (KW + 1);  // of a group: consumers, and with the producer
  static constexpr int THREADS = (GROUPS * GROUP_THREADS + 127) / 128 * 128;
  static constexpr int CTAS = GROUPS;  // shares per SM
  static constexpr int PRODUCERS = 1;
  static constexpr int COLS = 128, KREG = (D + COLS - 1) / COLS;
  static constexpr int REGION = kPagedTile * 128, TILE = KREG * REGION;
  static constexpr int STAGES = D == 256 ? (NT == 1 ? 2 : 3) : NT == 1 ? 3 : 4;
  static constexpr bool QREG = NT * D <= 128;
  static constexpr int QREGION = ROWS * 128, QREGS = (D + 63) / 64;
  static constexpr int OP = D + 4;
  // A unit's beginning and end take as long as two of a group's tiles (64 ragged sequences 104
  // us when they count for nothing, 98 for one, 95 for two; 128 of half the length 113, 102, 96).
  static constexpr int OVER = kOver8;
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = OFF_KV + STAGES * 2 * TILE;
  static constexpr int OFF_O = OFF_Q + QREGS * QREGION;  // the warps' rows side by side
  static constexpr int OFF_ML = OFF_O + KW * ROWS * OP * 4;
  static constexpr int GROUP_BYTES = (OFF_ML + KW * ROWS * 8 + 1023) / 1024 * 1024;
  static constexpr int SMEM_BYTES = GROUPS * GROUP_BYTES + 1024;
  static_assert(SMEM_BYTES <= 225000, "shared memory");  // beside the static variables
};

// The shares of a CTA's groups, found by all its threads: as find_share, for part
// GROUPS * blockIdx.x + g of group g. The caller's group gets its own, and its window filled.
template <class C>
__device__ __forceinline__ Share find_shares8(const PagedFwdArgs& p, const ListShape& list, int parts, int group,
                                              ItemLens (*slots)[kItemWindow]) {
  __shared__ int sums[C::THREADS / 32];
  __shared__ int found_rest[C::GROUPS], found_item[C::GROUPS];
  const int per = (list.items + C::THREADS - 1) / C::THREADS;
  const int i0 = min(list.items, static_cast<int>(threadIdx.x) * per), i1 = min(list.items, i0 + per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool whole = list.items <= kItemWindow;  // the windows hold the list: one item per thread
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    const ItemLens x = load_lens(p, i);
    if (whole) {
#pragma unroll
      for (int g = 0; g < C::GROUPS; ++g) slots[g][i] = x;
    }
    mine += unit_places(list, make_item(list, x)) * list.mult;
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  if (threadIdx.x < C::GROUPS) found_item[threadIdx.x] = found_rest[threadIdx.x] = 0;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  Share own;
#pragma unroll
  for (int g = 0; g < C::GROUPS; ++g) {
    Share s;
    s.divide(total, C::GROUPS * blockIdx.x + g, parts);
    if (s.lo >= before && s.lo < before + mine) {
      int rest = s.lo - before;
      int i = i0;
      for (; i < i1 - 1; ++i) {
        const int n = unit_places(list, make_item(list, load_lens(p, i))) * list.mult;
        if (rest < n) break;
        rest -= n;
      }
      found_item[g] = i;
      found_rest[g] = rest;
    }
    if (g == group) own = s;
  }
  __syncthreads();
  own.item = found_item[group];
  own.rest = found_rest[group];
  if (!whole) {  // (a read of the lengths per group, agreed on by its warps)
    for (int i = threadIdx.x; i < C::GROUPS * kItemWindow; i += C::THREADS) {
      const int g = i / kItemWindow, item = found_item[g] + i - g * kItemWindow;
      if (item < list.items) slots[g][i - g * kItemWindow] = load_lens(p, item);
    }
    __syncthreads();
  }
  return own;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
fa_paged8_split_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const PagedFwdArgs p, int parts) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[C::GROUPS][C::STAGES], empty[C::GROUPS][C::STAGES];
  __shared__ int key_pos[C::GROUPS][C::STAGES][C::KW];      // of each warp's 16 keys
  __shared__ float2 kv_scale[C::GROUPS][C::STAGES][C::KW];  // of their page
  __shared__ float row_scale[C::GROUPS][C::ROWS];
  __shared__ ItemLens item_lens[C::GROUPS][kItemWindow];
  __shared__ int abort_flag;
  constexpr int D = C::D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps: the groups' consumers, then their producers
  const bool consumer = warp < C::GROUPS * C::KW;
  const int group = consumer ? warp / C::KW : min(warp - C::GROUPS * C::KW, C::GROUPS - 1), kw = warp % C::KW;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u) + group * C::GROUP_BYTES;
  const uint32_t sbase = smem_u32(smem);
  ListShape list = list_shape<C>(p);
  list.over = C::OVER;
  const int part = C::GROUPS * blockIdx.x + group;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int g = 0; g < C::GROUPS; ++g)
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(smem_u32(&full[g][i]), 1 + C::KW);  // the tile, and the scales of each 16 keys
        mbar_init(smem_u32(&empty[g][i]), C::KW);
      }
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * C::GROUPS * C::KW) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  grid_wait_prior();
  grid_release_next();
  prefetch_inputs<C>(p, blockIdx.x);
  const Share share = find_shares8<C>(p, list, parts, group, item_lens);  // barriers inside
  if (warp >= C::GROUPS * (C::KW + 1) || part >= parts) return;
  ItemWindow<C::GROUP_THREADS> window{p, item_lens[group], list.items, list.items <= kItemWindow ? 0 : share.item,
                                      4 + group, consumer ? 32 * kw + lane : 32 * C::KW + lane};
  if (!consumer) {
    TileRing<C> ring(p, map_k, map_v, sbase + C::OFF_KV, full[group], empty[group], key_pos[group], &abort_flag, 0,
                     kv_scale[group]);
    produce_share<C>(p, list, share, window, ring);
    ring.drain();
    return;
  }
  const int tid = 32 * kw + lane;  // of the group's consumers
  float* om = reinterpret_cast<float*>(smem + C::OFF_O);
  float2* mls = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [KW][ROWS]
  auto sync_rows = [&] { named_bar_sync(1 + group, 32 * C::KW); };
  if (tid == 0 && !p.by_unit) p.joins[part] = make_int2(-1, 0);
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  Walk w;
  bool more = w.start(list, share, window);
  QueryRows<C> ahead;  // of the segment to come
  auto load_ahead = [&] {
    const int rb = row_block(p, w);
    ahead.load(p, block_row0(p, item_seq(p, w.item), kv_head(p, w), rb, C::ROWS), min(C::ROWS, p.rows - rb * C::ROWS), kw,
               lane);
  };
  if (more) load_ahead();
  while (more) {
    const int rb = row_block(p, w), rows = min(C::ROWS, p.rows - rb * C::ROWS);
    const int64_t row0 = block_row0(p, item_seq(p, w.item), kv_head(p, w), rb, C::ROWS);
    // this thread's columns are rows 2 (lane % 4) and the next of each group of 8
    const int col0 = 2 * (lane & 3);
    uint64_t tokens = 0;  // of this thread's rows, four bits each
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        tokens |= static_cast<uint64_t>((rb * C::ROWS + col0 + 8 * nt + e) % p.Tq) << (8 * nt + 4 * e);
    ahead.store(smem + C::OFF_Q, row_scale[group], kw, lane);
    sync_rows();
    const uint32_t qs = sbase + C::OFF_Q;
    auto query_frag = [&](uint32_t (&f)[4], int nt, int k2) {
      const int row = nt * 8 + (lane & 7), ch = 4 * k2 + (lane >> 3);
      ldsm4(f, qs + (ch >> 3) * C::QREGION + sw128_offset(row, ch & 7));
    };
    uint32_t qf[C::QREG ? C::NT : 1][C::QREG ? D / 32 : 1][4];
    if constexpr (C::QREG) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) query_frag(qf[nt][k2], nt, k2);
    }
    auto query = [&](uint32_t (&b)[4], int nt, int k2) {
      if constexpr (C::QREG) {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = qf[nt][k2][e];
      } else {
        query_frag(b, nt, k2);
      }
    };
    float2 rs[C::NT];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
      rs[nt] = make_float2(row_scale[group][col0 + 8 * nt], row_scale[group][col0 + 8 * nt + 1]);
    float m[C::NT][2], l[C::NT][2], acc[C::NT][D / 16][4], unit = 0.f;
    bool large = false;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoMax;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }
    const int len = w.it.len, n = w.it.n, p_lo = len - n;
    for (int t = w.t0; t < w.t1; ++t) {
      ok = ok && mbar_wait(smem_u32(&full[group][slot]), phase, p.wc.timeout_cycles, &abort_flag, p.wc.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int at_keys = key_pos[group][slot][kw], j0 = at_keys & ~kSeenByAll;
      const bool all = at_keys < 0;
      if (all || (j0 < len && !(p.window > 0 && j0 + 15 <= p_lo - p.window && j0 >= p.sinks))) {
        const uint32_t ks = sbase + C::OFF_KV + slot * 2 * C::TILE + kw * 16 * 128;
        step8<C, C::REGION>(p, ks, ks + C::TILE, lane, kv_scale[group][slot][kw], j0, all, len, n, tokens, query, rs, m, l,
                            acc, unit, large);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[group][slot]));
      if (++slot == C::STAGES) {
        slot = 0;
        phase ^= 1;
      }
    }
    // the warps' maxima and sums, and their rows side by side
    const float out = unit * (1.f / kWeightLift);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float& x = l[nt][h];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        // padding rows (tokens the sequence does not have) see nothing; a row that has
        // met nothing but NaN keeps it
        if ((static_cast<int>(tokens >> (8 * nt + 4 * h)) & 15) >= n || (m[nt][h] == kNoMax && x == 0.f)) {
          m[nt][h] = -INFINITY;
          x = 0.f;
        }
        if (lane < 4) mls[kw * C::ROWS + col0 + 8 * nt + h] = make_float2(m[nt][h], x);
      }
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          om[(kw * C::ROWS + col0 + 8 * nt + (e & 1)) * C::OP + acc_column<C>(i, lane, e)] = acc[nt][i][e] * out;
    const Walk done = w;
    more = w.next(list, window);
    if (more) load_ahead();
    sync_rows();  // (the next segment's first barrier comes before anybody writes here again)
    const bool begins = done.t0 == 0, ends = done.t1 == done.it.tiles;
    for (int i = tid; i < rows * (D / 8); i += 32 * C::KW) {
      const int r = i / (D / 8), ch = i - r * (D / 8);
      const float2 ml = warps_max_sum<C>(mls, r);
      float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
#pragma unroll
      for (int k = 0; k < C::KW; ++k) {
        const float mk = mls[k * C::ROWS + r].x;
        if (mk == -INFINITY) continue;  // nothing seen: not even 0 * inf
        const float f = ex2(mk - ml.x);
        const float* x = om + (k * C::ROWS + r) * C::OP + 8 * ch;
        add4(s0, *reinterpret_cast<const float4*>(x), f);
        add4(s1, *reinterpret_cast<const float4*>(x + 4), f);
      }
      put_piece<C>(p, begins && ends, 2 * part + (begins ? 1 : 0), row0, r, ch, s0, s1, ml);
    }
    if (tid == 0) record_unit(p, list, share, done, part);
  }
  write_empty_units<C>(p, list, part, parts, tid, 32 * C::KW);
}

}  // namespace fa
