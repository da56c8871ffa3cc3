// What the two kinds of fa_kv_append share: rows in units that close over their rotation
// pairs, the rotation, and the place of a sequence's new tokens.
#pragma once

#include "fa_inst.cuh"
#include "fa_paged_launch.h"

namespace fa {

struct AppendArgs {
  PagedView c;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  TokenStrides ks, vs, qs;
  int Hq, T;
  const int* new_lens;
  const float *cos_table, *sin_table;
  int rope_len, rot_dim, interleaved;
};

// The two 16-byte chunks of unit u of a row: element offsets.
struct UnitPos {
  int a, b;
  bool rotated;
};
__device__ __forceinline__ UnitPos unit_pos(const AppendArgs& p, int u) {
  UnitPos r;
  r.rotated = 16 * u < p.rot_dim;
  const bool halves = r.rotated && !p.interleaved;
  r.a = halves ? 8 * u : 16 * u;
  r.b = halves ? 8 * u + p.rot_dim / 2 : 16 * u + 8;
  return r;
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles load_angles(const AppendArgs& p, int pos, int u) {
  Angles g;
  const int64_t at = static_cast<int64_t>(pos) * (p.rot_dim / 2) + 8 * u;
  const float4* c = reinterpret_cast<const float4*>(p.cos_table + at);
  const float4* s = reinterpret_cast<const float4*>(p.sin_table + at);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 x = c[i], y = s[i];
    g.c[4 * i] = x.x; g.c[4 * i + 1] = x.y; g.c[4 * i + 2] = x.z; g.c[4 * i + 3] = x.w;
    g.s[4 * i] = y.x; g.s[4 * i + 1] = y.y; g.s[4 * i + 2] = y.z; g.s[4 * i + 3] = y.w;
  }
  return g;
}

// Rotate a unit in place (fp32 arithmetic, one rounding per value).
template <bool BF16>
__device__ __forceinline__ void rotate_unit(uint4& a, uint4& b, const Angles& g, bool interleaved) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF16>(wa[i]), y = unpack2<BF16>(wb[i]);
    if (interleaved) {  // pairs (x.x, x.y) and (y.x, y.y)
      wa[i] = pack2<BF16>(x.x * g.c[i] - x.y * g.s[i], x.y * g.c[i] + x.x * g.s[i]);
      wb[i] = pack2<BF16>(y.x * g.c[4 + i] - y.y * g.s[4 + i], y.y * g.c[4 + i] + y.x * g.s[4 + i]);
    } else {  // pairs (x.x, y.x) and (x.y, y.y)
      const float c0 = g.c[2 * i], c1 = g.c[2 * i + 1], s0 = g.s[2 * i], s1 = g.s[2 * i + 1];
      wa[i] = pack2<BF16>(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
      wb[i] = pack2<BF16>(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
    }
  }
}

struct Unit {
  uint4 a, b;
};
__device__ __forceinline__ Unit load_unit(const uint16_t* src, const UnitPos& at) {
  return {*reinterpret_cast<const uint4*>(src + at.a), *reinterpret_cast<const uint4*>(src + at.b)};
}
__device__ __forceinline__ void store_unit(uint16_t* dst, const UnitPos& at, const Unit& x) {
  *reinterpret_cast<uint4*>(dst + at.a) = x.a;
  *reinterpret_cast<uint4*>(dst + at.b) = x.b;
}

// The new tokens of a sequence that have a place: [t0, t1) of its rows, token t at
// position first + t.
struct NewTokens {
  int first, t0, t1;
};
__device__ __forceinline__ NewTokens new_tokens(const AppendArgs& p, int b) {
  const SeqLens sl = seq_lens(p.c, p.new_lens, b, p.T);
  NewTokens r;
  r.first = sl.len - sl.n;
  r.t0 = max(0, -r.first);
  r.t1 = p.rot_dim > 0 ? min(sl.n, p.rope_len - r.first) : sl.n;
  if (r.t0 > 0 || r.t1 < sl.n) flag_bad_index(p.c);
  return r;
}


// Up to this many new tokens per sequence count as few.
constexpr int kFewTokens = 8;

inline AppendArgs append_args(const AppendLaunch& a) {
  AppendArgs p;
  p.c = a.c;
  p.k = a.k; p.v = a.v; p.q = a.q;
  p.q_out = a.q_out;
  p.ks = a.ks; p.vs = a.vs; p.qs = a.qs;
  p.Hq = a.q != nullptr ? a.Hq : 0;
  p.T = a.T;
  p.new_lens = a.new_lens;
  p.cos_table = a.cos_table; p.sin_table = a.sin_table;
  p.rope_len = a.rope_len; p.rot_dim = a.rot_dim; p.interleaved = a.interleaved;
  return p;
}

}  // namespace fa
