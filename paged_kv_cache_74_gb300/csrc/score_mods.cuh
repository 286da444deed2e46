// score_mods.cuh -- the modified scores of the masked attention calls: a tanh
// cap, a distance bias and a visible part of the keys (ScoreMods).
//
// A query at position p of a request with seq_len keys scores key j
//   y = cap log2(e) tanh(scale q.k / cap) - slope log2(e) |p - j|
// in log2 units (without a cap: scale log2(e) q.k) and sees it if
//   j < prefix  or  start <= j <= p.
#pragma once

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// cap log2(e) tanh(t), t = x cap_in: the odd Taylor polynomial below
// |t| = 0.3 (first term left out: 0.0089 t^10 relative, 6e-8), where 1 - 2 / (1 +
// e^2t) would lose the leading digits of a small score; that quotient above
// (2e-7 absolute, 7e-7 relative at 0.3).  The hardware's tanh
// approximation is off by 2^-11 of the score: a capped score of 30 would
// shift its weight by 1.5 %.
__device__ __forceinline__ float capped_score(float x, const ScoreMods& m) {
  const float t = x * m.cap_in;
  const float t2 = t * t;
  float q = fmaf(t2, 62.f / 2835.f, -17.f / 315.f);
  q = fmaf(t2, q, 2.f / 15.f);
  q = fmaf(t2, q, -1.f / 3.f);
  const float small = fmaf(t * t2, q, t);
  const float e = fast_exp2(t * (2.f * kLog2e));  // 0 and infinity at the ends are fine
  const float big = fmaf(-2.f, fast_rcp(1.f + e), 1.f);
  return m.cap_log2 * (t2 < 0.09f ? small : big);
}

// The same for a pair of scores with |t| <= kCapNear, on the fused multiply-add
// pipe alone: cap log2(e) t Q(t^2), Q the minimax polynomial of tanh(t) / t in
// t^2 for |t| <= 1 (5e-8 relative, 2e-7 with fp32 evaluation).
constexpr float kCapNear = 1.0f;
constexpr float kTanhQ0 = 0.99999994f, kTanhQ1 = -0.3333284f, kTanhQ2 = 0.13325204f,
                kTanhQ3 = -0.05345703f, kTanhQ4 = 0.020289982f, kTanhQ5 = -0.0062033795f,
                kTanhQ6 = 0.0010410226f;

__device__ __forceinline__ float2 capped_near(float2 x, const ScoreMods& m) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 t = __fmul2_rn(x, both(m.cap_in));
  const float2 t2 = __fmul2_rn(t, t);
  float2 q = __ffma2_rn(t2, both(kTanhQ6), both(kTanhQ5));
  q = __ffma2_rn(t2, q, both(kTanhQ4));
  q = __ffma2_rn(t2, q, both(kTanhQ3));
  q = __ffma2_rn(t2, q, both(kTanhQ2));
  q = __ffma2_rn(t2, q, both(kTanhQ1));
  q = __ffma2_rn(t2, q, both(kTanhQ0));
  return __fmul2_rn(__fmul2_rn(t, both(m.cap_log2)), q);
}

// The 16-token tiles of a request that hold a key its (single) row sees:
// tiles [0, n1) and [n1 + gap, n1 + gap + nb - n1).
struct TileSpan {
  int n1, gap, nb;
  int prefix, start;  // clipped to [0, seq_len]
  bool empty;         // no visible key: one tile without data
  __device__ __forceinline__ int tile(int t) const { return t < n1 ? t : t + gap; }
};

__device__ __forceinline__ TileSpan make_span(int len, int prefix, int start) {
  TileSpan s;
  s.prefix = min(max(prefix, 0), len);
  s.start = min(max(start, 0), len);
  const int total = (len + kBlockSize - 1) / kBlockSize;
  s.n1 = (s.prefix + kBlockSize - 1) / kBlockSize;
  const int second = max(s.n1, s.start < len ? s.start / kBlockSize : total);
  s.gap = second - s.n1;
  s.nb = s.n1 + total - second;
  s.empty = s.nb == 0;
  if (s.empty) {
    s.nb = 1;
    s.gap = 0;
  }
  return s;
}

// The tiles of request r (one query row at `row`, `len` keys).
__device__ __forceinline__ TileSpan tile_span(const ScoreMods& m, int r, int row, int len) {
  return make_span(len, m.prefix_lens != nullptr ? __ldg(m.prefix_lens + r) : 0,
                   m.key_starts != nullptr ? __ldg(m.key_starts + row) : 0);
}

// Whether the row at the last position sees key t; vis = {prefix, start}.
__device__ __forceinline__ bool sees_key(int t, int seq_len, int2 vis) {
  return t < seq_len && (t < vis.x || t >= vis.y);
}

}  // namespace
}  // namespace pa
