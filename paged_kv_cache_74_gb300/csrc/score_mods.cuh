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

// tanh(t) / t for |t| <= kCapNear as a polynomial in t^2, minimax in the relative
// error (6e-7).  Up to there 1 - 2 / (1 + e^2t) would lose leading digits, and
// two special-function operations cost more than five fused multiply-adds.
constexpr float kCapNear = 0.75f;
constexpr float kTanhQ0 = 0.99999946f, kTanhQ1 = -0.33328253f, kTanhQ2 = 0.13258983f,
                kTanhQ3 = -0.050056305f, kTanhQ4 = 0.012929632f;

// cap log2(e) tanh(t), t = x cap_in, for any x: the polynomial near 0, the
// quotient beyond (2e-7 absolute).  The hardware's tanh approximation is off by
// 2^-11 of the score: a capped score of 30 would shift its weight by 1.5 %.
__device__ __forceinline__ float capped_score(float x, const ScoreMods& m) {
  const float t = x * m.cap_in;
  const float t2 = t * t;
  float q = fmaf(t2, kTanhQ4, kTanhQ3);
  q = fmaf(t2, q, kTanhQ2);
  q = fmaf(t2, q, kTanhQ1);
  q = fmaf(t2, q, kTanhQ0);
  const float e = fast_exp2(t * (2.f * kLog2e));  // 0 and infinity at the ends are fine
  const float far = fmaf(-2.f, fast_rcp(1.f + e), 1.f);
  return m.cap_log2 * (t2 < kCapNear * kCapNear ? t * q : far);
}

// The same for a pair of scores with |t| <= kCapNear, by packed fused
// multiply-adds (cap_log2 folded into the coefficients).
__device__ __forceinline__ float2 capped_near(float2 x, const ScoreMods& m) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 t = __fmul2_rn(x, both(m.cap_in));
  const float2 t2 = __fmul2_rn(t, t);
  float2 q = __ffma2_rn(t2, both(kTanhQ4 * m.cap_log2), both(kTanhQ3 * m.cap_log2));
  q = __ffma2_rn(t2, q, both(kTanhQ2 * m.cap_log2));
  q = __ffma2_rn(t2, q, both(kTanhQ1 * m.cap_log2));
  q = __ffma2_rn(t2, q, both(kTanhQ0 * m.cap_log2));
  return __fmul2_rn(t, q);
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
