// score_mods.cuh -- the modified scores of the masked attention calls: a tanh
// cap, a distance bias and a visible part of the keys (ScoreMods).
//
// A query at position p of a request with seq_len keys scores key j
//   y = cap log2(e) tanh(scale q.k / cap) - slope log2(e) |p - j|
// in log2 units (without a cap: scale log2(e) q.k) and sees it if
//   j < prefix  or  start <= j <= p.
#pragma once

#include "decode_common.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

// Which scores an instantiation computes: plain ones, modified, or also capped.
constexpr int kNoMods = 0;
constexpr int kMods = 1;
constexpr int kModsCap = 2;

constexpr float kLog2e = 1.4426950408889634f;

// tanh(t) / t for |t| <= kCapNear as a polynomial in t^2, minimax in the relative
// error (6e-7).  Up to there 1 - 2 / (1 + e^2t) would lose leading digits, and
// two special-function operations cost more than five fused multiply-adds.
constexpr float kCapNear = 0.75f;
constexpr float kTanhQ0 = 0.99999946f, kTanhQ1 = -0.33328253f, kTanhQ2 = 0.13258983f,
                kTanhQ3 = -0.050056305f, kTanhQ4 = 0.012929632f;

// cap log2(e) tanh(t) - ref, t = x cap_in, for any x: the polynomial near 0 (its
// coefficients times cap_log2), the quotient beyond (2e-7 absolute).  The
// hardware's tanh approximation is off by 2^-11 of the score: a capped score of
// 30 would shift its weight by 1.5 %.
__device__ __forceinline__ float capped_score(float x, const ScoreMods& m, float ref = 0.f) {
  const float t = x * m.cap_in;
  const float t2 = t * t;
  float q = fmaf(t2, kTanhQ4 * m.cap_log2, kTanhQ3 * m.cap_log2);
  q = fmaf(t2, q, kTanhQ2 * m.cap_log2);
  q = fmaf(t2, q, kTanhQ1 * m.cap_log2);
  q = fmaf(t2, q, kTanhQ0 * m.cap_log2);
  const float e = fast_exp2(t * (2.f * kLog2e));  // 0 and infinity at the ends are fine
  const float far = fmaf(-2.f, fast_rcp(1.f + e), 1.f);
  return t2 <= kCapNear * kCapNear ? fmaf(t, q, -ref) : fmaf(m.cap_log2, far, -ref);
}

// The same where a lane's scores stand alone, without ref: the coefficients as
// immediates (115 -> 113 us for the 8B-shaped decode batch; from the launch's
// parameters they took 123).
__device__ __forceinline__ float capped_alone(float x, const ScoreMods& m) {
  const float t = x * m.cap_in;
  const float t2 = t * t;
  float q = fmaf(t2, kTanhQ4, kTanhQ3);
  q = fmaf(t2, q, kTanhQ2);
  q = fmaf(t2, q, kTanhQ1);
  q = fmaf(t2, q, kTanhQ0);
  const float e = fast_exp2(t * (2.f * kLog2e));
  const float far = fmaf(-2.f, fast_rcp(1.f + e), 1.f);
  return m.cap_log2 * (t2 <= kCapNear * kCapNear ? t * q : far);
}

// Scores as floats or as their bits (as TMEM loads leave them).
__device__ __forceinline__ float as_float(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ void put_float(uint32_t& x, float v) { x = __float_as_uint(v); }
__device__ __forceinline__ void put_float(float& x, float v) { x = v; }

// The same for N pairs of scores with |t| <= kCapNear, in place and less `ref`, by
// packed fused multiply-adds, bit for bit what capped_score gives (so that it
// does not matter to a score which of the two its neighbours call for); the
// pairs go through the polynomial side by side, so that none waits for its own
// last step.
template <int N, typename T>
__device__ __forceinline__ void capped_near(T* r, const ScoreMods& m, float ref) {
  auto both = [](float c) { return make_float2(c, c); };
  const float qs[5] = {kTanhQ0 * m.cap_log2, kTanhQ1 * m.cap_log2, kTanhQ2 * m.cap_log2,
                       kTanhQ3 * m.cap_log2, kTanhQ4 * m.cap_log2};
  float2 t[N], t2[N], q[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    t[i] = __fmul2_rn(make_float2(as_float(r[2 * i]), as_float(r[2 * i + 1])), both(m.cap_in));
#pragma unroll
  for (int i = 0; i < N; ++i) t2[i] = __fmul2_rn(t[i], t[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = __ffma2_rn(t2[i], both(qs[4]), both(qs[3]));
#pragma unroll
  for (int k = 2; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __ffma2_rn(t2[i], q[i], both(qs[k]));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __ffma2_rn(t[i], q[i], both(-ref));
    put_float(r[2 * i], q[i].x);
    put_float(r[2 * i + 1], q[i].y);
  }
}

// Whether some lane of the warp holds a score beyond kCapNear among its N (squared
// as capped_score squares it).
template <int N, typename T>
__device__ __forceinline__ bool any_far(const T* r, const ScoreMods& m) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < N; e += 2)
    top[(e / 2) % 4] = fmax3(top[(e / 2) % 4], fabsf(as_float(r[e])), fabsf(as_float(r[e + 1])));
  const float t = fmaxf(fmax3(top[0], top[1], top[2]), top[3]) * m.cap_in;
  return __any_sync(0xffffffffu, t * t > kCapNear * kCapNear);
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

// What a decode row's tiles follow from, read in one round of loads (two where
// the row comes from query_start_loc).
struct RowInfo {
  int len, q0, q1, prefix, start;
};
__device__ __forceinline__ RowInfo row_info(const DecodeArgs& a, int r) {
  RowInfo i{0, 0, 0, 0, 0};
  if (r >= a.num_seqs) return i;
  i.len = __ldg(a.seq_lens + r);
  int row = r;
  if (a.query_start_loc != nullptr) {
    i.q0 = __ldg(a.query_start_loc + r);
    i.q1 = __ldg(a.query_start_loc + r + 1);
    row = i.q0 >= 0 && i.q0 < a.total_q ? i.q0 : 0;
  }
  if (a.mods.prefix_lens != nullptr) i.prefix = __ldg(a.mods.prefix_lens + r);
  if (a.mods.key_starts != nullptr) i.start = __ldg(a.mods.key_starts + row);
  return i;
}

// Its tiles (0: not a decode row, or lengths out of range).
__device__ __forceinline__ int tiles_from(const DecodeArgs& a, int r, const RowInfo& i) {
  int len = 0, row = 0;
  return blocks_from(a, r, i.len, i.q0, i.q1, &len, &row) > 0 ? make_span(len, i.prefix, i.start).nb : 0;
}

// Whether the row at the last position sees key t; vis = {prefix, start}.
__device__ __forceinline__ bool sees_key(int t, int seq_len, int2 vis) {
  return t < seq_len && (t < vis.x || t >= vis.y);
}

}  // namespace
}  // namespace pa
