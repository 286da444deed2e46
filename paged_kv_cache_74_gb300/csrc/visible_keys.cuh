// visible_keys.cuh -- which keys of its request a 128-row query tile of a masked
// prefill needs: host and device arithmetic shared by the plan, the tile kernel
// and its host-side checks.
//
// Row i of the tile sits at position own + i and sees the keys of [0, prefix)
// and of [start_i, own + i] (none of the latter if start_i lies behind it).
// The runs of all rows cover [lo, hi), lo the least start of a row that sees
// something and hi the last such row's position + 1, but for holes: key own + k
// is seen by some row i >= k with start_i <= own + k or by none.  A key in
// [lo, own) has no hole: the row that starts at lo sees it.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {
namespace {

constexpr int kNoHoles = 0x7fffffff;

// Whether the b-th 16-token block of own / 16, own / 16 + 1, .. holds a key that
// some row sees (bit k of seen: key own + k; keys of [lo, own) are all seen).
PA_HD bool own_block_seen(const uint32_t (&seen)[4], int own, int lo, int b) {
  const int s = 16 * b - (own & 15);  // the block holds bits s .. s + 15
  if (s < 0) return lo < own || (seen[0] & ((1u << (s + 16)) - 1u)) != 0;
  // (selects rather than indexed loads: `seen` stays in registers)
  const int w = s >> 5;
  const uint32_t low = w == 0 ? seen[0] : w == 1 ? seen[1] : w == 2 ? seen[2] : w == 3 ? seen[3] : 0u;
  const uint32_t high = w == 0 ? seen[1] : w == 1 ? seen[2] : w == 2 ? seen[3] : 0u;
  return ((static_cast<uint64_t>(high) << 32 | low) >> (s & 31) & 0xffffu) != 0;
}

// The keys that some row of a unit with modified scores sees, and the map from
// its steps to 128-key tiles.
struct PVis {
  int prefix, lo, hi, n1;
  int gap;
  int own;           // position of the tile's first row, or kNoHoles: all of [lo, hi) is seen
  uint32_t blocks;   // with holes: bit b is own_block_seen(b)
  int pad;
  uint32_t seen[4];  // with holes: bit k is set if some row sees key own + k

  PA_HD int tile(int j) const { return j < n1 ? j : j + gap; }
  PA_HD bool key(int t) const {
    if (t < prefix) return true;
    if (t < lo || t >= hi) return false;
    return t < own || (seen[(t - own) >> 5] >> ((t - own) & 31) & 1u) != 0;
  }
  // A 16-token block with such a key, from its first key.
  PA_HD bool block(int t) const {
    const uint32_t b = static_cast<uint32_t>((t >> 4) - (own >> 4));
    return t < prefix || (t + 16 > lo && t < hi && (b > 8 || (blocks >> b & 1u)));
  }
};
static_assert(sizeof(PVis) == 48, "three 16-byte words");

// What the softmax warps keep of it in registers.
struct PVisBrief {
  int prefix, lo, solid, n1, gap;  // solid: no key of [lo, solid) is unseen
  PA_HD explicit PVisBrief(const PVis& v)
      : prefix(v.prefix), lo(v.lo), solid(v.hi < v.own ? v.hi : v.own), n1(v.n1), gap(v.gap) {}
  PA_HD int tile(int j) const { return j < n1 ? j : j + gap; }
  // Whether all keys t .. t + n - 1 are seen by some row (holes: not looked for behind solid).
  PA_HD bool all(int t, int n) const {
    return t + n <= prefix || (t + n <= solid && (t >= lo || prefix >= lo));
  }
};

}  // namespace
}  // namespace pa

#undef PA_HD
