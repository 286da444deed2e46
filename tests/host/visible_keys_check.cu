// Host-side checks of PVis and PVisBrief (which keys, blocks and steps a masked query tile
// needs) against the definition, key by key.  Runs on the CPU only; prints
// "ok" or the first violation.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "visible_keys.cuh"

using namespace pa;

static unsigned state = 12345u;
static int rnd(int n) {
  state = state * 1664525u + 1013904223u;
  return static_cast<int>((state >> 8) % static_cast<unsigned>(n));
}

int main() {
  for (int trial = 0; trial < 60000; ++trial) {
    const int rows = trial % 3 == 0 ? 128 : 1 + rnd(128);
    const int own = rnd(4) == 0 ? 16 * rnd(30) : rnd(500);
    const int len = own + rows;
    const int prefix = rnd(3) == 0 ? rnd(len + 1) : 0;
    std::vector<int> start(rows);
    const int kind = rnd(5);
    int doc = rnd(own + 1);
    for (int i = 0; i < rows; ++i) {
      if (kind == 0) start[i] = rnd(own + rows + 30);
      if (kind == 1) start[i] = own + i - rnd(40);
      if (kind == 2) start[i] = rnd(3) ? own + i + 1 + rnd(9) : own + i;
      if (kind == 3) start[i] = rnd(30) ? doc : (doc = own + i + 1);
      if (kind == 4) start[i] = (i / 40) % 2 ? own + i + 1 : own + (i / 40) * 40;
      if (start[i] < 0) start[i] = 0;
    }
    // the definition
    std::vector<char> seen(len + 300, 0);
    int lo = 0x7fffffff, hi = 0;
    for (int i = 0; i < rows; ++i)
      for (int j = start[i]; j <= own + i; ++j) {
        seen[j] = 1;
        if (j < lo) lo = j;
        if (j + 1 > hi) hi = j + 1;
      }
    PVis v{};
    v.prefix = prefix;
    v.lo = lo;
    v.hi = hi;
    bool holes = false;
    for (int j = lo; j < hi; ++j) holes |= !seen[j];
    for (int k = 0; k < 128; ++k)
      if (own + k < len && seen[own + k]) v.seen[k / 32] |= 1u << (k & 31);
    v.own = holes ? own : kNoHoles;
    v.blocks = 0xffffffffu;
    if (holes) {
      v.blocks = 0;
      for (int b = 0; b < 9; ++b)
        if (own_block_seen(v.seen, own, lo, b)) v.blocks |= 1u << b;
    }
    v.n1 = (prefix + 127) / 128;
    const int second = hi > 0 ? (lo / 128 > v.n1 ? lo / 128 : v.n1) : v.n1;
    v.gap = second - v.n1;
    for (int j = 0; j < prefix; ++j) seen[j] = 1;
    for (int t = 0; t < len + 200; ++t)
      if (v.key(t) != (seen[t] != 0)) {
        std::printf("FAIL key %d of trial %d\n", t, trial);
        return 1;
      }
    for (int t = 0; t < len + 200; t += 16) {
      bool any = false;
      for (int j = t; j < t + 16; ++j) any |= seen[j] != 0;
      if (v.block(t) != any) {
        std::printf("FAIL block %d of trial %d\n", t, trial);
        return 1;
      }
    }
    for (int t = 0; t < len + 100; t += 128) {
      bool every = true;
      for (int j = t; j < t + 128; ++j) every &= seen[j] != 0;
      if (PVisBrief(v).all(t, 128) && !every) {
        std::printf("FAIL all %d of trial %d\n", t, trial);
        return 1;
      }
      if (!holes && PVisBrief(v).all(t, 128) != every) {
        std::printf("FAIL all (no holes) %d of trial %d\n", t, trial);
        return 1;
      }
    }
    // Every step of the map but that of a tile that sees nothing holds a seen
    // key, and every seen key lies in a step of the map.
    int steps = v.n1 + ((hi + 127) / 128 > second ? (hi + 127) / 128 - second : 0);
    std::vector<char> covered(len + 300, 0);
    for (int j = 0; j < steps; ++j) {
      bool any = false;
      if (PVisBrief(v).tile(j) != v.tile(j)) {
        std::printf("FAIL tile %d of trial %d\n", j, trial);
        return 1;
      }
      for (int t = 128 * v.tile(j); t < 128 * v.tile(j) + 128; ++t) {
        if (t < len + 300) covered[t] = 1;
        any |= t < len && seen[t];
      }
      if (!any) {
        std::printf("FAIL empty step %d of trial %d\n", j, trial);
        return 1;
      }
    }
    for (int t = 0; t < len; ++t)
      if (seen[t] && !covered[t]) {
        std::printf("FAIL key %d in no step, trial %d\n", t, trial);
        return 1;
      }
  }
  std::printf("ok\n");
  return 0;
}
