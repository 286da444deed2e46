// Host-side checks of the SM split of a masked mixed batch (masked_tile_sms).
// Runs on the CPU only; prints "ok" or the first violation.
#include <cstdio>

#include "work_split.cuh"

using namespace pa;

static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("FAIL %s %lld %lld %lld\n", what, a, b, c);
  return 1;
}

int main() {
  for (int sms : {1, 2, 8, 152})
    for (int e4m3 = 0; e4m3 < 2; ++e4m3) {
      const bool f8 = e4m3 != 0;
      if (masked_tile_sms(0, 1000, sms, f8) != 0) return fail("no tile work", sms, 0, 0);
      if (masked_tile_sms(1000, 0, sms, f8) != sms) return fail("no decode rows", sms, 0, 0);
      const long long tw = f8 ? kMaskedTileNsPerCost8 : kMaskedTileNsPerCost;
      const long long dw = f8 ? kDecodeNsPerTile8 : kDecodeNsPerTile;
      if (masked_tile_sms(kSplitMaxTileNsPerSm * sms / tw + 1000, 1, sms, f8) != sms)
        return fail("large tile batch", sms, 0, 0);
      // No other number of SMs ends earlier by the model.
      for (long long tc = 1; tc < 30000; tc = tc * 3 / 2 + 7)
        for (long long dt = 1; dt < 400000; dt = dt * 2 + 3) {
          const long long t = tc * tw, d = dt * dw;
          if (t > kSplitMaxTileNsPerSm * sms) continue;
          if (sms < 2) continue;
          auto end = [&](int n) -> long long {
            const long long a = t / n, b = d / (sms - n);
            return a > b ? a : b;
          };
          const int n = masked_tile_sms(tc, dt, sms, f8);
          if (n < 1 || n >= sms) return fail("range", tc, dt, n);
          for (int m = 1; m < sms; ++m)
            if (end(m) < end(n)) return fail("earlier end", tc, dt, m);
          if (decode_split_ctas(n, sms, 3 * sms, 3) < 3) return fail("no decode CTAs", tc, dt, n);
        }
    }
  std::printf("ok\n");
  return 0;
}
