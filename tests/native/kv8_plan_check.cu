// Prints the launch plans of the norm and 8-bit cache kernels for many shapes,
// one line each (key=value), for tests/test_kv8_plan.py.
#include <cstdio>

#include "sas_internal.h"

int main() {
  const int heads[][2] = {{1, 1}, {8, 1}, {32, 8}, {40, 8}, {64, 8}, {4096, 512}, {32, 0}, {0, 8}};
  const long long tokens[] = {1, 7, 31, 32, 33, 1000, 8168, 65536, 1 << 20, 1 << 29};
  for (auto& h : heads)
    for (long long n : tokens)
      for (int back = 0; back < 2; ++back) {
        const sas::NormRopeGrid g = sas::norm_rope_grid(1, static_cast<int>(n), h[0], h[1], back != 0);
        std::printf("kind=0 hq=%d hkv=%d n=%lld back=%d x=%d chunk=%d qc=%d kc=%d scratch=%zu\n", h[0], h[1], n, back,
                    g.x, g.chunk, g.q_chunks, g.k_chunks, sas::norm_rope_scratch_bytes());
      }
  const long long pairs[] = {1, 8, 37, 64, 128, 148, 512, 65535};
  const long long blocks[] = {1, 2, 4, 8, 16, 32, 128, 129, 512, 65535, 1 << 20};
  for (long long p : pairs)
    for (long long b : blocks)
      std::printf("kind=1 pairs=%lld blocks=%lld few=%d\n", p, b, sas::pool_few(p, b) ? 1 : 0);
  return 0;
}
