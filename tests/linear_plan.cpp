// The variant, split, ring depth and row tile that a matrix product takes, on
// the host: reads "M N K e4m3 gated whole" per line.
#include "kda_linear_plan.h"

#include <cstdio>

int main() {
  long M, N, K;
  int e4m3, gated, whole;
  for (const Variant& v : kVariants)
    std::printf("%d %d %d %d %d %d %d %d %d\n", v.rows, v.unit, v.channels, v.pair, v.interleaved, v.threads, v.stage_bytes, v.part_bytes, v.head_bytes);
  std::printf("-\n");
  while (std::scanf("%ld %ld %ld %d %d %d", &M, &N, &K, &e4m3, &gated, &whole) == 6) {
    const long bytes = K * (e4m3 ? 1 : 2);
    const Plan p = plan_of(static_cast<int>(M), static_cast<int>(gated ? N / 2 : N), static_cast<int>((bytes + kBlock - 1) / kBlock), gated != 0,
                           static_cast<double>(bytes) * N, 152, whole != 0);
    std::printf("%d %d %d %d\n", p.variant, p.split, p.stages, p.tile_rows);
  }
}
