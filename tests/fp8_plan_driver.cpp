// Command-line driver of the kernel choice of block-scaled e4m3 products
// (csrc/ar_fp8_plan.h): reads lines "<by expert> <wide> <R> <N> <K> <E>" on stdin and prints
// "<kind> <K sets>" for each.
#include <cstdio>

#include "../autoround_signsgd_rounding_amd/csrc/ar_fp8_plan.h"

int main() {
  static const char* const names[] = {"rows", "32x64", "64x64", "64x128", "128x128", "256x256"};
  int grouped, wide;
  long long R, N, K, E;
  while (std::scanf("%d %d %lld %lld %lld %lld", &grouped, &wide, &R, &N, &K, &E) == 6) {
    const ArFp8Plan p = ar_fp8_plan(ArFp8Shape{grouped != 0, wide != 0, R, N, K, E});
    std::printf("%s %d\n", names[p.kind], p.two ? 2 : 1);
  }
  return 0;
}
