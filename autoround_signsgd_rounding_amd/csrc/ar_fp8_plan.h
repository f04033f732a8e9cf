// Which kernel of ar_fp8_gemm.hip a block-scaled e4m3 product takes: arithmetic on the
// host, without HIP.
#pragma once

#include <math.h>
#include <stdint.h>

struct ArFp8Shape {
  bool grouped;   // by expert
  bool wide;      // float32 sums throughout (a float32 Y, or asked for)
  int64_t R, N, K, E;
};

// Which kernel: the one with the least estimated time, in us. A tile takes `step`
// of a CU per block of K when two workgroups share it, and `ends` for its prologue
// and epilogue (`gap` of it where W's streaming is the cost and the rest is hidden
// under it); with two K sets, which are taken when no CU gets a second workgroup,
// a workgroup takes `step2` for two blocks. Streaming from memory (5.3 TB/s
// measured; 12% less with two sets) and from the caches into LDS (14 TB/s; 12
// where rows of K bytes break the 64-byte sectors) bound the time from below.
// Measured (us), M x N x K, the rule's pick first:
//   16 x 4096 x 4096            rows                6.2   32x64, two sets 8.7, 32x64 10.6
//   16 x 11008 x 4096           32x64, two sets    10.3   32x64 10.9, 64x64, two sets 11.5
//   64 x 11008 x 4096           64x64, two sets    12.0   64x64 13.2, 32x64 14.4
//   512 x 4096 x 4096           64x128, two sets   15.2   64x128 17.2, 64x64 18.1
//   1024 x 4096 x 4096          128x128, two sets  22.4   64x128 24.3, 128x128 24.8
//   2048 x 4096 x 4096          128x128            37.2   128x128, two sets 43.9, 256x256 46.7
//   3806 x 2584 x 8656          256x256             111   128x128 137, 64x128 153
//   4096 x 4096 x 4096          256x256            58.9   128x128 75.2, 128x128, two sets 88.1
//   24 tokens, 4 of 64 experts, 2048 x 2048: 64x128 21.2; 32x64 23.2, 128x128 23.4
//   333 x 4096 x 4096, float32  64x128, two sets   22.1   64x64 24.7, 64x128 26.1
// Over 106 shapes, dense and by expert, with even and with very uneven routing, the
// pick takes 1.03 times the best one's time in the mean, and 1.53 times it at the most
// (50 rows of 100 experts, 500 x 800: 11.3 us by rows, 7.4 by 32x64 tiles). The rule
// knows how many experts and rows there are, not how the rows are spread. The float32
// form runs at half the matrix rate and on more registers: it has its own times, and
// no 256 x 256 tile.
enum ArFp8Kind { kRows, k32x64, k64x64, k64x128, k128x128, k256x256, kKinds };
struct ArFp8Times {
  int tm, tn;
  float step, ends, gap, step2;
};
inline const ArFp8Times& ar_fp8_times(bool wide, int kind) {
  static constexpr ArFp8Times times[2][kKinds] = {
      {{16, 16, 0, 0, 0, 0}, {32, 64, .1175f, 1.2f, .4f, .30f}, {64, 64, .1675f, 2.0f, .5f, .43f},
       {64, 128, .287f, 2.4f, .7f, .62f}, {128, 128, .456f, 3.0f, 1.1f, .92f},
       {256, 256, 1.52f, 9.0f, 9.0f, 0}},
      {{16, 16, 0, 0, 0, 0}, {32, 64, .2025f, 1.2f, .4f, .50f}, {64, 64, .28f, 2.0f, .5f, .72f},
       {64, 128, .505f, 2.4f, .7f, 1.12f}, {128, 128, .83f, 3.0f, 1.1f, 1.75f}, {}}};
  return times[wide][kind];
}

// Tiles of tm rows to expect: what E ranges of equal size need, and half a tile more
// for each where sizes differ.
inline double ar_fp8_expected_tiles(const ArFp8Shape& g, int tm) {
  if (!g.grouped) return (double)((g.R + tm - 1) / tm);
  const double used = (double)(g.E < g.R ? g.E : g.R);
  const double t = (double)g.R / tm + 0.5 * used;
  return t > used ? t : used;
}
// Tiles of tm rows that there can be at most.
inline int64_t ar_fp8_most_tiles(const ArFp8Shape& g, int64_t tm) {
  if (!g.grouped) return (g.R + tm - 1) / tm;
  const int64_t t = g.R / tm + g.E;   // every range adds at most one ragged tile
  return t < g.R ? t : g.R;
}

struct ArFp8Plan {
  ArFp8Kind kind;
  bool two;   // two K sets
};
inline ArFp8Plan ar_fp8_plan(const ArFp8Shape& g) {
  constexpr int block = 128;   // of K, with a scale of its own
  const double K = (double)g.K, N = (double)g.N, KB = (double)((g.K + block - 1) / block);
  const double used = (double)(g.E < g.R ? g.E : g.R), mean = (double)g.R / used;
  const double memory = (used * N + (double)g.R) * K / 5.3e6;
  ArFp8Plan best{k32x64, false};
  double least = -1.0;
  // Rows: every tile of 16 rows streams W, at 5.8 TB/s less X's share of the loads;
  // by expert at 4.6 with a row each, at 4.0 with more. A CU takes 0.7 us per
  // workgroup.
  const double columns = (double)((g.N + 15) / 16);
  if (mean <= 256 && ar_fp8_most_tiles(g, 16) <= 65535) {
    const double tiles = ar_fp8_expected_tiles(g, 16);
    const double share = 1.0 + 0.4 * (mean < 16 ? mean : 16) / 16;
    const double rate = !g.grouped ? 5.8e6 : g.R <= g.E ? 4.6e6 : 4.0e6;
    const double stream = tiles * N * K * share / rate;
    least = KB / 8 * 0.45;
    if (least < stream) least = stream;
    if (least < tiles * columns / 256 * 0.7) least = tiles * columns / 256 * 0.7;
    least += 3.0;
    best.kind = kRows;
  }
  const double cache_rate = g.K % 64 == 0 ? 14e6 : 12e6;
  for (int k = k32x64; k < kKinds; ++k) {
    const ArFp8Times& c = ar_fp8_times(g.wide, k);
    if (!c.tm) continue;
    // by expert: some of the ragged tiles that uneven ranges add
    const double t = ar_fp8_expected_tiles(g, c.tm) * (double)((g.N + c.tn - 1) / c.tn) *
                     (g.grouped ? 1.15 : 1.0);
    const bool two = c.step2 > 0 && t <= 256;
    const double rounds = ceil(t / 256);
    double us = two ? 4.0 + 0.5 * (KB + 1) * c.step2 : 3.0 + rounds * (KB * c.step + c.ends);
    const double stream = two ? 3.0 + 1.12 * memory : 3.0 + memory + rounds * c.gap;
    const double cache = 3.0 + t * KB * (c.tm + c.tn) * block / cache_rate;
    if (us < stream) us = stream;
    if (us < cache) us = cache;
    if (least < 0 || us < least) {
      least = us;
      best = ArFp8Plan{(ArFp8Kind)k, two};
    }
  }
  return best;
}
