// Attention of each sequence's newest tokens over its pages of the 4-bit cache (gfx950),
// straight from the codes (layout: ar_kv4.h).
//
//   out = softmax(scale·q·Kᵀ)·V,   K = ks·(ck - kz), V = vs·(cv - vz) per group of channels
//
// The cache is read once and nothing else is large, so memory bounds it; what the codes
// cost on the way is kept below that. The products run on v_mfma_f32_16x16x32_f16 with the
// codes themselves on the cache's side: masked out of a word, (word & 0x000F000F) is two f16
// subnormals, code·2^-24, which the matrix unit takes; one instruction for two codes. What the
// zero-points take off, Σ q·zp and Σ p·vs·zp, is one more such product each, and the scales
// stay outside: ks multiplies the finished score, vs the weight.
//
// q goes to f16 as q·2^k, its row's largest magnitude in [2^11, 2^12): exact but for what
// lies 2^-31 below that. A row is one query head of one new token; up to 16·RT rows share a
// key head's codes. Scores are formed transposed (A: 16 tokens, B: 16 rows), so a lane
// holds one row's scores of eight neighbouring tokens (8·(l/16) .. + 7 of 32, by the choice
// which token is which row of A), and these are the eight that it supplies to the second
// product, Oᵀ = Vᵀ·Pᵀ: nothing passes between lanes.
// The weights of that product are p·vs in f16, times a power of 2 for each row and group that
// keeps the largest that the row has met in f16's upper half: half a step of 2^-11 each, an eighth
// of what rounding to bf16 would cost, and below 2^-30 of the row's largest nothing counts. What a
// row does not see, or gives no weight, takes no part in that. p = 2^(x - m) <= 1 with a running
// reference m, a whole number so that a step of it goes into that power of 2, that is set 8 above
// the maximum when that has passed it; the sums of p and all accumulators are float32.
//
// Each wave goes through its tokens alone, 32 at a time. A tile goes straight to one of two
// LDS stages of the wave, and the one after next is asked for as soon as it has been used; no
// wave waits for another until all are joined in LDS, and the workgroups that share a long
// sequence are joined through the workspace, in order. How the sequences are divided follows
// from their lengths, on the device: every workgroup makes the same plan.
//
// Measured: 2 x 131072 tokens, 64 heads over 8 of 128, groups of 64 (302 MB) 63 us, 4.8 TB/s;
// 64 x 8192, groups of 128 (570 MB) 107 us, 5.3 TB/s; 64 x up to 8192 (123 MB) 38 us, 3.2 TB/s,
// where plan, joins and the last workgroups' ends are a third; one sequence of 1000 tokens,
// 32 heads, 9.8 us, a chain of launch, lengths, table, tiles and joins with nothing to hide it
// under.
#include <math.h>

#include "ar_kv4.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256;
constexpr int GRAIN = 128;        // a workgroup's tokens are a multiple of that
constexpr float NO_MAX = -3.0e38f;
constexpr float RISE = 8.0f;      // m lies so far above the maximum when it is set
constexpr float APART = 0x1p24f;  // a reference whose rounding 2^x would feel
constexpr int W_NEW = 7;          // the largest weight when its factor is set is in [2^6, 2^7),
constexpr float W_MOST = 0x1p15f; // and at most that later

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  ArKv4 c;
  const int32_t *table, *lengths;
  int width, max_len, B, news, heads, ratio, rows, tiles;
  int target, least;       // log2 of the workgroups wanted; tokens of one at least
  float sl;                // scale·log2 e
  uint16_t* out;
  float* lse;
  float *po, *pm;          // partial sums [workgroup][row][Dh] and (m, l) of each row
  // where the parts of a sequence went: how many there are, the full ones among them, the
  // place of the first of these and that of the rest
  struct Parts {
    int all, full, first, rest;
  } * parts;
};

// Codes as f16: a code at bit b of a half word is the subnormal code·2^(b - 24), which the
// matrix unit takes as it is. (It adds the products of 8 neighbours to 24 bits below the
// largest one's exponent, and a subnormal's exponent there is -14: of a product of such a code
// what lies 2^-(14 + b) below the largest factor on the other side is cut off.)
// Values: bits 0 and 4, for weights of 11 bits.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) { return w & 0x000F000Fu; }
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return w & 0x00F000F0u; }
// Keys: bits 3 and 7, for scores, at one more shift. Eight codes of one token: element 2i is
// code i, 2i + 1 code i + 4, those of odd i 16-fold.
__device__ __forceinline__ f16x8_t keys_of(uint32_t w) {
  const uint32_t u = w << 3, v = w >> 5;
  return __builtin_bit_cast(f16x8_t, u32x4_t{u & 0x00780078u, u & 0x07800780u, v & 0x00780078u,
                                             v & 0x07800780u});
}
// The zero-points of two tokens' scales, side by side.
__device__ __forceinline__ uint32_t zeros_of(float a, float b) {
  return low_codes(__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x05040100u));
}

// Largest over the four lanes of a row.
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// 32 tokens of a key head in LDS, as they lie in memory: codes of the keys, of the values,
// scales of the keys, of the values.
template <int DH, int GS>
struct Tile {
  static constexpr int G = DH / GS, CODES = 16 * DH, SCALES = 128 * G;
  static constexpr int BYTES = 2 * (CODES + SCALES), LOADS = 2 * (CODES / 1024) + G;
};
// Scales of groups g .. g + N - 1 of an octet (p: those of its first token).
template <int G, int N>
__device__ __forceinline__ void octet_scales(const float* p, int g, float (&s)[N][8]) {
  if constexpr (N == G) {
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const f32x4_t w = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[(4 * i + e) % G][(4 * i + e) / G] = w[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i][e] = p[e * G + g + i];
  }
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  asm volatile("" ::: "memory");
}

// How the sequences are divided, from their lengths alone and so the same for every
// workgroup: into parts of `chunk` tokens, 2^target workgroups over all the tokens, and one
// for what is left of each. The full parts come first, sequence by sequence, then the
// shorter ones: a round of workgroups ends evenly, and the short parts fill its gaps.
__device__ __forceinline__ int length_of(const AttnArgs& a, int b) {
  return b < a.B ? min(max(a.lengths[b], 0), a.max_len) : 0;
}
constexpr int KEPT = 4;   // times 64 sequences whose lengths stay in registers
struct Division {
  int chunk, full;   // tokens of a part, full parts in all
  int len[KEPT];     // lengths of the sequences lane, lane + 64, ..
  __device__ __forceinline__ int full_of(int len) const { return (uint32_t)len / (uint32_t)chunk; }
  // a rest, or the one part of an empty sequence
  __device__ __forceinline__ int rest_of(int len) const {
    return len == 0 || full_of(len) * chunk < len;
  }
  __device__ __forceinline__ int parts_of(int len) const { return full_of(len) + rest_of(len); }
};
// f(base, length of sequence base + lane) for base = 0, 64, .. below `to`, while f is true.
template <class F>
__device__ __forceinline__ void each_64(const AttnArgs& a, const Division& d, int to, F f) {
#pragma unroll
  for (int i = 0; i < KEPT; ++i)
    if (64 * i >= to || !f(64 * i, d.len[i])) return;
  for (int base = 64 * KEPT; base < to; base += 64)
    if (!f(base, length_of(a, base + (threadIdx.x & 63)))) return;
}
__device__ __forceinline__ Division divide(const AttnArgs& a) {
  const int lane = threadIdx.x & 63;
  Division d;
#pragma unroll
  for (int i = 0; i < KEPT; ++i) d.len[i] = length_of(a, 64 * i + lane);
  float tokens = 0.0f;   // (rounded alike everywhere)
  each_64(a, d, a.B, [&](int, int len) {
    tokens += (float)len;
    return true;
  });
  const float each = wave_total(wave_scan(tokens)) * (float)(a.c.heads * a.tiles) *
                     ldexpf(1.001f, -a.target);
  // (above the quotient whatever the roundings, so that there are no more full parts than
  // workgroups; no length is 2^30)
  const int c = (int)fminf(fmaxf(each + 1.0f, (float)a.least), 0x1p30f);
  d.chunk = __builtin_amdgcn_readfirstlane((c + GRAIN - 1) / GRAIN * GRAIN);
  int full = 0;
  each_64(a, d, a.B, [&](int, int len) {
    full += d.full_of(len);   // (0 beyond the last sequence)
    return true;
  });
  d.full = wave_total(wave_scan(full));
  return d;
}
// Part `at` of all: sequence b's part `part`; false when there is none.
__device__ __forceinline__ bool find_part(const AttnArgs& a, const Division& d, int at, int& b,
                                          int& part, int& len) {
  const int lane = threadIdx.x & 63;
  const bool whole = at < d.full;
  int before = whole ? 0 : d.full;
  bool found = false;
  each_64(a, d, a.B, [&](int base, int mine) {
    const int n = base + lane < a.B ? (whole ? d.full_of(mine) : d.rest_of(mine)) : 0;
    const int sum = wave_scan(n);
    const uint64_t past = __ballot(before + sum > at);
    found = past != 0;
    if (found) {
      const int l = __ffsll((unsigned long long)past) - 1;
      b = base + l;
      len = __builtin_amdgcn_readlane(mine, l);
      part = whole ? at - before - __builtin_amdgcn_readlane(sum - n, l) : d.full_of(len);
    }
    before += wave_total(sum);
    return !found;
  });
  return found;
}

// Four channels of a row's output from its sums relative to 2^m, and its lse.
template <int DH>
__device__ __forceinline__ void write_row(const AttnArgs& a, int b, int h, int at, int c,
                                          const f32x4_t& v, float m, float sum) {
  const int i = at / a.ratio;
  const int64_t to = ((int64_t)b * a.news + i) * a.heads + h * a.ratio + at - i * a.ratio;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees no key is 0
  *reinterpret_cast<u32x2_t*>(a.out + to * DH + c) =
      u32x2_t{bf16_pair(v[0] * inv, v[1] * inv), bf16_pair(v[2] * inv, v[3] * inv)};
  if (a.lse && c == 0)
    a.lse[to] = sum == 0.0f ? -INFINITY : 0.69314718f * (m - RISE + __log2f(ldexpf(sum, (int)RISE)));
}

// Waves a SIMD that the registers are held to. (From two on, products stay out of the
// accumulation registers, which the softmax would have to copy from.)
constexpr int occupancy(int DH, int G, int RT, int WAVES) {
  return WAVES == 8 || RT == 2 ? 2 : DH == 64 ? 4 : G == 4 ? 2 : 3;
}

// WHOLE: sequences are not divided.
template <int DH, int GS, int RT, int WAVES, int STAGES, bool WHOLE>
__global__ __launch_bounds__(64 * WAVES, occupancy(DH, DH / GS, RT, WAVES)) void k_kv4_attention(AttnArgs a) {
  constexpr int G = DH / GS, KW = GS / 32, NB = DH / 64, NO = DH / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int Hk = a.c.heads, per = Hk * a.tiles;
  const int at = blockIdx.x / per, rest = blockIdx.x - at * per;
  const int h = rest / a.tiles, tile = rest - h * a.tiles;
  int b = at, len, first = 0, last;
  int chunk = 1 << 30;   // tokens of a part
  if constexpr (WHOLE) {
    len = last = __builtin_amdgcn_readfirstlane(length_of(a, b));
  } else {
    const Division d = divide(a);
    int part;
    if (!find_part(a, d, at, b, part, len)) return;
    first = part * d.chunk;
    last = min(len, first + d.chunk);
    chunk = d.chunk;
  }

  // the lane's row of each of the RT products and its queries
  u32x4_t qraw[RT][G][KW];
  int sees[RT];        // keys before this one
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = (tile * RT + t) * 16 + n, i = row / a.ratio;
    const uint16_t* p = a.q + ((int64_t)b * a.news + i) * a.q_stride +
                        (h * a.ratio + row - i * a.ratio) * DH;
    sees[t] = row < a.rows ? len - a.news + 1 + i : 0;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        qraw[t][g][k] = u32x4_t{0u, 0u, 0u, 0u};
        if (row < a.rows)
          qraw[t][g][k] = *reinterpret_cast<const u32x4_t*>(p + g * GS + g4 * (GS / 4) + 8 * k);
      }
  }

  // (read through the scalar cache: a wait for an entry is then none for the loads before it)
  typedef __attribute__((address_space(4))) const int32_t* table_t;
  const table_t tab = (table_t)(a.table + (int64_t)b * a.width);
  const int npages = (int)a.c.pages;
  auto page_of = [&](int t) {   // page of token t, -1 where there is none
    const int e = t >> a.c.shift;
    const int p = e < a.width ? tab[e] : -1;
    return (uint32_t)p < (uint32_t)npages ? p : -1;
  };
  const int ktok = 8 * (n >> 2) + (n & 3), vtok = 8 * g4;   // the lane's tokens in a tile
  using Tl = Tile<DH, GS>;
  constexpr int R = 16 * RT, LD = DH + 4, RING = STAGES * Tl::BYTES;
  constexpr int JOIN = WAVES * R * (LD + 2) * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * RING > JOIN ? WAVES * RING : JOIN];
  uint8_t* const ring = lds + wave * RING;

  // the tile at token t, whose halves lie in pages p0 and p1 (any page stands in for none),
  // straight to LDS: each load 1 KiB of codes or 256 bytes of scales
  const int64_t page_rows = (int64_t)2 * Hk * a.c.page, head_row = (int64_t)h * a.c.page;
  const int64_t to_values = (int64_t)Hk * a.c.page;
  auto fetch = [&](int t, int p0, int p1, uint8_t* to) {
    typedef __attribute__((address_space(1))) const void* from_t;
    typedef __attribute__((address_space(3))) void* to_t;
    const int in = t & (a.c.page - 1);
    const int64_t row0 = max(p0, 0) * page_rows + head_row + in;
    // (with pages of 16 the second half begins a page of its own)
    const int64_t more = a.c.page == 16 ? (max(p1, 0) - max(p0, 0)) * page_rows - 16 : 0;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < Tl::CODES / 1024; ++i) {
        const int at = i * 1024 + lane * 16;
        const uint8_t* p = a.c.codes + (row0 + w * to_values) * (DH / 2);
        if (a.c.page == 16 && at >= 8 * DH) p += more * (DH / 2);
        __builtin_amdgcn_global_load_lds((from_t)(p + (uint32_t)at),
                                         (to_t)(to + w * Tl::CODES + i * 1024), 16, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int at = i * 64 + lane, w = at / (32 * G), k = at - w * 32 * G;
      const float* p = a.c.scale + row0 * G;
      if (G == 1 ? w != 0 : 2 * i >= G) p += to_values * G;
      if (a.c.page == 16 && k >= 16 * G) p += more * G;
      __builtin_amdgcn_global_load_lds((from_t)(p + (uint32_t)k), (to_t)(to + 2 * Tl::CODES + i * 256),
                                       4, 0, 0);
    }
  };
  f16x8_t qf[RT][G][KW], qz[RT][G];
  float qs[RT];        // takes a sum of products to the exponent of 2
  int power[RT];       // that of 2 in it
  // A wave's scores are scaled as they are formed, qs being only that power of 2, where
  // - it is far from 1: scale times queries above 2^91 or below 2^-109;
  // - a row's reference is beyond APART: half a step of it, which the product within an fma does
  //   not share, is more than 2^x holds, so the scores are rounded before they are compared.
  bool apart = false;
  const float sl1 = __builtin_amdgcn_frexp_mantf(a.sl);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float x[G][KW][8];
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = qraw[t][g][k][e / 2], f = e & 1 ? w & 0xFFFF0000u : w << 16;
          x[g][k][e] = __uint_as_float(f);
          top = max(top, f & 0x7FFFFFFFu);
        }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const float big = __uint_as_float(top);
    // (a row with an infinity or a NaN is NaN whatever its other channels become)
    const int up = top == 0 || top >= 0x7F800000u ? 0 : 12 - __builtin_amdgcn_frexp_expf(big);
    power[t] = __builtin_amdgcn_frexp_expf(a.sl) + 21 - up;   // (codes are 2^-21 of themselves)
    apart |= abs(power[t]) > 100;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {   // in keys_of's order
          const float v = ldexpf(x[g][k][(e >> 1) + 4 * (e & 1)], up);
          sum += v;
          qf[t][g][k][e] = (_Float16)(e & 2 ? v * 0.0625f : v);
        }
      // what a zero-point takes off: the group's sum in three parts of 11 bits, for the
      // products with 128·zp of lanes 0 .. 15
      sum = row_sum(sum) * -0.0625f;   // (at most 2^19: 128 channels)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const _Float16 part = e < 3 && g4 == 0 ? (_Float16)sum : (_Float16)0.0f;
        qz[t][g][e] = part;
        sum -= (float)part;
      }
    }
  }

  apart = __any(apart);
#pragma unroll
  for (int t = 0; t < RT; ++t) qs[t] = apart ? __int_as_float(power[t]) : ldexpf(sl1, power[t]);

  // STAGES tiles on their way, and the pages of those that are not yet worked on
  constexpr int STEP = 32 * WAVES, LOADS = Tl::LOADS;
  const int t0 = first + 32 * wave;
  int p0[STAGES], p1[STAGES];
#pragma unroll
  for (int i = 0; i < STAGES; ++i) {
    const int t = t0 + i * STEP;
    p0[i] = page_of(t), p1[i] = page_of(t + 16);
    if (t < last) fetch(t, p0[i], p1[i], ring + i * Tl::BYTES);
  }

  f32x4_t o[RT][NO];
  // what the values' zero-points take off, in every element (a group's own, so that a NaN
  // stays within it)
  f32x4_t oz[RT][G];
  float m[RT], l[RT], wk[RT][G];   // wk: powers of 2
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = NO_MAX;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < NO; ++d) o[t][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < G; ++g) oz[t][g] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, wk[t][g] = 0x1p120f;
  }
  // o and oz of a row and group times f
  auto rescale = [&](int t, int g, float f) {
#pragma unroll
    for (int d = g * GS / 16; d < (g + 1) * GS / 16; ++d) o[t][d] *= f;
    oz[t][g] *= f;
  };

  // Groups whose scales are held at once: all of four would take 64 registers; with fewer a
  // tile looks once whether any reference has to follow (two long sequences, two groups: 63 us
  // instead of 76).
  constexpr int AT = G <= 2 && (DH == 64 || G * RT < 4) ? G : 1;
  float s[RT][8];   // of token t0 + 8·g4 + e
  auto scale_scores = [&]() {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[t][e] = ldexpf(s[t][e] * sl1, __float_as_int(qs[t]));
  };
  auto scores = [&](const uint8_t* tile) {
    const float* scale = reinterpret_cast<const float*>(tile + 2 * Tl::CODES);
    float ks[AT][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g % AT == 0) octet_scales<G, AT>(scale + vtok * G, g, ks);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t z = kv4_zero(scale[(ktok + 4 * j) * G + g]) * 0x00800080u;   // 128·zp, twice
        // (of the same shape as the products that it is chained to: between one of 16x16x16 and
        // these the compiler puts no wait, and they took half of its result too early)
        const f16x8_t zf = __builtin_bit_cast(f16x8_t, u32x4_t{z, z, z, z});
        f32x4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(zf, qz[t][g],
                                                          f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
        uint32_t words[KW];   // the lane's token's codes of GS/4 channels
        const uint8_t* from = tile + (ktok + 4 * j) * (DH / 2) + g * (GS / 2) + g4 * (GS / 8);
        if constexpr (KW == 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(from);
#pragma unroll
          for (int i = 0; i < 4; ++i) words[i] = v[i];
        } else if constexpr (KW == 2) {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(from);
          words[0] = v[0];
          words[1] = v[1];
        } else {
          words[0] = *reinterpret_cast<const uint32_t*>(from);
        }
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const f16x8_t f = keys_of(words[k]);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, qf[t][g][k], acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[t][4 * j + r] = g == 0 ? acc[t][r] * ks[g % AT][4 * j + r]
                                     : fmaf(acc[t][r], ks[g % AT][4 * j + r], s[t][4 * j + r]);
      }
    }
    if (apart) scale_scores();
  };
  auto weigh = [&](const uint8_t* tile, int t0, int p0, int p1) {
    u32x4_t yv[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
      yv[i] = *reinterpret_cast<const u32x4_t*>(tile + Tl::CODES + kv4_value_at(vtok, i, n, 0, NB));
    const bool bad = p0 < 0 || p1 < 0;
    const bool tail = bad || t0 + 32 > len - a.news + 1;
    const bool gone = (vtok >= 16 ? p1 : p0) < 0;
    const float* vscale =
        reinterpret_cast<const float*>(tile + 2 * Tl::CODES + Tl::SCALES) + vtok * G;
    float ys[AT][8];
    if constexpr (AT == G) octet_scales<G, AT>(vscale, 0, ys);
    if (tail)   // some token is hidden from some row
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          s[t][e] = gone || t0 + vtok + e >= sees[t] ? -INFINITY : s[t][e];
    auto largest = [&](const float (&x)[8]) {
      float m = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) m = fmaxf(m, x[e]);
      return m;
    };
    bool rises = false;
    float top[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      top[t] = largest(s[t]) * (apart ? 1.0f : qs[t]);
      rises |= top[t] > m[t];
    }
    if (__any(rises)) {
      bool beyond = false;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float high = row_max(top[t]), mn = high > m[t] ? ceilf(high) + RISE : m[t];
        const int by = (int)fmaxf(m[t] - mn, -1000.0f);
        m[t] = mn;
        beyond |= fabsf(mn) >= APART && mn != NO_MAX;
        l[t] = ldexpf(l[t], by);
#pragma unroll
        for (int g = 0; g < G; ++g) {   // the sums stay as they are, as long as wk can make up for it
          const int k = __builtin_amdgcn_frexp_expf(wk[t][g]) - 1 - by, kn = min(k, 120);
          wk[t][g] = ldexpf(1.0f, kn);
          rescale(t, g, ldexpf(1.0f, kn - k));
        }
      }
      if (!apart && __any(beyond)) {
        apart = true;
#pragma unroll
        for (int t = 0; t < RT; ++t) qs[t] = __int_as_float(__builtin_amdgcn_frexp_expf(qs[t]));
        scale_scores();
      }
    }
    float p[RT][8];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], apart ? 1.0f : qs[t], -m[t]));
        l[t] += p[t][e];
      }
    // weights p·vs of the groups g .. g + AT - 1, eight tokens of the lane's row
    float w[RT][AT][8];
    auto weights = [&](int g) {
      bool rises = false;
      float top[RT][AT];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < AT; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[t][i][e] = p[t][e] * ys[i][e];
          float size[8];   // (a cache's owner may hold scales below 0)
#pragma unroll
          for (int e = 0; e < 8; ++e) size[e] = fabsf(w[t][i][e]);
          top[t][i] = largest(size);
          rises |= top[t][i] * wk[t][g + i] > W_MOST;
        }
      if (__any(rises))
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < AT; ++i) {
            const float high = row_max(top[t][i]);
            const int k = __builtin_amdgcn_frexp_expf(wk[t][g + i]) - 1;
            const int kn = high * wk[t][g + i] > W_MOST ? W_NEW - __builtin_amdgcn_frexp_expf(high) : k;
            wk[t][g + i] = ldexpf(1.0f, kn);
            rescale(t, g + i, ldexpf(1.0f, kn - k));
          }
    };
    if constexpr (AT == G) weights(0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if constexpr (AT < G) {
        octet_scales<G, AT>(vscale, g, ys);
        weights(g);
      }
      f16x8_t wh[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) wh[t][e] = (_Float16)(w[t][g % AT][e] * wk[t][g]);
      if (tail)   // hidden tokens weigh nothing, whatever they hold
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (s[t][e] == -INFINITY) wh[t][e] = (_Float16)0.0f;
      u32x4_t z;
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = zeros_of(ys[g % AT][2 * i], ys[g % AT][2 * i + 1]);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        oz[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, z), wh[t],
                                                          oz[t][g], 0, 0, 0);
#pragma unroll
      for (int q = g * GS / 32; q < (g + 1) * GS / 32; ++q) {   // 32 channels each
        u32x4_t lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = q & 1 ? yv[q / 2][i] >> 8 : yv[q / 2][i];
          lo[i] = low_codes(u);
          hi[i] = high_codes(u);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4_t* d = &o[t][2 * q];
          d[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, lo), wh[t], d[0],
                                                        0, 0, 0);
          d[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hi), wh[t], d[1],
                                                        0, 0, 0);
        }
      }
    }
  };

  for (int base = t0; base < last; base += STAGES * STEP)
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      const int t = base + i * STEP;
      if (t >= last) break;
      // the loads of this tile have come once no more than the others' are left
      if (t + (STAGES - 1) * STEP < last) wait_loads<(STAGES - 1) * LOADS>();
      else wait_loads<0>();
      const int n0 = page_of(t + STAGES * STEP), n1 = page_of(t + STAGES * STEP + 16);
      scores(ring + i * Tl::BYTES);
      weigh(ring + i * Tl::BYTES, t, p0[i], p1[i]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the tile has been read
      if (t + STAGES * STEP < last) fetch(t + STAGES * STEP, n0, n1, ring + i * Tl::BYTES);
      p0[i] = n0, p1[i] = n1;
    }

  // join the waves: rows x channels in LDS, each wave's relative to its own m
  float(&so)[WAVES][R][LD] = *reinterpret_cast<float(*)[WAVES][R][LD]>(lds);
  float(&sm)[WAVES][R] = *reinterpret_cast<float(*)[WAVES][R]>(lds + sizeof(so));
  float(&sl)[WAVES][R] = *reinterpret_cast<float(*)[WAVES][R]>(lds + sizeof(so) + sizeof(sm));
  const int waves = max(1, min(WAVES, (last - first + 31) / 32));   // those that had tokens
  __syncthreads();   // the tiles have been read
  if (wave < waves)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = 16 * t + n;
      const float sum = row_sum(l[t]);
      if (tile * R + row >= a.rows) continue;
      if (g4 == 0) sm[wave][row] = m[t], sl[wave][row] = sum;
#pragma unroll
      for (int q = 0; q < NO / 2; ++q) {
        // (codes are 2^-24 of themselves, those of odd channels 2^-20)
        const int k = 25 - __builtin_amdgcn_frexp_expf(wk[t][32 * q / GS]);
        const f32x4_t z = oz[t][32 * q / GS], x = o[t][2 * q], y = o[t][2 * q + 1];
#pragma unroll
        for (int r = 0; r < 4; r += 2)   // channels 32·q + 8·g4 + 2·r ..
          *reinterpret_cast<f32x4_t*>(&so[wave][row][32 * q + 8 * g4 + 2 * r]) =
              f32x4_t{ldexpf(x[r] - z[r], k), ldexpf(y[r] * 0.0625f - z[r], k),
                      ldexpf(x[r + 1] - z[r + 1], k), ldexpf(y[r + 1] * 0.0625f - z[r + 1], k)};
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (DH / 4); e += 64 * WAVES) {
    const int row = e / (DH / 4), c = 4 * (e % (DH / 4)), at = tile * R + row;
    if (at >= a.rows) break;
    float mm = sm[0][row];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
      if (w < waves) mm = fmaxf(mm, sm[w][row]);
    float sum = 0.0f;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w >= waves) break;
      const float f = __builtin_amdgcn_exp2f(sm[w][row] - mm);
      sum += f * sl[w][row];
      v += f * *reinterpret_cast<const f32x4_t*>(&so[w][row][c]);
    }
    if (!WHOLE && len > chunk) {
      const int64_t to = (int64_t)blockIdx.x * R + row;
      *reinterpret_cast<f32x4_t*>(a.po + to * DH + c) = v;
      if (c == 0) a.pm[2 * to] = mm, a.pm[2 * to + 1] = sum;
    } else {
      write_row<DH>(a, b, h, at, c, v, mm, sum);
    }
  }
  if (!WHOLE && rest == 0 && wave == 0) {   // (by all lanes alike)
    const int full = len / chunk, all = full + (len == 0 || full * chunk < len);
    if (first == full * chunk) a.parts[b].rest = at;
    if (first == 0) a.parts[b].all = all, a.parts[b].full = full, a.parts[b].first = at;
  }
}

// Joins the parts of a row, where there are several: GROUPS groups of Dh/4 lanes take the
// parts in turn, a lane four channels, and the groups' sums are added in order. GROUPS = 1 for
// many rows of few parts each. A workgroup's rows are of one sequence and key head.
template <int DH, int GROUPS>
__global__ __launch_bounds__(NT) void k_kv4_join(AttnArgs a, int R) {
  constexpr int LPR = DH / 4, ROWS = NT / LPR / GROUPS;   // rows a workgroup
  const int each = (a.rows + ROWS - 1) / ROWS;
  const int bh = blockIdx.x / each, b = bh / a.c.heads, h = bh - b * a.c.heads;
  const int row = (blockIdx.x - bh * each) * ROWS + threadIdx.x / LPR / GROUPS;
  const int g = threadIdx.x / LPR % GROUPS, c = threadIdx.x % LPR;
  const AttnArgs::Parts p = a.parts[b];
  if (p.all < 2) return;   // a single one has written its rows
  float mm = NO_MAX, sum = 0.0f;
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (row < a.rows) {
    const int64_t step = (int64_t)a.c.heads * a.tiles * R, from = (int64_t)h * a.tiles * R + row;
    auto at = [&](int s) { return from + (s < p.full ? p.first + s : p.rest) * step; };
    for (int s = c; s < p.all; s += LPR) mm = fmaxf(mm, a.pm[2 * at(s)]);
    mm = group_max<LPR>(mm);
#pragma unroll 4
    for (int s = g; s < p.all; s += GROUPS) {
      const int64_t to = at(s);
      const float f = __builtin_amdgcn_exp2f(a.pm[2 * to] - mm);
      sum += f * a.pm[2 * to + 1];
      v += f * *reinterpret_cast<const f32x4_t*>(a.po + to * DH + 4 * c);
    }
  }
  if constexpr (GROUPS > 1) {
    __shared__ f32x4_t sv[GROUPS][LPR];
    __shared__ float sl[GROUPS];
    sv[g][c] = v;
    if (c == 0) sl[g] = sum;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      v += sv[i][c];
      sum += sl[i];
    }
  }
  if (row < a.rows) write_row<DH>(a, b, h, row, 4 * c, v, mm, sum);
}

struct Plan {
  int RT, tiles, least, target;
  bool whole, wide;   // sequences undivided; eight waves for each
  int64_t groups;     // workgroups at most
};
Plan plan_of(int64_t B, int64_t heads, int DH, int GS, int64_t rows, int64_t max_len) {
  Plan p;
  // 512 workgroups run at once (2 x 131072 tokens: 62.8 us; 256 wanted 80.0, 1024 70.7), of
  // 256 tokens at least (1 x 2000: 10.3; of 512 11.8, of 128 10.0)
  p.least = 256;
  p.target = 9;
  // Up to 1024 tokens, eight waves of four tiles each are done before a join would be, unless
  // there are many (8 x 900 tokens, 8 key heads: 9.9 us, divided 10.7; 1 x 2000: 13.7, divided
  // 10.3; 64 x 900: 17.4 and 18.7). (Their sequences are not divided: see `whole`.)
  p.wide = B * heads * ((rows + 15) / 16) <= 512 && max_len > 256 && max_len <= 1024;
  // Two tiles of rows halve what each token's codes cost, where there is enough of that (8 key
  // heads, 32 rows; 8 x 8192 tokens: 29.9 us instead of 32.6; 64 x 1200: 30.4 and 33.6), and the
  // time of a single workgroup counts where there is not (2 x 8192: 22.0 instead of 17.7; just
  // at the border 32 x 1500: 26.1 and 24.8). Those of four groups do not fit.
  p.RT = !p.wide && rows > 16 && DH / GS < 4 && B * heads * max_len >= 3 << 17 ? 2 : 1;
  p.tiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  const int64_t per = heads * p.tiles;
  // Undivided, a call has neither plan nor join; what that saves is lost where few workgroups wait
  // for a long one. (7 query heads a key head; 150 x up to 960 tokens, 4 key heads: 13.4 us,
  // divided 17.1; 100 x 1000, 8: 28.6 and 31.7. 200 x up to 2000, 4: 23.0 either way; 100 x 2000, 8:
  // 49.5 and 52.8. 150 x up to 4000, 8: 46.2 and 43.0; 240: 66.5 and 69.2.) The rule for very many
  // is not borne out beyond such lengths: 255 x 1000 tokens and one of 131072, 8 key heads, take 889
  // us, and 101 with one sequence fewer, divided.
  const int64_t units = B * per;
  p.whole = max_len <= (units > 512 ? 2048 : 1024) || units >= int64_t(4) << p.target;
  p.groups = (B + (p.whole ? 0 : ((int64_t(1) << p.target) + per - 1) / per)) * per;
  return p;
}

template <int DH, int GS, int RT>
void launch_4(const AttnArgs& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.groups);
  if (p.whole) hipLaunchKernelGGL((k_kv4_attention<DH, GS, RT, 4, 2, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_kv4_attention<DH, GS, RT, 4, 2, false>), grid, dim3(256), 0, st, a);
}
template <int DH, int GS>
void launch(const AttnArgs& a, const Plan& p, hipStream_t st) {
  if constexpr (DH / GS < 4)
    if (p.RT == 2) {
      launch_4<DH, GS, 2>(a, p, st);
      return;
    }
  if (p.wide)
    hipLaunchKernelGGL((k_kv4_attention<DH, GS, 1, 8, 2, true>), dim3((unsigned)p.groups), dim3(512), 0, st, a);
  else
    launch_4<DH, GS, 1>(a, p, st);
}
template <int DH>
void join(const AttnArgs& a, const Plan& p, hipStream_t st) {
  constexpr int ALL = NT / (DH / 4);
  // one group a row where there are many rows (64 x 1200 tokens, 32 rows a key head: 30.4 us and
  // 34.6 by all groups; 150 x up to 4000, 7: 43.0 and 45.4), all of them for the many parts of
  // few rows (2 x 30000 tokens: 21.1 us and 23.8 by one)
  const int64_t units = (int64_t)a.B * a.c.heads;
  if (units * a.rows >= 2048)
    hipLaunchKernelGGL((k_kv4_join<DH, 1>), dim3((unsigned)(units * ((a.rows + ALL - 1) / ALL))),
                       dim3(NT), 0, st, a, 16 * p.RT);
  else
    hipLaunchKernelGGL((k_kv4_join<DH, ALL>), dim3((unsigned)(units * a.rows)), dim3(NT), 0, st, a,
                       16 * p.RT);
}

}  // namespace

// Floats of the workspace: partial sums and (m, l) of every row of every workgroup, and where
// the parts of each sequence went.
int64_t ar_kv4_attention_floats(const ar_kv4_cache& c, int64_t B, int64_t news, int64_t heads,
                                int64_t max_len) {
  const Plan p = plan_of(B, c.heads, c.head_dim, c.group_size, news * (heads / c.heads), max_len);
  return p.whole ? 0 : p.groups * 16 * p.RT * (c.head_dim + 2) + 4 * B;
}

ar_status ar_launch_kv4_attention(const ArKv4Attention& g, hipStream_t st) {
  const ar_kv4_cache& c = *g.cache;
  const int64_t rows = g.news * (g.heads / c.heads);
  const Plan p = plan_of(g.B, c.heads, c.head_dim, c.group_size, rows, g.max_len);
  AttnArgs a;
  a.q = g.q;
  a.q_stride = g.q_stride;
  a.c = ArKv4{c.codes, c.scale, c.pages, (int)c.heads, c.page_size, __builtin_ctz(c.page_size)};
  a.table = g.table;
  a.lengths = g.lengths;
  a.width = (int)g.width;
  a.max_len = (int)g.max_len;
  a.B = (int)g.B;
  a.news = (int)g.news;
  a.heads = (int)g.heads;
  a.ratio = (int)(g.heads / c.heads);
  a.rows = (int)rows;
  a.tiles = p.tiles;
  a.target = p.target;
  a.least = p.least;
  a.sl = (float)((double)g.scale * 1.4426950408889634);
  a.out = g.out;
  a.lse = g.lse;
  a.po = g.ws;
  a.pm = g.ws + p.groups * 16 * p.RT * c.head_dim;
  a.parts = reinterpret_cast<AttnArgs::Parts*>(a.pm + p.groups * 16 * p.RT * 2);
  const int DH = c.head_dim, GS = c.group_size;
  if (DH == 64 && GS == 32) launch<64, 32>(a, p, st);
  else if (DH == 64) launch<64, 64>(a, p, st);
  else if (GS == 32) launch<128, 32>(a, p, st);
  else if (GS == 64) launch<128, 64>(a, p, st);
  else launch<128, 128>(a, p, st);
  if (!p.whole) {
    if (DH == 64) join<64>(a, p, st);
    else join<128>(a, p, st);
  }
  return last_status();
}
