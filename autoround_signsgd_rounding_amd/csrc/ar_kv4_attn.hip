// Attention of each sequence's newest tokens over its pages of the 4-bit cache (gfx950),
// straight from the codes (layout: ar_kv4.h).
//
//   out = softmax(scale·q·Kᵀ)·V,   K = ks·(ck - kz), V = vs·(cv - vz) per group of channels
//
// The cache is read once and nothing else is large, so memory bounds it; what the codes
// cost on the way is kept below that. The products run on v_mfma_f32_16x16x32_f16 with the
// codes themselves on the cache's side: masked out of a word, (word & 0x000F000F) is two f16
// subnormals, code·2^-24, which the matrix unit takes; one instruction for two codes. What the zero-points take off, Σ q·zp and Σ p·vs·zp, is one more such product each,
// and the scales stay outside: ks multiplies the finished score, vs the weight.
//
// q goes to f16 as q·2^k, its row's largest magnitude in [2^11, 2^12): exact but for what
// lies 2^-31 below that. A row is one query head of one new token; up to 16·RT rows share a
// key head's codes. Scores are formed transposed (A: 16 tokens, B: 16 rows), so a lane
// holds one row's scores of eight neighbouring tokens (8·(l/16) .. + 7 of 32, by the choice
// which token is which row of A), and these are the eight that it supplies to the second
// product, Oᵀ = Vᵀ·Pᵀ: nothing passes between lanes.
// The weights of that product are p·vs in f16, relative to sv, the largest vs seen but for a
// factor of 2: half a step of 2^-11 each, an eighth of what rounding to bf16 would cost, and below
// 2^-30 of the largest nothing counts. p = 2^(x - m) with a running reference m that follows
// the maximum only when that has risen by more than 8 (p <= 256); the sums of p and all
// accumulators are float32.
//
// Each wave goes through its tokens alone, 32 at a time, and asks for the next keys once the
// scores are formed, for the next values once the product is; the waves of a workgroup are joined in LDS, and the workgroups that
// share a long sequence through the workspace, in order.
#include <math.h>

#include <type_traits>

#include "ar_kv4.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256;
constexpr int GRAIN = 128;        // a workgroup's tokens are a multiple of that
constexpr float NO_MAX = -3.0e38f;
constexpr float RISE = 8.0f;      // m follows the maximum when that is so far above it
constexpr float W_TOP = 64.0f;    // weight of p = 1 at vs = sv: 2^15 at p = 2^RISE, vs = 2·sv

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  ArKv4 c;
  const int32_t *table, *lengths;
  int width, max_len, B, news, heads, ratio, rows, tiles;
  int whole;               // sequences are not divided
  int target, least;       // log2 of the workgroups wanted; tokens of one at least
  float sl;                // scale·log2 e
  uint16_t* out;
  float* lse;
  float *po, *pm;          // partial sums [workgroup][row][Dh] and (m, l) of each row
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

// 32 tokens' keys and values as they lie in memory: a lane takes its channels of one key
// token in each half j of the tile, and the values of its octet.
template <int DH, int GS>
struct Keys {
  static constexpr int G = DH / GS, KW = GS / 32;
  uint32_t k[2][G][KW];
  float zero[2][G];   // that token's scales, for their zero-points
  float s[8][G];      // scales of the octet
};
template <int DH, int GS>
struct Values {
  static constexpr int G = DH / GS, NB = DH / 64;
  u32x4_t v[NB];
  float s[8][G];
};
template <int G>
__device__ __forceinline__ void load_scales(const float* p, float (&s)[8][G]) {
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) {
    const f32x4_t w = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[(4 * i + e) / G][(4 * i + e) % G] = w[e];
  }
}
// p + at: the lane's codes of its token in half 0 of the tile, which is four tokens before
// that in half 1; s + az that token's scales, s + as those of the octet.
template <int DH, int GS>
__device__ __forceinline__ void load_keys(Keys<DH, GS>& x, const uint8_t* p, uint32_t at,
                                          const float* s, uint32_t az, uint32_t as) {
  constexpr int G = DH / GS, KW = GS / 32;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t* w = p + (at + (uint32_t)(j * 4 * (DH / 2) + g * (GS / 2)));
      if constexpr (KW == 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.k[j][g][i] = v[i];
      } else if constexpr (KW == 2) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(w);
        x.k[j][g][0] = v[0];
        x.k[j][g][1] = v[1];
      } else {
        x.k[j][g][0] = *reinterpret_cast<const uint32_t*>(w);
      }
      x.zero[j][g] = s[az + (uint32_t)(j * 4 * G + g)];
    }
  }
  load_scales<G>(s + as, x.s);
}
template <int DH, int GS>
__device__ __forceinline__ void load_values(Values<DH, GS>& x, const uint8_t* p, uint32_t at,
                                            const float* s, uint32_t as) {
#pragma unroll
  for (int b = 0; b < DH / 64; ++b)
    x.v[b] = *reinterpret_cast<const u32x4_t*>(p + (at + (uint32_t)(b * 256)));
  load_scales<DH / GS>(s + as, x.s);
}

// Sum over a wave, inclusive of the lane's own and from lane 0 on.
template <class T>
__device__ __forceinline__ T wave_scan(T x) {
  auto add = [&](auto ctrl, auto rows) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                              decltype(rows)::value, 0xF, false);
    x += __builtin_bit_cast(T, o);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>(), integral_constant<int, 0xF>());   // from 1, 2, 4, 8 lanes
  add(integral_constant<int, 0x112>(), integral_constant<int, 0xF>());   // before in the row
  add(integral_constant<int, 0x114>(), integral_constant<int, 0xF>());
  add(integral_constant<int, 0x118>(), integral_constant<int, 0xF>());
  add(integral_constant<int, 0x142>(), integral_constant<int, 0xA>());   // from the rows before
  add(integral_constant<int, 0x143>(), integral_constant<int, 0xC>());
  return x;
}
template <class T>
__device__ __forceinline__ T wave_total(T scanned) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scanned), 63));
}

// How the sequences are divided, from their lengths alone and so the same for every
// workgroup: into parts of `chunk` tokens, 2^target workgroups over all the tokens, and one
// for what is left of each. The full parts come first, sequence by sequence, then the
// shorter ones: a round of workgroups ends evenly, and the short parts fill its gaps.
__device__ __forceinline__ int length_of(const AttnArgs& a, int b) {
  return b < a.B ? min(max(a.lengths[b], 0), a.max_len) : 0;
}
struct Division {
  int chunk, full, len0;   // tokens of a part, full parts in all, length of sequence `lane`
  __device__ __forceinline__ int full_of(int len) const { return (uint32_t)len / (uint32_t)chunk; }
  // a rest, or the one part of an empty sequence
  __device__ __forceinline__ int rest_of(int len) const {
    return len == 0 || full_of(len) * chunk < len;
  }
  __device__ __forceinline__ int parts_of(int len) const { return full_of(len) + rest_of(len); }
};
__device__ __forceinline__ Division divide(const AttnArgs& a) {
  const int lane = threadIdx.x & 63;
  Division d;
  d.len0 = length_of(a, lane);
  float tokens = (float)d.len0;   // (rounded alike everywhere)
  for (int b = lane + 64; b < a.B; b += 64) tokens += (float)length_of(a, b);
  const float each = wave_total(wave_scan(tokens)) * (float)(a.c.heads * a.tiles) *
                     ldexpf(1.0f, -a.target);
  // (above `each`, so that there are no more full parts than workgroups; no length is 2^30)
  const int c = (int)fminf(fmaxf(each + 1.0f, (float)a.least), 0x1p30f);
  d.chunk = __builtin_amdgcn_readfirstlane((c + GRAIN - 1) / GRAIN * GRAIN);
  d.full = 0;
  for (int base = 0; base < a.B; base += 64)
    d.full += wave_total(wave_scan(
        base + lane < a.B ? d.full_of(base ? length_of(a, base + lane) : d.len0) : 0));
  return d;
}
// Part `at` of all: sequence b's part `part`; false when there is none.
__device__ __forceinline__ bool find_part(const AttnArgs& a, const Division& d, int at, int& b,
                                          int& part, int& len) {
  const int lane = threadIdx.x & 63;
  const bool whole = at < d.full;
  int before = whole ? 0 : d.full;
  for (int base = 0; base < a.B; base += 64) {
    const int mine = base ? length_of(a, base + lane) : d.len0;
    const int n = base + lane < a.B ? (whole ? d.full_of(mine) : d.rest_of(mine)) : 0;
    const int sum = wave_scan(n);
    const uint64_t past = __ballot(before + sum > at);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      b = base + l;
      len = __builtin_amdgcn_readlane(mine, l);
      part = whole ? at - before - __builtin_amdgcn_readlane(sum - n, l) : d.full_of(len);
      return true;
    }
    before += wave_total(sum);
  }
  return false;
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
  if (a.lse && c == 0) a.lse[to] = sum == 0.0f ? -INFINITY : 0.69314718f * (m + __log2f(sum));
}

// Waves a SIMD that the registers are held to. (From two on, products stay out of the
// accumulation registers, which the softmax would have to copy from.)
constexpr int occupancy(int DH, int G, int RT, int WAVES) {
  return WAVES == 8 || DH + RT * G == 130 ? 2
         : DH == 64                         ? (RT == 2 ? 2 : G == 1 ? 4 : 3)
                                            : (G * RT == 1 ? 3 : 1);
}

template <int DH, int GS, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, occupancy(DH, DH / GS, RT, WAVES)) void k_kv4_attention(AttnArgs a) {
  constexpr int G = DH / GS, KW = GS / 32, NB = DH / 64, NO = DH / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int Hk = a.c.heads, per = Hk * a.tiles;
  const int at = blockIdx.x / per, rest = blockIdx.x - at * per;
  const int h = rest / a.tiles, tile = rest - h * a.tiles;
  int b = at, len, first = 0, last;
  bool joined = false;
  if (a.whole) {
    len = last = __builtin_amdgcn_readfirstlane(length_of(a, b));
  } else {
    const Division d = divide(a);
    int part;
    if (!find_part(a, d, at, b, part, len)) return;
    joined = len > d.chunk;
    first = part * d.chunk;
    last = min(len, first + d.chunk);
  }

  // the lane's row of each of the RT products, its queries and what it sees
  f16x8_t qf[RT][G][KW], qz[RT][G];
  float qs[RT];        // takes a sum of products to the exponent of 2
  int sees[RT];        // keys before this one
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = (tile * RT + t) * 16 + n, i = row / a.ratio;
    const bool live = row < a.rows;
    const uint16_t* p = a.q + ((int64_t)b * a.news + i) * a.q_stride +
                        (h * a.ratio + row - i * a.ratio) * DH;
    sees[t] = live ? len - a.news + 1 + i : 0;
    float x[G][KW][8];
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < KW; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][k][e] = 0.0f;
        if (live) load8(p + g * GS + g4 * (GS / 4) + 8 * k, x[g][k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[g][k][e]) & 0x7FFFFFFFu);
      }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const float big = __uint_as_float(top);
    // (a row with an infinity or a NaN is NaN whatever its other channels become)
    // (and one below 2^-120 throughout has scores of 0)
    const int up = top == 0 || top >= 0x7F800000u ? 0 : min(12 - __builtin_amdgcn_frexp_expf(big), 100);
    qs[t] = fmaxf(ldexpf(a.sl, 21 - up), 0x1p-126f);   // (codes are 2^-21 of themselves)
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

  f32x4_t o[RT][NO];
  // what the values' zero-points take off, in every element (a group's own, so that a NaN
  // stays within it)
  f32x4_t oz[RT][G];
  float m[RT], l[RT], sv[G], wk[G];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = NO_MAX;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < NO; ++d) o[t][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < G; ++g) oz[t][g] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int g = 0; g < G; ++g) sv[g] = 0x1p-120f, wk[g] = W_TOP * 0x1p120f;

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
  const int64_t page_rows = (int64_t)2 * Hk * a.c.page, head_row = (int64_t)h * a.c.page;
  const int64_t to_values = (int64_t)Hk * a.c.page;
  Keys<DH, GS> x;
  Values<DH, GS> y;
  // the tile at token t, whose halves lie in pages p0 and p1 (any page stands in for none)
  auto keys = [&](int t, int p0, int p1) {
    if (a.c.page > 16) {   // one page: the lanes' places in it are always the same
      const int64_t row = max(p0, 0) * page_rows + head_row + (t & (a.c.page - 1));
      load_keys<DH, GS>(x, a.c.codes + row * (DH / 2), ktok * (DH / 2) + g4 * (GS / 8),
                        a.c.scale + row * G, ktok * G, vtok * G);
    } else {
      const int64_t rk = max(ktok >= 16 ? p1 : p0, 0) * page_rows + head_row + (ktok & 15);
      const int64_t rv = max(vtok >= 16 ? p1 : p0, 0) * page_rows + head_row + (vtok & 15);
      load_keys<DH, GS>(x, a.c.codes + rk * (DH / 2), g4 * (GS / 8), a.c.scale + rk * G, 0,
                        (uint32_t)0);
      load_scales<G>(a.c.scale + rv * G, x.s);
    }
  };
  auto values = [&](int t, int p0, int p1) {
    if (a.c.page > 16) {
      const int in = t & (a.c.page - 1);
      const int64_t row = max(p0, 0) * page_rows + head_row + to_values;
      load_values<DH, GS>(y, a.c.codes + row * (DH / 2) + kv4_value_at(in, 0, 0, 0, NB),
                          kv4_value_at(vtok, 0, n, 0, NB), a.c.scale + (row + in) * G, vtok * G);
    } else {
      const int64_t row = max(vtok >= 16 ? p1 : p0, 0) * page_rows + head_row + to_values;
      load_values<DH, GS>(y, a.c.codes + row * (DH / 2), kv4_value_at(vtok & 15, 0, n, 0, NB),
                          a.c.scale + row * G, (vtok & 15) * G);
    }
  };
  float s[RT][8];   // of token t0 + 8·g4 + e
  auto scores = [&]() {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t z = kv4_zero(x.zero[j][g]) * 0x00800080u;   // 128·zp, twice
        // (of the same shape as the products that it is chained to: behind a 16x16x16 one they
        // took half of its result too early)
        const f16x8_t zf = __builtin_bit_cast(f16x8_t, u32x4_t{z, z, z, z});
        f32x4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(zf, qz[t][g],
                                                          f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const f16x8_t f = keys_of(x.k[j][g][k]);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, qf[t][g][k], acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[t][4 * j + r] = g == 0 ? acc[t][r] * x.s[4 * j + r][g]
                                     : fmaf(acc[t][r], x.s[4 * j + r][g], s[t][4 * j + r]);
      }
  };
  auto weigh = [&](int t0, int p0, int p1) {
    float vs[8][G];
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int g = 0; g < G; ++g) vs[e][g] = y.s[e][g];
    const bool bad = p0 < 0 || p1 < 0;
    const bool tail = bad || t0 + 32 > len - a.news + 1;
    if (tail) {   // some token is hidden from some row
      const bool gone = (vtok >= 16 ? p1 : p0) < 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int tok = t0 + vtok + e;
#pragma unroll
        for (int t = 0; t < RT; ++t)
          s[t][e] = gone || tok >= sees[t] ? -INFINITY : s[t][e];
#pragma unroll
        for (int g = 0; g < G; ++g) vs[e][g] = gone || tok >= len ? 0.0f : vs[e][g];
      }
    }
    bool rises = false;
    float top[RT], vtop[G];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      top[t] = s[t][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top[t] = fmaxf(top[t], s[t][e]);
      top[t] *= qs[t];
      rises |= top[t] > m[t] + RISE;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      vtop[g] = vs[0][g];
#pragma unroll
      for (int e = 1; e < 8; ++e) vtop[g] = fmaxf(vtop[g], vs[e][g]);
      rises |= vtop[g] > 2.0f * sv[g];
    }
    if (__any(rises)) {
      float by[RT], vby[G];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float mn = fmaxf(m[t], row_max(top[t]));
        by[t] = __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= by[t];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float sn = fmaxf(sv[g], group_max<64>(vtop[g]));
        vby[g] = sv[g] / sn;
        sv[g] = sn;
        wk[g] = W_TOP / sn;
      }
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int d = 0; d < NO; ++d) o[t][d] *= by[t] * vby[16 * d / GS];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int g = 0; g < G; ++g) oz[t][g] *= by[t] * vby[g];
    }
    float p[RT][8];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], qs[t], -m[t]));
        l[t] += p[t][e];
      }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // weights p·vs, eight tokens of the lane's row
      f16x8_t w[RT];
      float k[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = vs[e][g] * wk[g];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[t][e] = (_Float16)(p[t][e] * k[e]);
      if (tail)   // hidden tokens weigh nothing, whatever they hold
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (s[t][e] == -INFINITY) w[t][e] = (_Float16)0.0f;
      u32x4_t z;
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = zeros_of(y.s[2 * i][g], y.s[2 * i + 1][g]);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        oz[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, z), w[t],
                                                          oz[t][g], 0, 0, 0);
#pragma unroll
      for (int q = g * GS / 32; q < (g + 1) * GS / 32; ++q) {   // 32 channels each
        u32x4_t lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = q & 1 ? y.v[q / 2][i] >> 8 : y.v[q / 2][i];
          lo[i] = low_codes(u);
          hi[i] = high_codes(u);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4_t* d = &o[t][2 * q];
          d[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, lo), w[t], d[0],
                                                        0, 0, 0);
          d[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hi), w[t], d[1],
                                                        0, 0, 0);
        }
      }
    }
  };

  constexpr int STEP = 32 * WAVES;
  int t = first + 32 * wave;
  if (t < last) {
    // keys and values of the next tile are asked for as soon as the registers are free
    int p0 = page_of(t), p1 = page_of(t + 16);
    keys(t, p0, p1);
    values(t, p0, p1);
    for (; t < last; t += STEP) {
      const bool more = t + STEP < last;
      const int n0 = page_of(t + STEP), n1 = page_of(t + STEP + 16);
      scores();
      if (more) keys(t + STEP, n0, n1);
      weigh(t, p0, p1);
      if (more) values(t + STEP, n0, n1);
      p0 = n0, p1 = n1;
    }
  }

  // join the waves: rows x channels in LDS, each wave's relative to its own m
  constexpr int R = 16 * RT, LD = DH + 4;
  __shared__ float sm[WAVES][R], sl[WAVES][R], so[WAVES][R][LD];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = 16 * t + n;
    const float sum = row_sum(l[t]);
    if (g4 == 0) sm[wave][row] = m[t], sl[wave][row] = sum;
#pragma unroll
    for (int d = 0; d < NO; ++d) {
      // (codes are 2^-24 of themselves, those of odd d 2^-20)
      const float k = sv[16 * d / GS] * (0x1p24f / W_TOP), odd = d & 1 ? 0.0625f : 1.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r)   // channel 32·(d/2) + 2·(4·g4 + r) + d%2
        so[wave][row][32 * (d >> 1) + 2 * (4 * g4 + r) + (d & 1)] =
            (o[t][d][r] * odd - oz[t][16 * d / GS][r]) * k;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (DH / 4); e += 64 * WAVES) {
    const int row = e / (DH / 4), c = 4 * (e % (DH / 4)), at = tile * R + row;
    if (at >= a.rows) continue;
    float mm = sm[0][row];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mm = fmaxf(mm, sm[w][row]);
    float sum = 0.0f;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][row] - mm);
      sum += f * sl[w][row];
      v += f * *reinterpret_cast<const f32x4_t*>(&so[w][row][c]);
    }
    if (joined) {
      const int64_t to = (int64_t)blockIdx.x * R + row;
      *reinterpret_cast<f32x4_t*>(a.po + to * DH + c) = v;
      if (c == 0) a.pm[2 * to] = mm, a.pm[2 * to + 1] = sum;
    } else {
      write_row<DH>(a, b, h, at, c, v, mm, sum);
    }
  }
}

// Joins the parts of a row, where there are several: GROUPS groups of Dh/4 lanes take the
// parts in turn, a lane four channels, and the groups' sums are added in order. GROUPS = 1 for
// many rows of few parts each. A workgroup's rows are of one sequence and key head.
template <int DH, int GROUPS>
__global__ __launch_bounds__(NT) void k_kv4_join(AttnArgs a, int R) {
  constexpr int LPR = DH / 4, ROWS = NT / LPR / GROUPS;   // rows a workgroup
  const int lane = threadIdx.x & 63, each = (a.rows + ROWS - 1) / ROWS;
  const int bh = blockIdx.x / each, b = bh / a.c.heads, h = bh - b * a.c.heads;
  const int row = (blockIdx.x - bh * each) * ROWS + threadIdx.x / LPR / GROUPS;
  const int g = threadIdx.x / LPR % GROUPS, c = threadIdx.x % LPR;
  const Division d = divide(a);
  const int len = length_of(a, b), parts = d.parts_of(len);
  if (parts < 2) return;   // a single one has written its rows
  // parts of the sequences before this one
  int full = 0, rests = d.full;
  for (int base = 0; base < b; base += 64) {
    const int mine = base ? length_of(a, base + lane) : d.len0;
    full += wave_total(wave_scan(base + lane < b ? d.full_of(mine) : 0));
    rests += wave_total(wave_scan(base + lane < b ? d.rest_of(mine) : 0));
  }
  const int whole = d.full_of(len);
  float mm = NO_MAX, sum = 0.0f;
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (row < a.rows) {
    const int64_t step = (int64_t)a.c.heads * a.tiles * R, from = (int64_t)h * a.tiles * R + row;
    auto at = [&](int s) { return from + (s < whole ? full + s : rests) * step; };
    for (int s = c; s < parts; s += LPR) mm = fmaxf(mm, a.pm[2 * at(s)]);
    mm = group_max<LPR>(mm);
#pragma unroll 4
    for (int s = g; s < parts; s += GROUPS) {
      const int64_t p = at(s);
      const float f = __builtin_amdgcn_exp2f(a.pm[2 * p] - mm);
      sum += f * a.pm[2 * p + 1];
      v += f * *reinterpret_cast<const f32x4_t*>(a.po + p * DH + 4 * c);
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
  p.RT = rows > 16 && DH / GS < 4 ? 2 : 1;   // (four groups of scales for two rows do not fit)
  p.tiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  p.least = 256;
  p.target = 9;
  const int64_t per = heads * p.tiles;
  p.wide = p.RT == 1 && DH / GS < 4 && max_len > 256 && max_len <= 1024;
  p.whole = p.wide || max_len <= p.least || B * per >= int64_t(4) << p.target;
  p.groups = (B + (p.whole ? 0 : ((int64_t(1) << p.target) + per - 1) / per)) * per;
  return p;
}

template <int DH, int GS>
void launch(const AttnArgs& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.groups);
  if constexpr (DH / GS < 4) {
    if (p.RT == 2) {
      hipLaunchKernelGGL((k_kv4_attention<DH, GS, 2, 4>), grid, dim3(256), 0, st, a);
      return;
    }
    if (p.wide) {
      hipLaunchKernelGGL((k_kv4_attention<DH, GS, 1, 8>), grid, dim3(512), 0, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((k_kv4_attention<DH, GS, 1, 4>), grid, dim3(256), 0, st, a);
}
template <int DH>
void join(const AttnArgs& a, const Plan& p, hipStream_t st) {
  constexpr int ALL = NT / (DH / 4);
  const int64_t units = (int64_t)a.B * a.c.heads;
  if (units * a.rows >= 2048)
    hipLaunchKernelGGL((k_kv4_join<DH, 1>), dim3((unsigned)(units * ((a.rows + ALL - 1) / ALL))),
                       dim3(NT), 0, st, a, 16 * p.RT);
  else
    hipLaunchKernelGGL((k_kv4_join<DH, ALL>), dim3((unsigned)(units * a.rows)), dim3(NT), 0, st, a,
                       16 * p.RT);
}

}  // namespace

// Floats of the workspace: partial sums and (m, l) of every row of every workgroup.
int64_t ar_kv4_attention_floats(const ar_kv4_cache& c, int64_t B, int64_t news, int64_t heads,
                                int64_t max_len) {
  const Plan p = plan_of(B, c.heads, c.head_dim, c.group_size, news * (heads / c.heads), max_len);
  return p.whole ? 0 : p.groups * 16 * p.RT * (c.head_dim + 2);
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
  a.whole = p.whole;
  a.target = p.target;
  a.least = p.least;
  a.sl = (float)((double)g.scale * 1.4426950408889634);
  a.out = g.out;
  a.lse = g.lse;
  a.po = g.ws;
  a.pm = g.ws + p.groups * 16 * p.RT * c.head_dim;
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
