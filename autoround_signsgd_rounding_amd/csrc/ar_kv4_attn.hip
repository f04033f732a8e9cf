// Attention of each sequence's newest tokens over its pages of the 4-bit cache (gfx950),
// straight from the codes (layout: ar_kv4.h).
//
//   out = softmax(scale·q·Kᵀ)·V,   K = ks·(ck - kz), V = vs·(cv - vz) per group of channels
//
// The cache is read once and nothing else is large, so memory bounds it; what the codes
// cost on the way is kept below that. A code less its zero-point is a small integer, exact
// in f16, so the products run on v_mfma_f32_16x16x32_f16 with integers on the cache's side
// and the scales outside: ks multiplies the finished score, vs the weight. Two codes become
// two f16 in two instructions: (word & 0x000F000F) | 0x64006400 is 1024 + code twice, and
// one packed addition takes 1024 + zp off (the codes 4 bits up, 1024 + 16·code, by a packed
// fma with 1/16).
//
// q goes to f16 as q·2^k, its row's largest magnitude in [2^14, 2^15): exact but for what
// lies 2^-39 below that. A row is one query head of one new token; up to 16·RT rows share a
// key head's codes. Scores are formed transposed (A: 16 tokens, B: 16 rows), so a lane
// holds one row's scores of eight neighbouring tokens (8·(l/16) .. + 7 of 32, by the choice
// which token is which row of A), and these are the eight that it supplies to the second
// product, Oᵀ = Vᵀ·Pᵀ: nothing passes between lanes.
// The weights of that product are p·vs in f16, relative to the largest vs seen (Sv): half a
// step of 2^-11 each, an eighth of what rounding to bf16 would cost, and below 2^-31 of
// the largest nothing counts. p = 2^(x - m) with a running reference m that follows the maximum
// only when that has risen by more than 8 (p <= 256); the sums of p and all accumulators
// are float32.
//
// Each wave goes through its tokens alone, 32 at a time with the next 32 on their way in
// registers; the four waves of a workgroup are joined in LDS, and the workgroups that
// share a long sequence through the workspace, in order.
#include <math.h>

#include "ar_kv4.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256, WAVES = NT / 64;
constexpr float NO_MAX = -3.0e38f;
constexpr float RISE = 8.0f;      // m follows the maximum when that is so far above it
constexpr float W_TOP = 128.0f;   // weight of p = 1 at the largest vs: 2^15 at p = 2^RISE

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  ArKv4 c;
  const int32_t *table, *lengths;
  int width, max_len, B, news, heads, ratio, rows, tiles, splits, chunk;
  float sl;                // scale·log2 e
  uint16_t* out;
  float* lse;
  float *po, *pm;          // partial sums [split][b][tile][row][Dh] and (m, l) of each row
};

__device__ __forceinline__ uint32_t both(uint32_t w) { return w | (w << 16); }
__device__ __forceinline__ uint32_t minus(uint32_t w, uint32_t z) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, w) + __builtin_bit_cast(f16x2_t, z));
}
__device__ __forceinline__ uint32_t minus16(uint32_t w, uint32_t z) {
  const f16x2_t s = {(_Float16)0.0625f, (_Float16)0.0625f};
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, w), s,
                                                      __builtin_bit_cast(f16x2_t, z)));
}
constexpr uint32_t LOW = 0x000F000Fu, HIGH = 0x00F000F0u, ONE = 0x64006400u;

// Eight codes of one token, zero-point off; element 2i is code i, 2i + 1 code i + 4. z and
// z16: -(1024 + zp) and -(64 + zp) in both halves.
__device__ __forceinline__ f16x8_t keys_of(uint32_t w, uint32_t z, uint32_t z16) {
  const uint32_t u = w >> 8;
  const u32x4_t o = {minus((w & LOW) | ONE, z), minus16((w & HIGH) | ONE, z16),
                     minus((u & LOW) | ONE, z), minus16((u & HIGH) | ONE, z16)};
  return __builtin_bit_cast(f16x8_t, o);
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

// 32 tokens as they lie in memory.
template <int DH, int GS>
struct Tile {
  static constexpr int G = DH / GS, KW = GS / 32, NB = DH / 64;
  uint32_t k[2][G][KW];   // 16-token half j: the lane's token, its channels of each group
  float kz[2][G];         // that token's scales, for their zero-points
  float ks[8][G];         // scales of the octet's keys
  u32x4_t v[NB];          // the octet's values
  float vs[8][G];

  // pk, pv: the pages of the lane's key token and of its octet; tk: that token in its page
  // (half 0; half 1 is four on), tv: the octet's first.
  __device__ __forceinline__ void load(const ArKv4& c, int h, int64_t pk, int64_t pv, int tk,
                                       int tv, int g4, int n) {
    const int64_t rows = (int64_t)2 * c.heads * c.page;
    const int64_t krow = pk * rows + (int64_t)h * c.page, vrow = pv * rows + (int64_t)h * c.page;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint8_t* p = c.codes + (krow + tk + 4 * j) * (DH / 2) + g4 * (GS / 8);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (KW == 4) {
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p + g * (GS / 2));
#pragma unroll
          for (int i = 0; i < 4; ++i) k[j][g][i] = w[i];
        } else if constexpr (KW == 2) {
          const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + g * (GS / 2));
          k[j][g][0] = w[0];
          k[j][g][1] = w[1];
        } else {
          k[j][g][0] = *reinterpret_cast<const uint32_t*>(p + g * (GS / 2));
        }
        kz[j][g] = c.scale[(krow + tk + 4 * j) * G + g];
      }
    }
    scales(c.scale + (vrow + tv) * G, ks);
    const int64_t voff = (int64_t)c.heads * c.page;   // from a head's keys to its values
    const uint8_t* pvv = c.codes + (vrow + voff) * (DH / 2) + kv4_value_at(tv, 0, n, 0, NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) v[b] = *reinterpret_cast<const u32x4_t*>(pvv + b * 256);
    scales(c.scale + (vrow + voff + tv) * G, vs);
  }
  static __device__ __forceinline__ void scales(const float* p, float (&s)[8][G]) {
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const f32x4_t w = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[(4 * i + e) / G][(4 * i + e) % G] = w[e];
    }
  }
};

template <int DH, int GS, int RT>
__global__ __launch_bounds__(NT) void k_kv4_attention(AttnArgs a) {
  using Tl = Tile<DH, GS>;
  constexpr int G = Tl::G, KW = Tl::KW, NB = Tl::NB, NO = DH / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int Hk = a.c.heads, per = a.B * Hk * a.tiles;
  const int split = blockIdx.x / per, unit = blockIdx.x - split * per;
  const int tile = unit % a.tiles, bh = unit / a.tiles, h = bh % Hk, b = bh / Hk;
  const int len = min(max(a.lengths[b], 0), a.max_len);
  const int first = split * a.chunk, last = min(len, first + a.chunk);
  if (split && first >= len) return;   // the join leaves it out too

  // the lane's row of each of the RT products, its queries and what it sees
  f16x8_t qf[RT][G][KW];
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
    const int up = top == 0 || top >= 0x7F800000u ? 0 : 15 - __builtin_amdgcn_frexp_expf(big);
    qs[t] = ldexpf(a.sl, -up);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e)   // channel order of keys_of
          qf[t][g][k][e] = (_Float16)ldexpf(x[g][k][(e >> 1) + 4 * (e & 1)], up);
  }

  f32x4_t o[RT][NO];
  float m[RT], l[RT], sv[G], wk[G];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = NO_MAX;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < NO; ++d) o[t][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int g = 0; g < G; ++g) sv[g] = 0x1p-120f, wk[g] = W_TOP * 0x1p120f;

  const int32_t* tab = a.table + (int64_t)b * a.width;
  auto page_of = [&](int t) {   // page of token t, -1 where there is none
    const int at = t >> a.c.shift;
    const int p = at < a.width ? tab[at] : -1;
    return (uint32_t)p < (uint64_t)a.c.pages ? p : -1;
  };
  const int ktok = 8 * (n >> 2) + (n & 3), vtok = 8 * g4;   // the lane's tokens in a tile
  auto load = [&](Tl& x, int t, int p0, int p1) {
    const int mask = a.c.page - 1, in = t & mask, step = a.c.page == 16 ? 16 : 0;
    const int64_t pk = max(ktok >= 16 ? p1 : p0, 0), pv = max(vtok >= 16 ? p1 : p0, 0);
    // tokens 16.. of the tile start their page anew where a page is 16 tokens
    x.load(a.c, h, pk, pv, in + ktok - (ktok >= 16 ? step : 0), in + vtok - (vtok >= 16 ? step : 0),
           g4, n);
  };
  auto work = [&](const Tl& x, int t0, int p0, int p1) {
    // scores: x[t][e] of token t0 + 8·g4 + e
    float s[RT][8];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t zp = kv4_zero(x.kz[j][g]);
        const uint32_t z = both(0xE400u | zp), z16 = both(0xD400u | (zp << 4));
        f32x4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const f16x8_t f = keys_of(x.k[j][g][k], z, z16);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, qf[t][g][k], acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            s[t][4 * j + r] = g == 0 ? acc[t][r] * x.ks[4 * j + r][g]
                                     : fmaf(acc[t][r], x.ks[4 * j + r][g], s[t][4 * j + r]);
      }
    float vs[8][G];
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int g = 0; g < G; ++g) vs[e][g] = x.vs[e][g];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[t][e] *= qs[t];
    const bool bad = p0 < 0 || p1 < 0;
    if (bad || t0 + 32 > len - a.news + 1) {   // some token is hidden from some row
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
      rises |= top[t] > m[t] + RISE;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      vtop[g] = vs[0][g];
#pragma unroll
      for (int e = 1; e < 8; ++e) vtop[g] = fmaxf(vtop[g], vs[e][g]);
      rises |= vtop[g] > sv[g];
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
    }
    // weights p·vs, eight tokens of the lane's row
    f16x8_t w[RT][G];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(s[t][e] - m[t]);
        l[t] += p[e];
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[t][g][e] = (_Float16)(p[e] * (vs[e][g] * wk[g]));
    }
    if (bad || t0 + 32 > len - a.news + 1) {   // hidden tokens weigh nothing, whatever they hold
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (s[t][e] == -INFINITY)
#pragma unroll
            for (int g = 0; g < G; ++g) w[t][g][e] = (_Float16)0.0f;
    }
    uint32_t z[G][4], z16[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t zp = kv4_zero(x.vs[2 * i][g]) | (kv4_zero(x.vs[2 * i + 1][g]) << 16);
        z[g][i] = zp | 0xE400E400u;
        z16[g][i] = (zp << 4) | 0xD400D400u;
      }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int g = (64 * b + 32 * c) / GS;
        u32x4_t lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = c ? x.v[b][i] >> 8 : x.v[b][i];
          lo[i] = minus((u & LOW) | ONE, z[g][i]);
          hi[i] = minus16((u & HIGH) | ONE, z16[g][i]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4_t* d = &o[t][4 * b + 2 * c];
          d[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, lo), w[t][g],
                                                        d[0], 0, 0, 0);
          d[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, hi), w[t][g],
                                                        d[1], 0, 0, 0);
        }
      }
  };

  constexpr int STEP = 32 * WAVES;
  int t = first + 32 * wave;
  if (t < last) {
    Tl x;
    int p0 = page_of(t), p1 = page_of(t + 16);
    load(x, t, p0, p1);
    int n0 = page_of(t + STEP), n1 = page_of(t + STEP + 16);
    for (; t < last; t += STEP) {
      Tl y;
      if (t + STEP < last) load(y, t + STEP, n0, n1);
      const int f0 = page_of(t + 2 * STEP), f1 = page_of(t + 2 * STEP + 16);
      work(x, t, p0, p1);
      x = y;
      p0 = n0, p1 = n1, n0 = f0, n1 = f1;
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
      const float k = sv[16 * d / GS] * (1.0f / W_TOP);
#pragma unroll
      for (int r = 0; r < 4; ++r)   // channel 32·(d/2) + 2·(4·g4 + r) + d%2
        so[wave][row][32 * (d >> 1) + 2 * (4 * g4 + r) + (d & 1)] = o[t][d][r] * k;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (DH / 4); e += NT) {
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
    if (a.splits > 1) {
      const int64_t to = (int64_t)blockIdx.x * R + row;
      *reinterpret_cast<f32x4_t*>(a.po + to * DH + c) = v;
      if (c == 0) a.pm[2 * to] = mm, a.pm[2 * to + 1] = sum;
    } else {
      const int i = at / a.ratio;
      const int64_t to = ((int64_t)b * a.news + i) * a.heads + h * a.ratio + at - i * a.ratio;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees no key is 0
      *reinterpret_cast<u32x2_t*>(a.out + to * DH + c) =
          u32x2_t{bf16_pair(v[0] * inv, v[1] * inv), bf16_pair(v[2] * inv, v[3] * inv)};
      if (a.lse && c == 0)
        a.lse[to] = sum == 0.0f ? -INFINITY : 0.69314718f * (mm + __log2f(sum));
    }
  }
}

// Joins the splits of each row, in their order.
template <int DH>
__global__ __launch_bounds__(NT) void k_kv4_join(AttnArgs a, int R) {
  constexpr int LPR = DH / 4;
  const int64_t id = ((int64_t)blockIdx.x * NT + threadIdx.x) / LPR;
  const int c = 4 * (threadIdx.x % LPR);
  const int64_t per = (int64_t)a.B * a.c.heads * a.tiles;
  const int64_t unit = id / R;
  const int row = (int)(id - unit * R);
  if (unit >= per) return;
  const int tile = (int)(unit % a.tiles), bh = (int)(unit / a.tiles);
  const int h = bh % a.c.heads, b = bh / a.c.heads, at = tile * R + row;
  if (at >= a.rows) return;
  const int len = min(max(a.lengths[b], 0), a.max_len);
  const int used = max(1, (len + a.chunk - 1) / a.chunk);
  float mm = NO_MAX, sum = 0.0f;
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < used; ++s) {
    const int64_t from = (s * per + unit) * R + row;
    const float ms = a.pm[2 * from], ls = a.pm[2 * from + 1];
    const float mn = fmaxf(mm, ms), f = __builtin_amdgcn_exp2f(mm - mn),
                g = __builtin_amdgcn_exp2f(ms - mn);
    mm = mn;
    sum = sum * f + ls * g;
    v = v * f + g * *reinterpret_cast<const f32x4_t*>(a.po + from * DH + c);
  }
  const int i = at / a.ratio;
  const int64_t to = ((int64_t)b * a.news + i) * a.heads + h * a.ratio + at - i * a.ratio;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2_t*>(a.out + to * DH + c) =
      u32x2_t{bf16_pair(v[0] * inv, v[1] * inv), bf16_pair(v[2] * inv, v[3] * inv)};
  if (a.lse && c == 0) a.lse[to] = sum == 0.0f ? -INFINITY : 0.69314718f * (mm + __log2f(sum));
}

struct Plan {
  int RT, tiles, splits, chunk;
};
Plan plan_of(int64_t B, int64_t heads, int64_t rows, int64_t max_len) {
  Plan p;
  p.RT = rows > 16 ? 2 : 1;
  p.tiles = (int)((rows + 16 * p.RT - 1) / (16 * p.RT));
  const int64_t units = B * heads * p.tiles;
  const int64_t want = units >= 4096 ? 1 : (4096 + units - 1) / units;
  const int64_t most = (max_len + 255) / 256;
  int64_t splits = want < most ? want : most;
  if (splits < 1) splits = 1;
  const int64_t chunk = ((max_len + splits - 1) / splits + 127) / 128 * 128;
  p.chunk = (int)(chunk < 128 ? 128 : chunk);
  p.splits = (int)((max_len + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}

template <int DH, int GS>
void launch(const AttnArgs& a, int RT, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.B * a.c.heads * a.tiles * a.splits));
  if (RT == 2) hipLaunchKernelGGL((k_kv4_attention<DH, GS, 2>), grid, dim3(NT), 0, st, a);
  else hipLaunchKernelGGL((k_kv4_attention<DH, GS, 1>), grid, dim3(NT), 0, st, a);
}

}  // namespace

// Floats of the workspace: partial sums and (m, l) of every row and split; 0 for one split.
int64_t ar_kv4_attention_floats(const ar_kv4_cache& c, int64_t B, int64_t news, int64_t heads,
                                int64_t max_len) {
  const Plan p = plan_of(B, c.heads, news * (heads / c.heads), max_len);
  if (p.splits == 1) return 0;
  return B * c.heads * p.tiles * p.splits * 16 * p.RT * (c.head_dim + 2);
}

ar_status ar_launch_kv4_attention(const ArKv4Attention& g, hipStream_t st) {
  const ar_kv4_cache& c = *g.cache;
  const int64_t rows = g.news * (g.heads / c.heads);
  const Plan p = plan_of(g.B, c.heads, rows, g.max_len);
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
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.sl = (float)((double)g.scale * 1.4426950408889634);
  a.out = g.out;
  a.lse = g.lse;
  a.po = g.ws;
  const int64_t units = g.B * c.heads * p.tiles, R = 16 * p.RT;
  a.pm = g.ws + units * p.splits * R * c.head_dim;
  const int DH = c.head_dim, GS = c.group_size;
  if (DH == 64 && GS == 32) launch<64, 32>(a, p.RT, st);
  else if (DH == 64) launch<64, 64>(a, p.RT, st);
  else if (GS == 32) launch<128, 32>(a, p.RT, st);
  else if (GS == 64) launch<128, 64>(a, p.RT, st);
  else launch<128, 128>(a, p.RT, st);
  if (p.splits > 1) {
    const dim3 grid((unsigned)((units * R * (DH / 4) + NT - 1) / NT));
    if (DH == 64) hipLaunchKernelGGL((k_kv4_join<64>), grid, dim3(NT), 0, st, a, (int)R);
    else hipLaunchKernelGGL((k_kv4_join<128>), grid, dim3(NT), 0, st, a, (int)R);
  }
  return last_status();
}
