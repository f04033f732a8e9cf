// Causal attention over packed sequences with grouped heads (gfx950):
//   out = softmax(scale·q·kᵀ)·v,  query i of a sequence of Lq queries and Lk keys seeing
//   the keys 0 .. i + Lk - Lq.
//
// A workgroup takes 128 rows, 32 a wave, of one sequence and key head. Rows are the
// queries of all the heads that share it, token by token: keys and values are staged once
// for the group, and a short prompt fills a tile with its heads. Keys and values pass
// through LDS in tiles of 64 or 32 tokens, two stages, loaded straight to LDS, their 16-byte
// chunks turned by the row so that no read meets a bank twice. Tiles that every row sees whole
// go through a loop without masks. A sequence's last rows, which see the most keys, come first.
//
// Scores are formed transposed, Sᵀ = K·Qᵀ on v_mfma_f32_32x32x16_bf16, so a lane holds one
// row's scores of half the tile's tokens. Which token is which row of K is chosen so that
// the lane's scores 8i .. 8i + 7 are neighbouring tokens, which are the eight that it
// supplies as the B operand of Oᵀ = Vᵀ·Pᵀ: the weights stay where they are. The A operand
// there is V transposed, which ds_read_b64_tr_b16 gives out of V as it lies in memory.
// p = 2^(s - m) <= 1 with a running reference m, a whole number, that is set 8 above the maximum
// when that has passed it; p is rounded to bf16 for the product (2^-8 of each weight, about as
// much in the output as its own rounding to bf16) or, where the caller asks for float32 weights,
// taken in three bf16 parts; the sums of p and all accumulators are float32.
//
// The matrix unit and what feeds it bound long prompts. Measured, counting the causal half:
// 16384 tokens, 64 heads of 128 over 8: 3694 us, 1.19 PFLOP/s (a large library product: 1.23),
// the unit busy 71% of the cycles at 1.58 GHz; 8 x 2048 tokens, 32 heads of 128: 302 us, 0.91
// PFLOP/s, where 4096 workgroups go in 5.3 rounds and each has 34 tiles of 32 keys in the mean;
// 16384 tokens, 32 heads of 64 over 8: 1100 us, 1.0 PFLOP/s, half as much product for each
// exponential; 37 tokens: 5 us, a launch and the first loads.
#include <math.h>

#include <type_traits>

#include "ar_device.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256, BM = 128;
constexpr int GRAIN = 64;   // parts of the keys are a multiple of that
// With few tiles the keys are divided: workgroups wanted, keys of one at least. A part costs its
// rows in float32, written and read, as much as 256 keys and values at 128 channels. (8 heads of 128,
// 4096 tokens: 55.7 us, 512 wanted 63.8, 1024 77.0; 4 heads over 1, 8192 tokens: 91.8, 113 and 123.
// 64 tokens behind 16000, 32 heads over 8: 38.5, parts of 512 keys 49.0; 2048 tokens, 8 heads:
// 31.6, parts of 768 keys 33.3.)
constexpr int TARGET = 768, LEAST = 1024;
constexpr int PER = 8;       // workgroups that join the parts of a tile (64 tokens behind 16000:
                             // 38.6 us; 4 of them 48.7)
constexpr int MANY = 768;    // workgroups from which on tiles are of 32 keys
constexpr float NO_MAX = -3.0e38f;
constexpr float FAR = 0x1p24f;  // a reference whose rounding 2^x would feel
constexpr float RISE = 8.0f;   // m lies so far above the maximum when it is set

typedef short s16x4_t __attribute__((ext_vector_type(4)));

#define AR_LDS(p) ((__attribute__((address_space(3))) void*)(p))

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct Args {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *q_off, *k_off;
  int64_t Tq, Tk;
  int B, heads, kv_heads, ratio;
  float sl;       // scale·log2 e
  uint16_t* out;
  float* lse;
  float *po, *pm; // partial sums [workgroup][row][Dh] and (m, l) of each row
  int64_t groups; // of those
};

// Sequence b's queries and keys, by offsets that lead nowhere outside the arrays.
struct Seq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  s.q0 = min(max(a.q_off[b], 0), (int)a.Tq);
  s.nq = min(max(a.q_off[b + 1], s.q0), (int)a.Tq) - s.q0;
  s.k0 = min(max(a.k_off[b], 0), (int)a.Tk);
  s.nk = min(max(a.k_off[b + 1], s.k0), (int)a.Tk) - s.k0;
  return s;
}

__device__ __forceinline__ int tiles_of(const Args& a, const Seq& s) {
  return (int)(((int64_t)s.nq * a.ratio + BM - 1) / BM);
}
// Tokens of the parts into which the keys are divided where there are few tiles: TARGET
// parts over all tiles and key heads, the same for every workgroup.
__device__ __forceinline__ int chunk_of(const Args& a) {
  float work = 0.0f;   // (rounded alike everywhere)
  for (int b = threadIdx.x & 63; b < a.B; b += 64) {
    const Seq s = seq_of(a, b);
    work += (float)tiles_of(a, s) * (float)s.nk;
  }
  // (above the quotient whatever the roundings, so that there are no more parts than workgroups)
  const float each = wave_total(wave_scan(work)) * (float)a.kv_heads * (1.001f / TARGET) + 1.0f;
  const int c = (int)fminf(fmaxf(each, (float)LEAST), 0x1p30f);
  return __builtin_amdgcn_readfirstlane((c + GRAIN - 1) / GRAIN * GRAIN);
}
// Unit `at` of the sequences' rows cut into tiles of BM (a sequence's last tile, the longest,
// first) and these (chunk > 0) into parts of the keys: its sequence, first row, part, and the
// units before its tile. `whole`: the count goes over tiles. False when there is no such unit.
struct Unit {
  int b, r0, part;
  int64_t before;
};
__device__ __forceinline__ bool find_unit(const Args& a, int chunk, int at, bool whole, Unit& u) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  int64_t units = 0;
  for (int base = 0; base < a.B; base += 64) {
    int tiles = 0, parts = 1;
    if (base + lane < a.B) {
      const Seq s = seq_of(a, base + lane);
      tiles = tiles_of(a, s);
      if (chunk) parts = max(1, (int)(((uint32_t)s.nk + (uint32_t)chunk - 1) / (uint32_t)chunk));
    }
    // (overlapping sequences may count more than there can be: bounded, so that 64 fit an int)
    const int n = (int)min((int64_t)tiles * (whole ? 1 : parts), (int64_t)1 << 24);
    const int m = (int)min((int64_t)tiles * parts, (int64_t)1 << 24);
    const int sum = wave_scan(n), all = whole && chunk ? wave_scan(m) : sum;
    const uint64_t past = __ballot(before + sum > at);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int local = at - before - __builtin_amdgcn_readlane(sum - n, l);
      const int p = __builtin_amdgcn_readlane(parts, l), tile = whole ? local : local / p;
      u.b = base + l;
      u.r0 = (__builtin_amdgcn_readlane(tiles, l) - 1 - tile) * BM;
      u.part = whole ? 0 : local - tile * p;
      u.before = units + __builtin_amdgcn_readlane(all - m, l) + (int64_t)tile * p;
      return true;
    }
    before += wave_total(sum);
    units += wave_total(all);
  }
  return false;
}

// Tile `at` of at most 64 sequences' tiles: sequence by sequence, so that workgroups that run
// together read the same keys, a sequence's last tile first, and those of a quarter of the most
// keys or less after all others, so that the last workgroups to end are short ones. (60 x up to
// 700 tokens, 32 heads over 8: 71.2 us instead of 75.7 without that; 8 x 2048, 32 heads of 64: 175
// and 180. In the order of the keys throughout 76.8 and 190, and 8 x 2048, 32 heads of 128, 348
// instead of 312.)
__device__ __forceinline__ bool find_tile(const Args& a, int at, Unit& u) {
  const int lane = threadIdx.x & 63;
  int tiles = 0, top = 0;   // the lane's sequence: its tiles, and those its keys would make
  if (lane < a.B) {
    const Seq s = seq_of(a, lane);
    tiles = tiles_of(a, s);   // (2^23 at most, as Tq·heads < 2^30)
    top = (int)min((int64_t)max(s.nk - s.nq, 0) * a.ratio / BM, (int64_t)1 << 23) + tiles;
  }
  const int cut = (int)group_max<64>((float)top) / 4;
  const int early = min(max(top - cut, 0), tiles);
  const int sum = wave_scan(early), all = wave_total(sum);
  const bool late = at >= all;
  const int n = late ? tiles - early : early, upto = late ? wave_scan(n) : sum;
  const int in = late ? at - all : at;
  const uint64_t past = __ballot(upto > in);
  if (!past) return false;
  const int l = __ffsll((unsigned long long)past) - 1;
  const int local = in - __builtin_amdgcn_readlane(upto - n, l);
  u.b = l;
  u.r0 = (__builtin_amdgcn_readlane(late ? n : tiles, l) - 1 - local) * BM;
  u.part = 0;
  u.before = 0;
  return true;
}

// ln of the sum of exponentials from the sum l relative to 2^m.
__device__ __forceinline__ float row_lse(float m, float l) {
  return 0.69314718f * (m - RISE + __log2f(ldexpf(l, (int)RISE)));
}

__device__ __forceinline__ bool finite_bits(uint32_t pair) {
  return (pair & 0x7F80u) != 0x7F80u && (pair & 0x7F800000u) != 0x7F800000u;
}

// One row by the definition over the keys first .. last, by one wave: for a row whose product
// met an infinity or a NaN of a value hidden from it (0·inf), or whose reference is beyond FAR
// (scores are rounded here before they are compared). The lane takes the channels
// lane, lane + 64 of o. False once all of o is NaN, if `early`, m and l then being those of the
// keys so far.
template <int DH>
__device__ __forceinline__ bool plain_row(const Args& a, const uint16_t* q, const uint16_t* k,
                                          const uint16_t* v, int first, int last, bool early, float& m,
                                          float& l, float (&o)[DH / 64]) {
  const int lane = threadIdx.x & 63;
  m = NO_MAX, l = 0.0f;
#pragma unroll
  for (int d = 0; d < DH / 64; ++d) o[d] = 0.0f;
  for (int t0 = first; t0 <= last; t0 += 64) {
    float s = -INFINITY;
    if (t0 + lane <= last) {
      const uint16_t* kr = k + (int64_t)(t0 + lane) * a.k_stride;
      s = 0.0f;
#pragma unroll 4
      for (int d = 0; d < DH; d += 8) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(q + d);
        const u32x4_t y = *reinterpret_cast<const u32x4_t*>(kr + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), s);
          s = fmaf(__uint_as_float(x[e] & 0xFFFF0000u), __uint_as_float(y[e] & 0xFFFF0000u), s);
        }
      }
      s *= a.sl;
    }
    const float mn = fmaxf(m, group_max<64>(s)), by = exp2f(m - mn);
    m = mn;
    const float p = t0 + lane <= last ? exp2f(s - m) : 0.0f;
    l = l * by + group_sum<64>(p);
#pragma unroll
    for (int d = 0; d < DH / 64; ++d) o[d] *= by;
    const int n = min(64, last + 1 - t0);
    for (int j0 = 0; j0 < n; j0 += 16) {   // (16 loads at a time)
      float x[16][DH / 64];
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int d = 0; d < DH / 64; ++d)
          x[j][d] = bf16_val(v[(int64_t)(t0 + min(j0 + j, n - 1)) * a.v_stride + lane + 64 * d]);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j0 + j < n) {
          const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), j0 + j));
#pragma unroll
          for (int d = 0; d < DH / 64; ++d) o[d] = fmaf(w, x[j][d], o[d]);
        }
    }
    bool lost = true;
#pragma unroll
    for (int d = 0; d < DH / 64; ++d) lost = lost && o[d] != o[d];
    if (early && __all(lost)) return false;
  }
  return true;
}

// KT keys a tile. 64 wait less often; 32 leave registers and LDS for a third workgroup on a
// CU, which pays where there are more of them than run at once (heads of 128; 16384 tokens, 64 over
// 8: 3720 us instead of 3887; 4096, 32 over 8: 135 and 146; 3000: 83.1 and 80.8; 2048: 48.8 and
// 47.8). With 64 channels four workgroups fit anyway (16384 tokens, 32 heads over 8: 1127 us
// instead of 1100).
//
// SPLIT: parts of a weight, 1 or 3 (16384 tokens, 64 over 8: 6972 us instead of 3923; 8 x 2048, 32
// heads: 492 and 302).
template <int DH, bool PARTS, int KT, int SPLIT>
__global__ __launch_bounds__(NT, KT == 32 ? 3 : 2) void k_attention_packed(Args a) {
  constexpr int C = DH / 8, ROW = 2 * DH;          // 16-byte chunks and bytes of a row
  constexpr int TILE = KT * ROW;                   // bytes of a tile of keys or values
  constexpr int LD = TILE / (NT * 16), LROWS = NT / C;   // loads a wave, rows between them
  constexpr int ND = DH / 32, NC = DH / 16;
  // Two stages of keys and values. With an array for each, the long loop going by twos, the
  // values' reads need not wait for the next tile's loads (16384 tokens, 64 heads of 128 over 8:
  // 3717 us instead of 3787). With 64 channels the registers for that cost a workgroup on each CU (8 x
  // 2048, 32 heads: 177 us instead of 173).
  constexpr bool APART = DH == 128;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[(APART ? 2 : 4) * TILE];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[APART ? 2 * TILE : 16];

  const int kvh = blockIdx.x % a.kv_heads, at = blockIdx.x / a.kv_heads;
  const int chunk = PARTS ? chunk_of(a) : 0;
  Unit un;
  const bool some = !PARTS && a.B > 1 && a.B <= 64;
  if (!(some ? find_tile(a, at, un) : find_unit(a, chunk, at, !PARTS, un))) return;
  const int b = un.b, r0 = un.r0;
  const Seq sq = seq_of(a, b);
  const int nk = __builtin_amdgcn_readfirstlane(sq.nk), nq = __builtin_amdgcn_readfirstlane(sq.nq);
  const int k0 = __builtin_amdgcn_readfirstlane(sq.k0), q0 = __builtin_amdgcn_readfirstlane(sq.q0);
  const int rows = nq * a.ratio;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l31 = lane & 31, half = lane >> 5;

  // the lane's row: query i of the sequence, seeing keys 0 .. last
  const int row = r0 + 32 * wave + l31, i = min(row, rows - 1) / a.ratio;
  const int head = kvh * a.ratio + min(row, rows - 1) - i * a.ratio;
  const int last = i + nk - nq;
  // what the workgroup, and what every row of the wave, sees
  const int wrow0 = r0 + 32 * wave;
  const int kall = min((min(r0 + BM, rows) - 1) / a.ratio + nk - nq + 1, nk);
  const int kfirst = PARTS ? un.part * chunk : 0;
  if (kfirst > 0 && kfirst >= kall) return;   // (the join leaves it out too)
  const int kend = PARTS ? min(kall, kfirst + chunk) : kall;
  const bool joined = PARTS && kall > chunk;
  const int wfirst = min(wrow0, rows - 1) / a.ratio + nk - nq;                    // least of last
  const int wend = wrow0 < rows ? (min(wrow0 + 32, rows) - 1) / a.ratio + nk - nq + 1 : 0;

  // loads: chunk p of a tile lies at its place with the chunk number turned by the row, so
  // that the reads below meet 64 different banks
  const int lrow = threadIdx.x / C, lpos = threadIdx.x % C;
  const int kswz = C == 16 ? lrow & 15 : (lrow >> 1) & 7;
  const int vswz = C == 16 ? (lrow & 3) << 2 : ((lrow >> 1) & 1) << 2;
  const uint32_t kvo = (uint32_t)(lrow * a.k_stride * 2 + ((lpos ^ kswz) << 4));
  const uint32_t vvo = (uint32_t)(lrow * a.v_stride * 2 + ((lpos ^ vswz) << 4));
  const uint16_t* kb = a.k + (int64_t)k0 * a.k_stride + kvh * DH;
  const uint16_t* vb = a.v + (int64_t)k0 * a.v_stride + kvh * DH;
  auto stage = [&](int t0, uint8_t* to) {
    const int n = min(nk - t0, KT);
    const auto bk = make_rsrc(kb + (int64_t)t0 * a.k_stride,
                              (uint32_t)(((n - 1) * a.k_stride + DH) * 2));
    const auto bv = make_rsrc(vb + (int64_t)t0 * a.v_stride,
                              (uint32_t)(((n - 1) * a.v_stride + DH) * 2));
#pragma unroll
    for (int j = 0; j < LD; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bk, AR_LDS(to + (j * 4 + wave) * 1024), 16,
                                               kvo + (uint32_t)(j * LROWS * a.k_stride * 2), 0, 0, 0);
#pragma unroll
    for (int j = 0; j < LD; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bv, AR_LDS(to + TILE + (j * 4 + wave) * 1024), 16,
                                               vvo + (uint32_t)(j * LROWS * a.v_stride * 2), 0, 0, 0);
  };

  if (kend > kfirst) stage(kfirst, lds0);

  const uint16_t* qp = a.q + (int64_t)(q0 + i) * a.q_stride + head * DH;
  bf16x8_t qf[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) qf[c] = *reinterpret_cast<const bf16x8_t*>(qp + 16 * c + 8 * half);

  // reads: key row of the lane (row r of the product is the token that puts neighbouring
  // tokens side by side in a lane's scores), chunk 2c + half
  const int kr = 16 * (l31 >> 4) + 8 * ((l31 >> 2) & 1) + 4 * ((l31 >> 3) & 1) + (l31 & 3);
  const int krs = C == 16 ? kr & 15 : (kr >> 1) & 7;
  int kat[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) kat[c] = kr * ROW + (((2 * c + half) ^ krs) << 4);
  // values: 16 lanes take 4 tokens x 16 channels, transposed
  const int l15 = lane & 15, vk = 8 * half + (l15 >> 2), dh16 = (lane >> 4) & 1;
  int vat[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    const int chunk = 4 * d + 2 * dh16 + ((l15 & 3) >> 1);
    const int sw = C == 16 ? (vk & 3) << 2 : ((vk >> 1) & 1) << 2;
    vat[d] = vk * ROW + ((chunk ^ sw) << 4) + 8 * (l15 & 1);
  }

  f32x16_t o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
  float m = NO_MAX, l = 0.0f;

  auto work = [&](auto masked, int t0, const uint8_t* lk, const uint8_t* lv) {
    f32x16_t s[KT / 32];
#pragma unroll
    for (int j = 0; j < KT / 32; ++j) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[j][r] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const bf16x8_t f = *reinterpret_cast<const bf16x8_t*>(lk + kat[c] + j * 32 * ROW);
        s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, qf[c], s[j], 0, 0, 0);
      }
    }
    if constexpr (decltype(masked)::value) {
#pragma unroll
      for (int j = 0; j < KT / 32; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (t0 + 32 * j + 16 * (r >> 3) + 8 * half + (r & 7) > last) s[j][r] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int j = 0; j < KT / 32; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[j][r]);
    top *= a.sl;
    if (__any(top > m)) {
      const float mn = fmaxf(m, ceilf(fmaxf(top, __shfl_xor(top, 32, 64))) + RISE);
      const float by = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= by;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= by;
    }
    u32x4_t p[SPLIT][KT / 16];
#pragma unroll
    for (int j = 0; j < KT / 32; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        float e0 = __builtin_amdgcn_exp2f(fmaf(s[j][r], a.sl, -m));
        float e1 = __builtin_amdgcn_exp2f(fmaf(s[j][r + 1], a.sl, -m));
        l += e0 + e1;
#pragma unroll
        for (int i = 0; i < SPLIT; ++i) {
          const uint32_t w = bf16_pair(e0, e1);
          p[i][2 * j + (r >> 3)][(r & 7) >> 1] = w;
          e0 -= __uint_as_float(w << 16);   // exact
          e1 -= __uint_as_float(w & 0xFFFF0000u);
        }
      }
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        typedef __attribute__((address_space(3))) s16x4_t* tr;
        const uint8_t* at = lv + vat[d] + 16 * kk * ROW;
        const s16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr)(at));
        const s16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr)(at + 4 * ROW));
        const auto f = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < SPLIT; ++i)
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                         __builtin_bit_cast(bf16x8_t, p[i][kk]),
                                                         o[d], 0, 0, 0);
      }
  };

  int t0 = kfirst;
  auto step = [&](auto masked, uint8_t* now, uint8_t* next) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // this wave's loads of the tile (vmcnt 0)
    __syncthreads();                      // everybody's; and the other stage has been read
    if (t0 + KT < kend) stage(t0 + KT, next);
    if (!decltype(masked)::value || t0 < wend) work(masked, t0, now, now + TILE);
    t0 += KT;
  };
  // tiles that every row of the workgroup sees whole, then the others
  const int full = min(r0 / a.ratio + nk - nq + 1, kend) - KT;
  int s = 0;
  auto of = [&](int s) { return APART ? s ? lds1 : lds0 : lds0 + s * 2 * TILE; };
  while (t0 <= full) {
    if constexpr (APART) {
      step(std::false_type(), lds0, lds1);
      if (t0 > full) {
        s = 1;
        break;
      }
      step(std::false_type(), lds1, lds0);
    } else {
      step(std::false_type(), of(s), of(s ^ 1));
      s ^= 1;
    }
  }
  for (; t0 < kend; s ^= 1) step(std::true_type(), of(s), of(s ^ 1));

  l += __shfl_xor(l, 32, 64);
  // A row that sees no key is 0: its weights of 0 have met whatever the others' values hold.
  const bool none = last < 0;
  if (none)
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
  const int64_t to = (int64_t)(q0 + i) * a.heads + head;
  const int64_t slot = ((int64_t)at * a.kv_heads + kvh) * BM, pto = slot + 32 * wave + l31;
  if (row < rows && joined) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f32x4_t*>(a.po + pto * DH + 32 * d + 8 * r + 4 * half) =
            f32x4_t{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
    if (half == 0) a.pm[2 * pto] = m, a.pm[2 * pto + 1] = l;
  } else if (row < rows) {
    const float inv = none ? 0.0f : 1.0f / l;
    uint16_t* op = a.out + to * DH + 4 * half;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<u32x2_t*>(op + 32 * d + 8 * r) =
            u32x2_t{bf16_pair(o[d][4 * r] * inv, o[d][4 * r + 1] * inv),
                    bf16_pair(o[d][4 * r + 2] * inv, o[d][4 * r + 3] * inv)};
    if (a.lse && half == 0) a.lse[to] = none ? -INFINITY : row_lse(m, l);
  }

  // An infinity or a NaN among the values of a tile meets weights of 0 in the rows that do
  // not see it, and makes them NaN: such rows are done again.
  float big = 0.0f;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      big = __builtin_elementwise_maximum(big, fabsf(o[d][r]));
  // And so are rows with a reference beyond FAR: half a step of it, which the product within
  // an fma does not share, is more than 2^x holds. (An infinite one has made NaN of its row.)
  const bool far = row < rows && fabsf(m) >= FAR && m != NO_MAX && m != INFINITY;
  const bool off = row < rows && !(big < INFINITY);
  auto of_rows = [&](bool x) {   // both halves of the wave hold the row
    const uint64_t w = __ballot(x);
    return (w | (w >> 32)) & 0xFFFFFFFFull;
  };
  const uint64_t fars = of_rows(far), offs = of_rows(off);
  uint64_t redo = fars;
  if (offs & ~fars) {
    bool found = false;   // (keys beyond the wave's rows, and so hidden from some of them)
    for (int t = max(wfirst + 1, kfirst) + lane; t < min(nk, (kend + KT - 1) / KT * KT); t += 64) {
      const uint16_t* vr = vb + (int64_t)t * a.v_stride;
      for (int d = 0; d < DH; d += 2)
        found |= !finite_bits(*reinterpret_cast<const uint32_t*>(vr + d));
    }
    if (__any(found)) redo |= offs;
  }
  if (redo) {
    __threadfence();   // behind the stores above
    while (redo) {
      const int r = __ffsll((unsigned long long)redo) - 1;
      redo &= redo - 1;
      const int ri = __shfl(i, r, 64), rh = __shfl(head, r, 64);
      const bool sums = (fars >> r) & 1;   // m and l have to be done again too
      float rm, rl, ro[DH / 64];
      const bool all =
          plain_row<DH>(a, a.q + (int64_t)(q0 + ri) * a.q_stride + rh * DH, kb, vb, kfirst,
                        min(ri + nk - nq, kend - 1), !sums, rm, rl, ro);
      const int64_t rto = (int64_t)(q0 + ri) * a.heads + rh;
      const int64_t rpto = slot + 32 * wave + r;
#pragma unroll
      for (int d = 0; d < DH / 64; ++d)
        if (joined) a.po[rpto * DH + lane + 64 * d] = ro[d];
        else a.out[rto * DH + lane + 64 * d] = (uint16_t)bf16_bits(ro[d] / rl);
      if (all && lane == 0) {
        if (joined) a.pm[2 * rpto] = rm, a.pm[2 * rpto + 1] = rl;
        else if (sums && a.lse) a.lse[rto] = row_lse(rm, rl);
      }
    }
  }
}

// Joins the parts of a tile's rows, where there are several: Dh/4 lanes a row, four channels
// each, the parts in order. Every row there sees a key: the last of the tile more than LEAST,
// the others at most BM fewer.
static_assert(LEAST >= BM);
template <int DH>
__global__ __launch_bounds__(NT) void k_attention_join(Args a) {
  constexpr int LPR = DH / 4, ROWS = NT / LPR;
  const int tile = blockIdx.x / PER, kvh = tile % a.kv_heads;
  const int chunk = chunk_of(a);
  Unit un;
  if (!find_unit(a, chunk, tile / a.kv_heads, true, un)) return;
  const Seq s = seq_of(a, un.b);
  const int rows = s.nq * a.ratio, c = threadIdx.x % LPR;
  const int kall = min((min(un.r0 + BM, rows) - 1) / a.ratio + s.nk - s.nq + 1, s.nk);
  if (kall <= chunk) return;   // a single part has written its rows
  const int parts = (kall + chunk - 1) / chunk;
  if ((un.before + parts) * a.kv_heads > a.groups) return;   // (overlapping sequences)
  const int first = (blockIdx.x - tile * PER) * (BM / PER) + threadIdx.x / LPR;
  for (int in = first; in < first + BM / PER && un.r0 + in < rows; in += ROWS) {
    const int row = un.r0 + in;
    auto at = [&](int p) { return ((int64_t)(un.before + p) * a.kv_heads + kvh) * BM + in; };
    float m = NO_MAX, sum = 0.0f;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < parts; ++p) m = fmaxf(m, a.pm[2 * at(p)]);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float f = __builtin_amdgcn_exp2f(a.pm[2 * at(p)] - m);
      sum += f * a.pm[2 * at(p) + 1];
      v += f * *reinterpret_cast<const f32x4_t*>(a.po + at(p) * DH + 4 * c);
    }
    const int i = row / a.ratio;
    const int64_t to = (int64_t)(s.q0 + i) * a.heads + kvh * a.ratio + row - i * a.ratio;
    const float inv = 1.0f / sum;
    *reinterpret_cast<u32x2_t*>(a.out + to * DH + 4 * c) =
        u32x2_t{bf16_pair(v[0] * inv, v[1] * inv), bf16_pair(v[2] * inv, v[3] * inv)};
    if (a.lse && c == 0) a.lse[to] = row_lse(m, sum);
  }
}

// The keys are divided where there is at most a tile for each CU, and then where a sequence may
// be so long that the time saved pays for the plan and the join: more than 1300 keys times the share
// of ROOM that the tiles leave free. The host does not know the longest; it is taken for a
// quarter of all keys at least. (32 heads of 128 over 8: 1500 tokens, 376 tiles, 34.9 us, divided
// 50.3; 1200 behind 16000, 304 tiles, 261 and 294. 256 tiles: 2048 tokens, 16 heads over 4, 40.1
// and 45.0; 4096 tokens, 8 heads, 71.3 and 64.0. 128 tiles: 4 x 100 behind 1500 27.4 and 31.1;
// 2048 tokens, 8 heads, 38.5 and 31.3. 64 tiles: 512 behind 8000, 16 heads of 64 over 2, 79.5 and
// 33.7.)
constexpr int ONE_EACH = 256, ROOM = 512, PAYS = 1300;   // (512 workgroups run at once)
struct Plan {
  int64_t tiles, groups;   // tiles and workgroups at most, both times key heads
  bool parts;
};
Plan plan_of(int64_t B, int64_t Tq, int64_t Tk, int64_t heads, int64_t kv_heads) {
  Plan p;
  const int64_t rows = Tq * (heads / kv_heads);
  // no fewer than the sequences': each of at most min(B, Tq) ends within a tile
  p.tiles = (rows + (B < Tq ? B : Tq) * (BM - 1)) / BM * kv_heads;
  const int64_t tiles = (rows + BM - 1) / BM * kv_heads;   // .. at least
  p.parts = p.tiles < ROOM && tiles <= ONE_EACH &&
            Tk / (B < 4 ? B : 4) * (ROOM - tiles) > (int64_t)PAYS * ROOM;
  p.groups = p.tiles + (p.parts ? (TARGET + kv_heads - 1) / kv_heads * kv_heads : 0);
  return p;
}

template <int DH, int SPLIT>
void launch(const Args& a, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.groups), block(NT);
  if (!p.parts) {
    if constexpr (DH == 128)
      if (p.groups >= MANY) {
        hipLaunchKernelGGL((k_attention_packed<DH, false, 32, SPLIT>), grid, block, 0, st, a);
        return;
      }
    hipLaunchKernelGGL((k_attention_packed<DH, false, 64, SPLIT>), grid, block, 0, st, a);
    return;
  }
  hipLaunchKernelGGL((k_attention_packed<DH, true, 64, SPLIT>), grid, block, 0, st, a);
  hipLaunchKernelGGL((k_attention_join<DH>), dim3((unsigned)(p.tiles * PER)), dim3(NT), 0, st, a);
}

}  // namespace

// Floats of the workspace: partial sums and (m, l) of every row of every workgroup.
int64_t ar_attention_packed_floats(int64_t B, int64_t Tq, int64_t Tk, int64_t heads,
                                   int64_t kv_heads, int64_t head_dim) {
  if (Tq == 0 || B == 0) return 0;
  const Plan p = plan_of(B, Tq, Tk, heads, kv_heads);
  return p.parts ? p.groups * BM * (head_dim + 2) : 0;
}

ar_status ar_launch_attention_packed(const ArAttentionPacked& g, hipStream_t st) {
  const Plan p = plan_of(g.B, g.Tq, g.Tk, g.heads, g.kv_heads);
  Args a;
  a.q = g.q, a.k = g.k, a.v = g.v;
  a.q_stride = g.q_stride, a.k_stride = g.k_stride, a.v_stride = g.v_stride;
  a.q_off = g.q_offsets, a.k_off = g.k_offsets;
  a.Tq = g.Tq, a.Tk = g.Tk;
  a.B = (int)g.B, a.heads = (int)g.heads, a.kv_heads = (int)g.kv_heads;
  a.ratio = (int)(g.heads / g.kv_heads);
  a.sl = (float)((double)g.scale * 1.4426950408889634);
  a.out = g.out, a.lse = g.lse;
  a.po = g.ws;
  a.groups = p.groups;
  a.pm = g.ws + p.groups * BM * g.head_dim;
  if (g.head_dim == 64) g.f32_weights ? launch<64, 3>(a, p, st) : launch<64, 1>(a, p, st);
  else g.f32_weights ? launch<128, 3>(a, p, st) : launch<128, 1>(a, p, st);
  return last_status();
}
