// e4m3 operands (gfx950): the quantizers of weights and activations and the
// RMSNorm that writes its output in e4m3, all for the block-scaled product of
// ar_fp8_gemm.hip.
//
// One scale per block of values, s = amax/448 (448 is the largest e4m3 value),
// 1 for a block of zeros and never below 2^-126; a code is e4m3(x/s), the quotient
// rounded to float32 first, round to nearest even. |x/s| exceeds 448 by float32 roundings
// only, far less than the half step of 16 that would round away from 448, so
// nothing has to be clamped. A NaN becomes a NaN code and leaves the scale alone; an
// infinity makes the scale infinite, and with it the block's products NaN.
// Activations: a block is 128 channels of one row, scales [KB][M] (KB =
// ceil(K/128)), so a product's tile reads the scales of its rows side by side.
// Weights: a block is 128 x 128, scales [NB][KB].
#include <type_traits>

#include "ar_device.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256;
constexpr int BLK = 128;      // channels per scale
constexpr int CH = 8;         // values per lane: a wave reads 1 KiB of bf16 in one piece
constexpr int LPB = BLK / CH; // lanes per block row

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

// Largest magnitude of a block: 8 values of a lane, then the 16 lanes of a DPP
// row, rotated by 8, 4, 2 and 1. fmaxf drops a NaN.
__device__ __forceinline__ float amax_row(const float (&v)[CH]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; i += 2) m = fmaxf(fmaxf(m, fabsf(v[i])), fabsf(v[i + 1]));
  auto turn = [&](auto by) {
    const int o = __builtin_amdgcn_mov_dpp(__float_as_int(m), 0x120 + decltype(by)::value, 0xF, 0xF,
                                           true);
    m = fmaxf(m, __int_as_float(o));
  };
  turn(std::integral_constant<int, 8>());
  turn(std::integral_constant<int, 4>());
  turn(std::integral_constant<int, 2>());
  turn(std::integral_constant<int, 1>());
  return m;
}
// amax/448, rounded once: the quotient by the reciprocal, corrected by the
// remainder (an infinite amax has none).
__device__ __forceinline__ float scale_of(float amax) {
  constexpr float R = 1.0f / 448.0f;
  const float q0 = amax * R;
  const float q = fmaf(fmaf(-q0, 448.0f, amax), R, q0);
  const float s = amax < __builtin_inff() ? fmaxf(q, 0x1p-126f) : amax;
  return amax == 0.0f ? 1.0f : s;
}
// 1/s in two floats, the first never above it: x·hi + x·lo is x/s to 2^-46 before it is
// rounded, where x·hi alone is off by up to 1.5 units in the last place and sends a
// quotient halfway between two codes to the wrong one. With lo >= 0 a zero keeps
// its sign. Of an infinite scale finite values become 0, an infinity NaN.
struct Inverse {
  float hi, lo;
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  float hi = __builtin_amdgcn_rcpf(s);   // 1 ulp; s is a normal number or infinite
  if (fmaf(-s, hi, 1.0f) < 0.0f) hi = __int_as_float(__float_as_int(hi) - 1);
  return {hi, s < __builtin_inff() ? hi * fmaf(-s, hi, 1.0f) : 0.0f};
}
__device__ __forceinline__ float divide(float x, const Inverse& d) { return fmaf(x, d.hi, x * d.lo); }

// Outputs are stored past the caches, whole 512-byte or 1-KiB pieces a wave:
// measured on a 16384 x 8192 norm 186 us instead of 197, on a 29568 x 8192 weight
// 124 instead of 134; a 1 x 4096 norm takes as long either way.
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[CH], float s) {
  const Inverse d = inverse_of(s);
  u32x2_t o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(divide(v[4 * i], d), divide(v[4 * i + 1], d), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(divide(v[4 * i + 2], d), divide(v[4 * i + 3], d), w, true);
    o[i] = (uint32_t)w;
  }
  __builtin_nontemporal_store(o, reinterpret_cast<u32x2_t*>(p));
}
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[CH]) {
  __builtin_nontemporal_store(u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                      bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                              reinterpret_cast<u32x4_t*>(p));
}
__device__ __forceinline__ void store_row(float* p, const float (&v)[CH]) {
  f32x4_t* d = reinterpret_cast<f32x4_t*>(p);
  __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, d);
  __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, d + 1);
}

// SiLU(g)·u in float32, to 8·2^-24: exp(-g) = 2^hi·(1 + lo·ln 2), hi the rounded product
// of g and log2 e and lo the rest of it, without which the result would be off by
// |g|·2^-24. As it stands that is good for |g| <= 64, which a wave's gates
// hardly ever leave together; with FAR, for every gate: where 2^hi would leave float32's
// range (and the sigmoid, of which a large u may still make a normal number), it is taken
// 2^160 lower, and u as mantissa and exponent. 2048 x 11008 bf16 takes 20.9 us.
template <bool FAR>
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float L = -1.44269502f, LREST = -1.92596299e-8f;   // their sum is -log2 e
  constexpr float LN2 = 0.69314718f;
  const float x = FAR ? __builtin_amdgcn_fmed3f(g, -300.0f, 300.0f) : g;
  const float hi = x * L, lo = fmaf(x, LREST, fmaf(x, L, -hi)) * LN2;
  if constexpr (!FAR) {
    const float p = __builtin_amdgcn_exp2f(hi);
    return g * __builtin_amdgcn_rcpf(fmaf(p, lo, p) + 1.0f) * u;
  } else {
    const bool low = hi > 96.0f;   // (hi - 160 is exact up to 320; from 288 on the result is 0)
    const float p = __builtin_amdgcn_exp2f(low ? hi - 160.0f : hi);
    const float e = p < __builtin_inff() ? fmaf(p, lo, p) : p;
    const float r = __builtin_amdgcn_rcpf(low ? e : e + 1.0f);
    return ldexpf(g * r * __builtin_amdgcn_frexp_mantf(u),
                  __builtin_amdgcn_frexp_expf(u) - (low ? 160 : 0));
  }
}
__device__ __forceinline__ void silu_mul(float (&g)[CH], const float (&u)[CH]) {
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < CH; e += 2) far = fmaxf(fmaxf(far, fabsf(g[e])), fabsf(g[e + 1]));
  if (__any(far > 64.0f)) {
#pragma unroll
    for (int e = 0; e < CH; ++e) g[e] = silu_mul<true>(g[e], u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e) g[e] = silu_mul<false>(g[e], u[e]);
  }
}

// Eight values of T as they lie in memory.
template <class T>
struct RowOf {
  u32x4_t raw[sizeof(T) / 2] = {};
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = reinterpret_cast<const u32x4_t*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&o)[CH]) const {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if constexpr (sizeof(T) == 4)
        o[i] = __uint_as_float(raw[i / 4][i % 4]);
      else
        o[i] = __uint_as_float(i % 2 ? raw[0][i / 2] & 0xFFFF0000u : raw[0][i / 2] << 16);
    }
  }
};

// ------------------------------------------------------------------ activations
// Units of one block of one row, 16 lanes each. A workgroup takes RT rows by BT
// blocks of them, row by row, a wave four units (1 KiB of bf16) at a time and
// ITERS times; the scales leave through LDS, the RT rows of a block side by
// side. Values wait as they were loaded: 62 registers at bf16, gated, where as floats
// they take 86 and five waves fit a SIMD instead of eight (2048 x 11008: 20.9 us instead
// of 23.7). ITERS = 1 spreads small inputs over more CUs: 16 x 11008, gated, takes 2.9 us
// instead of 6.5 at 32 rows a workgroup.
template <class T, bool GATE, int ITERS>
__global__ __launch_bounds__(NT) void k_fp8_quant_act(const T* X, int64_t M, int64_t K, uint8_t* q,
                                                      float* scale, int RT, int BT,
                                                      int chunks) {
  __shared__ float sc[ITERS * NT / LPB];
  const int64_t KB = (K + BLK - 1) / BLK;
  const int mt = blockIdx.x / chunks;   // consecutive workgroups share rows
  const int64_t j0 = (int64_t)(blockIdx.x - mt * chunks) * BT, m0 = (int64_t)mt * RT;
  const int c = threadIdx.x % LPB * CH;
  RowOf<T> v[ITERS], u[ITERS];
  int64_t at[ITERS];   // offset of the lane's values in q, -1: none
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int unit = i * (NT / LPB) + threadIdx.x / LPB, r = unit / BT;
    const int64_t m = m0 + r, k = (j0 + unit - r * BT) * BLK + c;
    at[i] = -1;
    if (r < RT && m < M && k < K) {   // K % 16 == 0: the 8 values are in or out
      at[i] = m * K + k;
      v[i].load(X + m * K * (GATE ? 2 : 1) + k);
      if constexpr (GATE) u[i].load(X + (2 * m + 1) * K + k);
    }
  }
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    float x[CH];
    v[i].get(x);
    if constexpr (GATE) {
      float up[CH];
      u[i].get(up);
      silu_mul(x, up);
    }
    const float s = scale_of(amax_row(x));
    if (at[i] >= 0) store_codes(q + at[i], x, s);
    if (threadIdx.x % LPB == 0) sc[i * (NT / LPB) + threadIdx.x / LPB] = s;
  }
  __syncthreads();
  const int b = threadIdx.x / RT, r = threadIdx.x - b * RT;
  if (b < BT && j0 + b < KB && m0 + r < M) scale[(j0 + b) * M + m0 + r] = sc[r * BT + b];
}

// ------------------------------------------------------------------ weights
// One workgroup per 128 x 128 block, held in registers between the maximum and
// the codes: sixteen lanes per row, 16 rows at a time.
template <class T>
__global__ __launch_bounds__(NT) void k_fp8_quant_weight(const T* W, int64_t N, int64_t K,
                                                         uint8_t* q, float* scale, int NB, int KB) {
  constexpr int PASS = NT / LPB, P = BLK / PASS;   // rows at a time, times
  __shared__ float red[NT / 64];
  const int64_t b = blockIdx.x;
  const int64_t e = b / ((int64_t)NB * KB);
  const int r = (int)(b - e * NB * KB), nb = r / KB, j = r - nb * KB;
  const int64_t k = (int64_t)j * BLK + (threadIdx.x % LPB) * CH;
  const int64_t n0 = (int64_t)nb * BLK + threadIdx.x / LPB;
  float v[P][CH];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int i = 0; i < CH; ++i) v[p][i] = 0.0f;
    if (n0 + p * PASS < N && k < K) load8(W + (e * N + n0 + p * PASS) * K + k, v[p]);
  }
  float m = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) m = fmaxf(m, amax_row(v[p]));
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = scale_of(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (n0 + p * PASS < N && k < K) store_codes(q + (e * N + n0 + p * PASS) * K + k, v[p], s);
  if (threadIdx.x == 0) scale[b] = s;
}

// ------------------------------------------------------------------ RMSNorm
// v = x + residual rounded to T (the stored sum is what is normalised, as the
// block's separate addition has it), the sum of squares in float64 (the block's
// norm does the same, and no square of a finite input overflows), y = (v/rms)·w in
// float32, codes from the unrounded y. A row of up to 2048 is a wave's or a part
// of a wave's, a longer one a workgroup's. It stays in registers, C chunks of 8
// values per lane; C = 0 reads it twice. Every lane reads an element before it
// writes any output at that place, so h may be x or the residual itself.
template <class T>
__device__ __forceinline__ void norm_input(const T* x, const T* res, int64_t o, float (&v)[CH]) {
  load8(x + o, v);
  if (res) {
    float u[CH];
    load8(res + o, u);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      v[i] += u[i];
      if constexpr (sizeof(T) == 2) v[i] = bf16_val(bf16_bits(v[i]));
    }
  }
}

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y;
  uint8_t* q;
  float* scale;
  int64_t M, D;
  float eps;
};

template <class T, int LANES, int C>   // LANES per row: 16, 32, 64 or NT
__global__ __launch_bounds__(NT) void k_rmsnorm_fp8(NormArgs a) {
  __shared__ double red[NT / 64];
  constexpr int ROWS = NT / LANES;
  // consecutive rows on one XCD, whose L2 then joins their scales (4 bytes a
  // row) into whole lines
  const int64_t per = gridDim.x >> 3, rem = gridDim.x & 7;
  const int64_t xcd = blockIdx.x & 7;
  const int64_t g = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const int64_t m = g * ROWS + threadIdx.x / LANES;
  if (m >= a.M) return;   // whole rows (ROWS > 1 has no barrier below)
  const T *x = static_cast<const T*>(a.x) + m * a.D;
  const T *res = a.res ? static_cast<const T*>(a.res) + m * a.D : nullptr;
  const T* w = static_cast<const T*>(a.w);
  const int t = threadIdx.x % LANES;
  float v[C > 0 ? C : 1][CH];
  RowOf<T> wr[C > 0 ? C : 1];   // w, requested with x so that it is there after the sum
  double ss = 0.0;
  auto add = [&](const float (&u)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) ss = fma((double)u[i], (double)u[i], ss);
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k = ((int64_t)c * LANES + t) * CH;
      if (k < a.D) {
        wr[c].load(w + k);
        norm_input(x, res, k, v[c]);
        add(v[c]);
      }
    }
  } else {
    for (int64_t k = (int64_t)t * CH; k < a.D; k += LANES * CH) {
      norm_input(x, res, k, v[0]);
      add(v[0]);
    }
  }
  ss = group_sum_f64<LANES < 64 ? LANES : 64>(ss);
  if constexpr (LANES > 64) {
    if ((t & 63) == 0) red[t >> 6] = ss;
    __syncthreads();
    ss = ((red[0] + red[1]) + red[2]) + red[3];
  }
  // 1/rms as mantissa and exponent: without an eps it may lie outside float32's normal
  // range while the normalised values, at most sqrt(D), do not
  const double inv = 1.0 / sqrt(ss / (double)a.D + (double)a.eps);
  const float r = (float)__builtin_amdgcn_frexp_mant(inv);
  const int rexp = __builtin_amdgcn_frexp_exp(inv);
  auto finish = [&](int64_t k, const float (&u)[CH], const RowOf<T>& wv) {
    const bool in = k < a.D;
    float y[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) y[i] = 0.0f;
    if (in) {
      if (a.h) store_row(static_cast<T*>(a.h) + m * a.D + k, u);
      wv.get(y);
#pragma unroll
      for (int i = 0; i < CH; ++i) y[i] = (ldexpf(u[i], rexp) * r) * y[i];
      if (a.y) store_row(static_cast<T*>(a.y) + m * a.D + k, y);
    }
    const float s = scale_of(amax_row(y));
    if (in) store_codes(a.q + m * a.D + k, y, s);
    if (in && t % LPB == 0) a.scale[(k / BLK) * a.M + m] = s;
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) finish(((int64_t)c * LANES + t) * CH, v[c], wr[c]);
  } else {
    // whole rounds, so that the lanes of a block stay together
    for (int64_t k = (int64_t)t * CH; k - t * CH < a.D; k += LANES * CH) {
      if (k < a.D) {
        wr[0].load(w + k);
        norm_input(x, res, k, v[0]);
      }
      finish(k, v[0], wr[0]);
    }
  }
}

template <class T, int LANES, int C>
void norm_go(const NormArgs& a, hipStream_t st) {
  constexpr int ROWS = NT / LANES;
  hipLaunchKernelGGL((k_rmsnorm_fp8<T, LANES, C>), dim3((unsigned)((a.M + ROWS - 1) / ROWS)),
                     dim3(NT), 0, st, a);
}
template <class T>
ar_status norm_launch(const NormArgs& a, hipStream_t st) {
  const int64_t D = a.D;
  if (D <= 128) norm_go<T, 16, 1>(a, st);
  else if (D <= 256) norm_go<T, 32, 1>(a, st);
  else if (D <= 512) norm_go<T, 64, 1>(a, st);
  else if (D <= 1024) norm_go<T, 64, 2>(a, st);
  else if (D <= 2048) norm_go<T, 64, 4>(a, st);
  else if (D <= 4096) norm_go<T, NT, 2>(a, st);
  else if (D <= 8192) norm_go<T, NT, 4>(a, st);
  else if (D <= 16384) norm_go<T, NT, 8>(a, st);
  else norm_go<T, NT, 0>(a, st);
  return last_status();
}

template <class T, bool GATE, int ITERS>
ar_status act_go(const void* X, int64_t M, int64_t K, uint8_t* q, float* scale, hipStream_t st) {
  constexpr int UNITS = ITERS * NT / LPB;
  const int64_t KB = (K + BLK - 1) / BLK;
  int RT = 1;
  while (RT < 16 && RT < M) RT *= 2;
  const int BT = (int)(KB < UNITS / RT ? KB : UNITS / RT);
  RT = UNITS / BT;
  const int64_t chunks = (KB + BT - 1) / BT, n = chunks * ((M + RT - 1) / RT);
  if (n >= int64_t(1) << 24) return AR_ERR_SHAPE;
  hipLaunchKernelGGL((k_fp8_quant_act<T, GATE, ITERS>), dim3((unsigned)n), dim3(NT), 0, st,
                     static_cast<const T*>(X), M, K, q, scale, RT, BT, (int)chunks);
  return last_status();
}
template <class T, bool GATE>
ar_status act_launch(const void* X, int64_t M, int64_t K, uint8_t* q, float* scale, hipStream_t st) {
  return M * K <= 1024 * 16 * BLK ? act_go<T, GATE, 1>(X, M, K, q, scale, st)
                                  : act_go<T, GATE, 4>(X, M, K, q, scale, st);
}
template <class T>
void weight_launch(const void* W, int64_t E, int64_t N, int64_t K, uint8_t* q, float* scale,
                   hipStream_t st) {
  const int64_t NB = (N + BLK - 1) / BLK, KB = (K + BLK - 1) / BLK;
  hipLaunchKernelGGL((k_fp8_quant_weight<T>), dim3((unsigned)(E * NB * KB)), dim3(NT), 0, st,
                     static_cast<const T*>(W), N, K, q, scale, (int)NB, (int)KB);
}

}  // namespace

ar_status ar_launch_fp8_quant_act(int xdt, const void* X, int gate, int64_t M, int64_t K,
                                  uint8_t* q, float* scale, hipStream_t st) {
  if (xdt == AR_BF16)
    return gate ? act_launch<uint16_t, true>(X, M, K, q, scale, st)
                : act_launch<uint16_t, false>(X, M, K, q, scale, st);
  return gate ? act_launch<float, true>(X, M, K, q, scale, st)
              : act_launch<float, false>(X, M, K, q, scale, st);
}

ar_status ar_launch_fp8_quant_weight(int wdt, const void* W, int64_t E, int64_t N, int64_t K,
                                     uint8_t* q, float* scale, hipStream_t st) {
  if (wdt == AR_BF16) weight_launch<uint16_t>(W, E, N, K, q, scale, st);
  else weight_launch<float>(W, E, N, K, q, scale, st);
  return last_status();
}

ar_status ar_launch_rmsnorm_fp8(int dt, const void* x, const void* res, const void* w, int64_t M,
                                int64_t D, float eps, void* h, void* y, uint8_t* q, float* scale,
                                hipStream_t st) {
  const NormArgs a{x, res, w, h, y, q, scale, M, D, eps};
  return dt == AR_BF16 ? norm_launch<uint16_t>(a, st) : norm_launch<float>(a, st);
}
