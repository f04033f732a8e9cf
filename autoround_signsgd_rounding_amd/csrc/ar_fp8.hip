// e4m3 operands (gfx950): the quantizers of weights and activations and the
// RMSNorm that writes its output in e4m3, all for the block-scaled product of
// ar_fp8_gemm.hip.
//
// One scale per block of values, s = amax/448 (448 is the largest e4m3 value),
// 1 for a block of zeros and never below 2^-126; a code is e4m3(x · (1/s)),
// round to nearest even. |x·(1/s)| exceeds 448 by float32 roundings only, far
// less than the half step of 16 that would round away from 448, so nothing
// has to be clamped. A NaN becomes a NaN code and leaves the scale alone; an
// infinity makes the scale infinite, and with it the block's products NaN.
// Activations: a block is 128 channels of one row, scales [KB][M] (KB =
// ceil(K/128)), so a product's tile reads the scales of its rows side by side.
// Weights: a block is 128 x 128, scales [NB][KB].
#include "ar_device.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256;
constexpr int BLK = 128;      // channels per scale
constexpr int CH = 16;        // values per lane: one 16-byte store of codes
constexpr int LPB = BLK / CH; // lanes per block row

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

__device__ __forceinline__ void load16(const uint16_t* p, float (&o)[CH]) {
  const u32x4_t a = reinterpret_cast<const u32x4_t*>(p)[0];
  const u32x4_t b = reinterpret_cast<const u32x4_t*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(a[i] << 16);
    o[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    o[8 + 2 * i] = __uint_as_float(b[i] << 16);
    o[8 + 2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load16(const float* p, float (&o)[CH]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4_t v = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[4 * i + e] = v[e];
  }
}
__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[CH]) {
  u32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    b[i] = bf16_pair(v[8 + 2 * i], v[8 + 2 * i + 1]);
  }
  reinterpret_cast<u32x4_t*>(p)[0] = a;
  reinterpret_cast<u32x4_t*>(p)[1] = b;
}
__device__ __forceinline__ void store16(float* p, const float (&v)[CH]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<f32x4_t*>(p)[i] = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}

__device__ __forceinline__ float amax16(const float (&v)[CH]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) m = fmaxf(m, fabsf(v[i]));   // fmaxf drops a NaN
  return m;
}
__device__ __forceinline__ float scale_of(float amax) {
  return amax == 0.0f ? 1.0f : fmaxf(amax / 448.0f, 0x1p-126f);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[CH], float inv) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, w, true);
    o[i] = (uint32_t)w;
  }
  *reinterpret_cast<u32x4_t*>(p) = o;
}

// SiLU(g)·u in float32: the exponential's argument is rounded once (a relative
// error of |g|·2^-24 in the result, for negative g), the reciprocal to 1 ulp.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// ------------------------------------------------------------------ activations
// Eight lanes per (row, block): a workgroup covers 32 rows of `bpw` blocks in
// turn, so the scales of one block leave as one 128-byte line.
template <class T, bool GATE>
__global__ __launch_bounds__(NT) void k_fp8_quant_act(const T* X, int64_t M, int64_t K, uint8_t* q,
                                                      float* scale, int bpw) {
  const int64_t m = (int64_t)blockIdx.x * 32 + threadIdx.x / LPB;
  const int c = threadIdx.x % LPB;
  const int64_t KB = (K + BLK - 1) / BLK;
  const int64_t j0 = (int64_t)blockIdx.y * bpw;
  const int64_t j1 = j0 + bpw < KB ? j0 + bpw : KB;
  if (m >= M) return;   // all eight lanes of a row
  const T* xr = X + m * K * (GATE ? 2 : 1);
  for (int64_t j = j0; j < j1; ++j) {
    const int64_t k = j * BLK + c * CH;
    float v[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = 0.0f;
    if (k < K) {   // K % 16 == 0: a lane's 16 values are wholly in or out
      load16(xr + k, v);
      if constexpr (GATE) {
        float u[CH];
        load16(xr + K + k, u);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[i] = silu_mul(v[i], u[i]);
      }
    }
    const float s = scale_of(group_max<LPB>(amax16(v)));
    if (k < K) store_codes(q + m * K + k, v, 1.0f / s);
    if (c == 0) scale[j * M + m] = s;
  }
}

// ------------------------------------------------------------------ weights
// One workgroup per 128 x 128 block, held in registers between the maximum and
// the codes: eight lanes per row, 32 rows at a time.
template <class T>
__global__ __launch_bounds__(NT) void k_fp8_quant_weight(const T* W, int64_t N, int64_t K,
                                                         uint8_t* q, float* scale, int NB, int KB) {
  __shared__ float red[NT / 64];
  const int64_t b = blockIdx.x;
  const int64_t e = b / ((int64_t)NB * KB);
  const int r = (int)(b - e * NB * KB), nb = r / KB, j = r - nb * KB;
  const int64_t k = (int64_t)j * BLK + (threadIdx.x % LPB) * CH;
  float v[4][CH];
  float m = 0.0f;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t n = (int64_t)nb * BLK + p * 32 + threadIdx.x / LPB;
#pragma unroll
    for (int i = 0; i < CH; ++i) v[p][i] = 0.0f;
    if (n < N && k < K) load16(W + (e * N + n) * K + k, v[p]);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) m = fmaxf(m, amax16(v[p]));
  m = group_max<64>(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = scale_of(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  const float inv = 1.0f / s;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t n = (int64_t)nb * BLK + p * 32 + threadIdx.x / LPB;
    if (n < N && k < K) store_codes(q + (e * N + n) * K + k, v[p], inv);
  }
  if (threadIdx.x == 0) scale[b] = s;
}

// ------------------------------------------------------------------ RMSNorm
// One workgroup per row: v = x + residual rounded to T (the stored sum is what
// is normalised, as the block's separate addition has it), the sum of squares
// in float64 (the block's norm does the same, and no square of a finite input
// overflows), y = (v·r)·w in float32, codes from the unrounded y. The row stays
// in registers (C chunks of 16 values per thread); C = 0 reads it twice.
// Every thread reads an element before it writes any output at that place, so
// h may be x or the residual itself.
template <class T>
__device__ __forceinline__ void norm_input(const T* x, const T* res, int64_t o, float (&v)[CH]) {
  load16(x + o, v);
  if (res) {
    float u[CH];
    load16(res + o, u);
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

template <class T, int THREADS, int C>
__global__ __launch_bounds__(THREADS) void k_rmsnorm_fp8(NormArgs a) {
  __shared__ double red[THREADS / 64];
  // consecutive rows on one XCD, whose L2 then joins their scales (4 bytes a
  // row) into whole lines
  const int64_t per = gridDim.x >> 3, rem = gridDim.x & 7;
  const int64_t xcd = blockIdx.x & 7;
  const int64_t m = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const T *x = static_cast<const T*>(a.x) + m * a.D;
  const T *res = a.res ? static_cast<const T*>(a.res) + m * a.D : nullptr;
  const T* w = static_cast<const T*>(a.w);
  const int t = threadIdx.x;
  constexpr int NC = C > 0 ? C : 1;
  float v[NC][CH];
  double ss = 0.0;
  auto add = [&](const float (&u)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) ss = fma((double)u[i], (double)u[i], ss);
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k = ((int64_t)c * THREADS + t) * CH;
      if (k < a.D) {
        norm_input(x, res, k, v[c]);
        add(v[c]);
      }
    }
  } else {
    for (int64_t k = (int64_t)t * CH; k < a.D; k += THREADS * CH) {
      norm_input(x, res, k, v[0]);
      add(v[0]);
    }
  }
  ss = group_sum_f64<64>(ss);
  if constexpr (THREADS > 64) {
    if ((t & 63) == 0) red[t >> 6] = ss;
    __syncthreads();
    ss = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) ss += red[i];
  }
  const float r = (float)(1.0 / sqrt(ss / (double)a.D + (double)a.eps));
  const int64_t KB = (a.D + BLK - 1) / BLK;
  auto finish = [&](int64_t k, float (&u)[CH]) {
    const bool in = k < a.D;
    float y[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) y[i] = 0.0f;
    if (in) {
      if (a.h) store16(static_cast<T*>(a.h) + m * a.D + k, u);
      float g[CH];
      load16(w + k, g);
#pragma unroll
      for (int i = 0; i < CH; ++i) y[i] = (u[i] * r) * g[i];
      if (a.y) store16(static_cast<T*>(a.y) + m * a.D + k, y);
    }
    const float s = scale_of(group_max<LPB>(amax16(y)));
    if (in) store_codes(a.q + m * a.D + k, y, 1.0f / s);
    if (k / BLK < KB && k % BLK == 0) a.scale[(k / BLK) * a.M + m] = s;
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) finish(((int64_t)c * THREADS + t) * CH, v[c]);
  } else {
    // whole rounds, so that the eight lanes of a block stay together
    for (int64_t k = (int64_t)t * CH; k - t * CH < a.D; k += THREADS * CH) {
      if (k < a.D) norm_input(x, res, k, v[0]);
      finish(k, v[0]);
    }
  }
}

template <class T>
ar_status norm_launch(const NormArgs& a, hipStream_t st) {
  const dim3 g((unsigned)a.M);
  if (a.D <= 64 * CH)
    hipLaunchKernelGGL((k_rmsnorm_fp8<T, 64, 1>), g, dim3(64), 0, st, a);
  else if (a.D <= 256 * CH)
    hipLaunchKernelGGL((k_rmsnorm_fp8<T, 256, 1>), g, dim3(256), 0, st, a);
  else if (a.D <= 512 * CH)
    hipLaunchKernelGGL((k_rmsnorm_fp8<T, 256, 2>), g, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_rmsnorm_fp8<T, 256, 0>), g, dim3(256), 0, st, a);
  return last_status();
}

template <class T, bool GATE>
void act_launch(const void* X, int64_t M, int64_t K, uint8_t* q, float* scale, hipStream_t st) {
  const int64_t KB = (K + BLK - 1) / BLK, rows = (M + 31) / 32;
  // four blocks per workgroup where that still leaves enough of them for 256 CUs
  const int bpw = rows * KB >= 4 * 2048 ? 4 : 1;
  hipLaunchKernelGGL((k_fp8_quant_act<T, GATE>), dim3((unsigned)rows, (unsigned)((KB + bpw - 1) / bpw)),
                     dim3(NT), 0, st, static_cast<const T*>(X), M, K, q, scale, bpw);
}

}  // namespace

ar_status ar_launch_fp8_quant_act(int xdt, const void* X, int gate, int64_t M, int64_t K,
                                  uint8_t* q, float* scale, hipStream_t st) {
  if (xdt == AR_BF16) {
    if (gate) act_launch<uint16_t, true>(X, M, K, q, scale, st);
    else act_launch<uint16_t, false>(X, M, K, q, scale, st);
  } else {
    if (gate) act_launch<float, true>(X, M, K, q, scale, st);
    else act_launch<float, false>(X, M, K, q, scale, st);
  }
  return last_status();
}

ar_status ar_launch_fp8_quant_weight(int wdt, const void* W, int64_t E, int64_t N, int64_t K,
                                     uint8_t* q, float* scale, hipStream_t st) {
  const int64_t NB = (N + BLK - 1) / BLK, KB = (K + BLK - 1) / BLK;
  const dim3 g((unsigned)(E * NB * KB));
  if (wdt == AR_BF16)
    hipLaunchKernelGGL((k_fp8_quant_weight<uint16_t>), g, dim3(NT), 0, st,
                       static_cast<const uint16_t*>(W), N, K, q, scale, (int)NB, (int)KB);
  else
    hipLaunchKernelGGL((k_fp8_quant_weight<float>), g, dim3(NT), 0, st,
                       static_cast<const float*>(W), N, K, q, scale, (int)NB, (int)KB);
  return last_status();
}

ar_status ar_launch_rmsnorm_fp8(int dt, const void* x, const void* res, const void* w, int64_t M,
                                int64_t D, float eps, void* h, void* y, uint8_t* q, float* scale,
                                hipStream_t st) {
  const NormArgs a{x, res, w, h, y, q, scale, M, D, eps};
  return dt == AR_BF16 ? norm_launch<uint16_t>(a, st) : norm_launch<float>(a, st);
}
