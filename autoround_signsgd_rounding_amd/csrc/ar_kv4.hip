// The 4-bit key/value cache (gfx950): tokens are quantized as they are written, and
// read back. Layout: ar_kv4.h.
//
// A group of g channels of a token's head (g = 32, 64 or 128) has the asymmetric integer
// grid of the weights' quantizer at alpha = beta = 1, in float32, each step rounded once:
//   lo = min(x, 0), hi = max(x, 0);   s = max((hi - lo)/15, 2^-100)
//   zp = clamp(rint(-lo/s), 0, 15);   s' = s with its four lowest bits replaced by zp
//   code = clamp(rint(x/s') + zp, 0, 15);   value s'·(code - zp)
// s' is off s by 15·2^-23 of it at most: 15 steps from zero that is 1/18600 of the half step that
// a code is rounded by. The codes are those of s': one word a group holds all there is to know.
// A NaN or an infinity in a group (or a range beyond float32) makes s' NaN and with it
// the group's values; its codes are 0.
//
// Memory bounds both: 16384 tokens of 8 heads x 128 in bf16 (67 MB, and 18 MB of cache) are
// written in 20.2 us and read back in 21.3, 4.2 and 4.0 TB/s, a launch's 2 us included (a
// large copy moves 4.89). A third fewer instructions a code, or two or four tokens a lane, changed
// nothing. The 32 tokens of a step take 2.7 and 3.0 us: a launch, a slot, what it points to.
#include "ar_kv4.h"
#include "ar_launch.h"

namespace {

constexpr int NT = 256;

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct Grid4 {
  float s, inv, zp;   // s', 1/s' rounded, the zero-point
};
__device__ __forceinline__ Grid4 grid_of(float lo, float hi) {
  const float d = hi - lo;
  const float s = fmaxf(d / 15.0f, 0x1p-100f);
  const float zp = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
  Grid4 g;
  g.zp = zp;
  g.s = __uint_as_float((__float_as_uint(s) & ~15u) | (uint32_t)zp);
  if (!(d < __builtin_inff())) {   // an infinity or a NaN (the maxima keep it)
    g.zp = 0.0f;
    g.s = __uint_as_float(0x7FC00000u);
  }
  g.inv = 1.0f / g.s;
  return g;
}
// The code of x: the quotient by the rounded reciprocal, off by one unit in the last
// place at most, corrected by its exact remainder to the rounded quotient.
__device__ __forceinline__ uint32_t code_of(float x, const Grid4& g) {
  const float q0 = x * g.inv;
  const float q = fmaf(fmaf(-q0, g.s, x), g.inv, q0);
  // (fmaxf makes a NaN's code 0)
  return (uint32_t)fminf(fmaxf(rintf(q) + g.zp, 0.0f), 15.0f);
}
// IEEE minimum and maximum keep a NaN, which marks the group.
__device__ __forceinline__ float low(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float high(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <int LANES>
__device__ __forceinline__ void group_range(float& lo, float& hi) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = low(lo, __shfl_xor(lo, o, 64));
    hi = high(hi, __shfl_xor(hi, o, 64));
  }
}

struct WriteArgs {
  const void *k, *v;
  int64_t k_stride, v_stride, T;
  const int32_t* slots;
  ArKv4 c;
};

// Page and token of a slot; false for a slot outside the cache.
__device__ __forceinline__ bool place_of(const ArKv4& c, int32_t slot, int64_t& page, int& t) {
  page = slot >> c.shift;
  t = slot & (c.page - 1);
  return slot >= 0 && page < c.pages;
}

template <class T>
__device__ __forceinline__ void load2(const T* p, float& a, float& b) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 w = *reinterpret_cast<const float2*>(p);
    a = w.x;
    b = w.y;
  }
}

// Keys (blockIdx.y = 0): a lane takes 8 neighbouring channels, Dh/8 lanes a token. Values
// (1): lane n takes channels 32·β + 2n, + 1, whose codes are one byte each, 16 lanes a
// token. A workgroup's tokens are neighbours and of one head.
template <class T, int DH, int GS>
__global__ __launch_bounds__(NT) void k_kv4_write(WriteArgs a) {
  constexpr int G = DH / GS;
  const int h = blockIdx.z;
  const int64_t rows = (int64_t)2 * a.c.heads * a.c.page;
  if (blockIdx.y == 0) {
    constexpr int LPT = DH / 8, TPB = NT / LPT;   // lanes a token, tokens a workgroup
    const int64_t tok = (int64_t)blockIdx.x * TPB + threadIdx.x / LPT;
    const int c = threadIdx.x % LPT;
    if (tok >= a.T) return;                        // (whole groups of lanes)
    int64_t page;
    int t;
    const bool live = place_of(a.c, a.slots[tok], page, t);
    float x[8];
    load8(static_cast<const T*>(a.k) + tok * a.k_stride + h * DH + 8 * c, x);
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = low(lo, x[i]);
      hi = high(hi, x[i]);
    }
    group_range<GS / 8>(lo, hi);
    const Grid4 g = grid_of(lo, hi);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= code_of(x[i], g) << (4 * i);
    if (!live) return;
    const int64_t row = page * rows + (int64_t)h * a.c.page + t;
    *reinterpret_cast<uint32_t*>(a.c.codes + row * (DH / 2) + 4 * c) = w;
    if (c % (GS / 8) == 0) a.c.scale[row * G + c / (GS / 8)] = g.s;
  } else {
    constexpr int TPB = NT / 16, NB = DH / 32;     // bytes a lane
    const int64_t tok = (int64_t)blockIdx.x * TPB + threadIdx.x / 16;
    const int n = threadIdx.x % 16;
    if (tok >= a.T) return;
    int64_t page;
    int t;
    const bool live = place_of(a.c, a.slots[tok], page, t);
    const T* p = static_cast<const T*>(a.v) + tok * a.v_stride + h * DH + 2 * n;
    float x[2 * NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) load2(p + 32 * b, x[2 * b], x[2 * b + 1]);
    uint32_t byte[NB];
    float s[G];
#pragma unroll
    for (int q = 0; q < G; ++q) {
      constexpr int E = 2 * NB / G;                // values of a lane in a group
      float lo = 0.0f, hi = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        lo = low(lo, x[q * E + i]);
        hi = high(hi, x[q * E + i]);
      }
      group_range<16>(lo, hi);
      const Grid4 g = grid_of(lo, hi);
      s[q] = g.s;
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        byte[q * E / 2 + i] =
            code_of(x[q * E + 2 * i], g) | (code_of(x[q * E + 2 * i + 1], g) << 4);
    }
    if (!live) return;
    const int64_t first = page * rows + (int64_t)(a.c.heads + h) * a.c.page;
    uint8_t* out = a.c.codes + first * (DH / 2);
#pragma unroll
    for (int b = 0; b < NB / 2; ++b)
      *reinterpret_cast<uint16_t*>(out + kv4_value_at(t, b, n, 0, NB / 2)) =
          (uint16_t)(byte[2 * b] | (byte[2 * b + 1] << 8));
#pragma unroll
    for (int q = 0; q < G; ++q)
      if (n == q) a.c.scale[(first + t) * G + q] = s[q];
  }
}

struct ReadArgs {
  const int32_t* slots;
  void *k, *v;
  int64_t T;
  ArKv4 c;
};

__device__ __forceinline__ void store2(uint16_t* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = bf16_pair(a, b);
}
__device__ __forceinline__ void store2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = float2{a, b};
}

// The same division of work; slots outside the cache give zeros.
template <class T, int DH, int GS>
__global__ __launch_bounds__(NT) void k_kv4_read(ReadArgs a) {
  constexpr int G = DH / GS;
  const int h = blockIdx.z;
  const int64_t rows = (int64_t)2 * a.c.heads * a.c.page;
  if (blockIdx.y == 0) {
    constexpr int LPT = DH / 8, TPB = NT / LPT;
    const int64_t tok = (int64_t)blockIdx.x * TPB + threadIdx.x / LPT;
    const int c = threadIdx.x % LPT;
    if (tok >= a.T) return;
    int64_t page;
    int t;
    uint32_t w = 0;
    float s = 0.0f;
    if (place_of(a.c, a.slots[tok], page, t)) {
      const int64_t row = page * rows + (int64_t)h * a.c.page + t;
      w = *reinterpret_cast<const uint32_t*>(a.c.codes + row * (DH / 2) + 4 * c);
      s = a.c.scale[row * G + c / (GS / 8)];
    }
    const float zp = (float)kv4_zero(s);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s * ((float)((w >> (4 * i)) & 15u) - zp);
    store8(static_cast<T*>(a.k) + (tok * a.c.heads + h) * DH + 8 * c, x);
  } else {
    constexpr int TPB = NT / 16, NB = DH / 32;
    const int64_t tok = (int64_t)blockIdx.x * TPB + threadIdx.x / 16;
    const int n = threadIdx.x % 16;
    if (tok >= a.T) return;
    int64_t page;
    int t;
    T* p = static_cast<T*>(a.v) + (tok * a.c.heads + h) * DH + 2 * n;
    const bool live = place_of(a.c, a.slots[tok], page, t);
    const int64_t first = live ? page * rows + (int64_t)(a.c.heads + h) * a.c.page : 0;
#pragma unroll
    for (int b = 0; b < NB / 2; ++b) {
      uint32_t w = 0;
      if (live)
        w = *reinterpret_cast<const uint16_t*>(a.c.codes + first * (DH / 2) +
                                               kv4_value_at(t, b, n, 0, NB / 2));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s = live ? a.c.scale[(first + t) * G + (2 * b + i) * 32 / GS] : 0.0f;
        const float zp = (float)kv4_zero(s);
        store2(p + 32 * (2 * b + i), s * ((float)((w >> (8 * i)) & 15u) - zp),
               s * ((float)((w >> (8 * i + 4)) & 15u) - zp));
      }
    }
  }
}

template <class A, class F>
ar_status go(const A& a, int DH, F launch) {
  const int tpb = NT / 16;   // the values' tokens a workgroup; the keys' are as many or twice
  const dim3 grid((unsigned)((a.T + tpb - 1) / tpb), 2, (unsigned)a.c.heads);
  launch(grid);
  return last_status();
}

template <class T>
ar_status write_as(const WriteArgs& a, int DH, int GS, hipStream_t st) {
  return go(a, DH, [&](dim3 grid) {
    if (DH == 64 && GS == 32) hipLaunchKernelGGL((k_kv4_write<T, 64, 32>), grid, dim3(NT), 0, st, a);
    else if (DH == 64) hipLaunchKernelGGL((k_kv4_write<T, 64, 64>), grid, dim3(NT), 0, st, a);
    else if (GS == 32) hipLaunchKernelGGL((k_kv4_write<T, 128, 32>), grid, dim3(NT), 0, st, a);
    else if (GS == 64) hipLaunchKernelGGL((k_kv4_write<T, 128, 64>), grid, dim3(NT), 0, st, a);
    else hipLaunchKernelGGL((k_kv4_write<T, 128, 128>), grid, dim3(NT), 0, st, a);
  });
}
template <class T>
ar_status read_as(const ReadArgs& a, int DH, int GS, hipStream_t st) {
  return go(a, DH, [&](dim3 grid) {
    if (DH == 64 && GS == 32) hipLaunchKernelGGL((k_kv4_read<T, 64, 32>), grid, dim3(NT), 0, st, a);
    else if (DH == 64) hipLaunchKernelGGL((k_kv4_read<T, 64, 64>), grid, dim3(NT), 0, st, a);
    else if (GS == 32) hipLaunchKernelGGL((k_kv4_read<T, 128, 32>), grid, dim3(NT), 0, st, a);
    else if (GS == 64) hipLaunchKernelGGL((k_kv4_read<T, 128, 64>), grid, dim3(NT), 0, st, a);
    else hipLaunchKernelGGL((k_kv4_read<T, 128, 128>), grid, dim3(NT), 0, st, a);
  });
}

ArKv4 cache_of(const ar_kv4_cache& c) {
  return ArKv4{c.codes, c.scale, c.pages, (int)c.heads, c.page_size, __builtin_ctz(c.page_size)};
}

}  // namespace

ar_status ar_launch_kv4_write(const ar_kv4_cache& c, int dt, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, const int32_t* slots, int64_t T,
                              hipStream_t st) {
  const WriteArgs a{k, v, k_stride, v_stride, T, slots, cache_of(c)};
  return dt == AR_BF16 ? write_as<uint16_t>(a, c.head_dim, c.group_size, st)
                       : write_as<float>(a, c.head_dim, c.group_size, st);
}

ar_status ar_launch_kv4_read(const ar_kv4_cache& c, const int32_t* slots, int64_t T, int dt,
                             void* k, void* v, hipStream_t st) {
  const ReadArgs a{slots, k, v, T, cache_of(c)};
  return dt == AR_BF16 ? read_as<uint16_t>(a, c.head_dim, c.group_size, st)
                       : read_as<float>(a, c.head_dim, c.group_size, st);
}
