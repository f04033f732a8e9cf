// Block-scaled e4m3 product, dense and by expert (gfx950):
//   Y[r, n] = sum over blocks j of 128 k:
//             xs[j, row(r)] · ws[e, n/128, j] · sum_{k in j} X[row(r), k]·W[e, n, k]
// with X [T, K], W [E, N, K] e4m3 row-major, xs [KB, T] and ws [E, NB, KB]
// float32 (ar_fp8.hip writes both). The rows offsets[e] <= r < offsets[e + 1]
// of Y are expert e's; row(r) = r or row_index[r]. The dense product is the
// case E = 1 with all rows.
//
// The inner sum of one block comes from the matrix unit, from a zero
// accumulator, and joins a float32 accumulator with one fma by the product of the
// two scales. W is the A operand and X the B operand, so a lane holds four
// neighbouring n of one row r: the row's scale is one value per lane, W's scale
// is one value for a whole wave, and Y is stored four values at a time. A and B
// use one assignment of k to lanes (two 16-byte chunks, 64 bytes apart: K is
// summed over, so any will do).
//
// Two kernels: k_fp8_rows for few rows, where W's bytes are the cost, and k_fp8_tile
// for the rest; ar_fp8_plan.h chooses. What bounds them, in a stream of calls on two
// inputs in turn, with a large copy at 4.85 TB/s and a library e4m3 product with one scale
// per operand at 2.41 PFLOP/s (16384 x 4096 x 4096) on the same card:
//   rows, 1 x 29568 x 8192            44 us, 5.5 TB/s: memory
//   32x64 tiles, 16 x 29568 x 8192    47 us, 5.1 TB/s: memory
//   64x128 tiles, 24 tokens, 4 of 64 experts (30 used), 2048 x 2048: 28 us, 4.5 TB/s: memory
//   256x256 tiles, 16384 x 4096 x 4096    232 us, 2.37 PFLOP/s; 8192^3 438 us, 2.51
//   the same by expert, 8192 tokens, 2 of 8, 11008 x 4096: 730 us, 2.02 PFLOP/s
//   128x128 tiles, float32 Y, 16384 x 4096 x 4096: 475 us, 1.16 PFLOP/s
// The 256x256 tile keeps the matrix unit busy 56% of the time at 1.85 GHz. On random codes, where
// it takes 265 us, it takes 220 without the loop's loads, 242 without the scale fmas
// and 247 without Y's stores: all CUs end their tiles at about the same time, and a
// round of tiles is 33 MB of Y. The float32 form converts every code a wave reads; its
// matrix work alone would take 250 us.
#include <type_traits>

#include "ar_device.h"
#include "ar_fp8_plan.h"
#include "ar_launch.h"

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

constexpr int BLK = 128;

inline ar_status last_status() { return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP; }

struct Args {
  const uint8_t* X;
  const float* xs;
  const uint8_t* W;
  const float* ws;
  const int32_t* off;   // [E + 1], NULL: one expert with all R rows
  const int32_t* idx;   // [R], NULL: row r of X
  void* Y;
  int ydt;
  int64_t T, R, N, K;
  int E, NB, KB;
};

// The dispatcher places workgroup w on XCD w mod 8; this gives each XCD one
// contiguous range of 0 .. n - 1.
__device__ __forceinline__ int xcd_range(int w, int n) {
  const int xcd = w & 7;
  return xcd * (n >> 3) + min(xcd, n & 7) + (w >> 3);
}

// Tile t of the rows cut into tiles of TM within each expert: expert e, first
// row r0 and row count (0: there is no such tile). Offsets are clamped to
// [0, R], so no table of offsets leads outside the arrays. The whole wave
// calls it; 64 experts are scanned at a time.
template <int TM>
__device__ __forceinline__ void find_tile(const Args& a, int t, int& e, int64_t& r0, int& rows) {
  e = 0;
  rows = 0;
  r0 = 0;
  if (!a.off) {
    r0 = (int64_t)t * TM;
    rows = (int)(a.R - r0 < TM ? a.R - r0 : TM);
    return;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int ee = base + lane;
    int lo = 0, hi = 0;
    if (ee < a.E) {
      const int R = (int)a.R;
      lo = min(max(a.off[ee], 0), R);
      hi = min(max(a.off[ee + 1], lo), R);
    }
    const int tiles = (hi - lo + TM - 1) / TM;
    int sum = tiles;   // inclusive scan over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d, 64);
      if (lane >= d) sum += up;
    }
    const uint64_t past = __ballot(before + sum > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __shfl(sum, l, 64) - __shfl(tiles, l, 64);
      const int elo = __shfl(lo, l, 64), ehi = __shfl(hi, l, 64);
      e = __builtin_amdgcn_readfirstlane(base + l);
      const int at = __builtin_amdgcn_readfirstlane(elo + (t - first) * TM);
      // (offsets that decrease may count more tiles than an int holds: no row then)
      const int lo0 = __builtin_amdgcn_readfirstlane(elo);
      r0 = at;
      rows = at >= lo0 ? min(__builtin_amdgcn_readfirstlane(ehi) - at, TM) : 0;
      return;
    }
    before += __shfl(sum, 63, 64);
  }
}

__device__ __forceinline__ void store_y(const Args& a, int64_t r, int64_t n, const float (&v)[4]) {
  if (a.ydt == AR_BF16) {
    uint16_t* y = static_cast<uint16_t*>(a.Y) + r * a.N + n;
    if (n + 3 < a.N && a.N % 4 == 0) {
      *reinterpret_cast<u32x2_t*>(y) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) y[i] = (uint16_t)bf16_bits(v[i]);
    }
  } else {
    float* y = static_cast<float*>(a.Y) + r * a.N + n;
    if (n + 3 < a.N && a.N % 4 == 0) {
      *reinterpret_cast<f32x4_t*>(y) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) y[i] = v[i];
    }
  }
}

// One block's products. A fragment is 32 codes of one row; the unscaled
// v_mfma_f32_16x16x128_f8f6f4 (scale operands 0) multiplies two of them at twice
// the bf16 rate, but adds 8 neighbouring products with 13 bits below the exponent of
// the largest, cutting the rest off (measured with single products beside a pair that
// cancels), and only those sums in float32: 1.3e-5 to 3.7e-5 of the block's sum on
// random operands, a hundredth of the half step of a bf16 output (2^-9 on
// average), and far below the operands' own rounding to e4m3 (2^-4 of a product). For
// a float32 output that would be the largest error by far, so there, and where float32
// sums are asked for, the codes are widened to bf16 (exact) and multiplied by
// v_mfma_f32_16x16x32_bf16 (1e-8, measured), at half the rate.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
struct WideFrag {
  bf16x8_t v[4];
};
template <bool WIDE>
struct FragOf {
  typedef i32x8_t type;
  static __device__ __forceinline__ type of(const i32x8_t& x) { return x; }
  static __device__ __forceinline__ f32x4_t mul(const type& w, const type& x) {
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
  }
};
template <>
struct FragOf<true> {
  typedef WideFrag type;
  static __device__ __forceinline__ type of(const i32x8_t& x) {
    WideFrag f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t d = (uint32_t)x[2 * c + h];
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false);
        const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true);
        f.v[c][4 * h] = lo[0];
        f.v[c][4 * h + 1] = lo[1];
        f.v[c][4 * h + 2] = hi[0];
        f.v[c][4 * h + 3] = hi[1];
      }
    return f;
  }
  static __device__ __forceinline__ f32x4_t mul(const type& w, const type& x) {
    f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[c], x.v[c], d, 0, 0, 0);
    return d;
  }
};

// A block's term is p·(sw·sx), |p| in 2^-18 .. 2^25 or 0, and one fma adds it. Where s = sw·sx
// leaves float32's normal range, though, the term need not. Below, s is off by up
// to 2^-150 and the term by 2^-125, all of K's (2^15 blocks) by 2^-110: no half step of a
// sum of 2^-86 or more. Above, the sum is infinite or NaN. So the kernels look at their sums when
// all is added: where one is below 2^-80 or no finite number, they go through the scales
// once Y is stored, and where there is such an s they sum that part of Y again, with
// the scales' mantissas and exponents apart. (Tested at every block instead, 2 to 5% slower.)
__device__ __forceinline__ bool out_of_range(float s) {
  return __builtin_amdgcn_classf(s, 0x2F4);   // infinite, subnormal or zero
}
__device__ __forceinline__ f32x4_t add_block(f32x4_t acc, const f32x4_t& p, float sw, float sx) {
  const float s = sw * sx;
  const float m = __builtin_amdgcn_frexp_mantf(sw) * __builtin_amdgcn_frexp_mantf(sx);
  const int e = __builtin_amdgcn_frexp_expf(sw) + __builtin_amdgcn_frexp_expf(sx);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc[i] = out_of_range(s) ? acc[i] + ldexpf(p[i] * m, e) : fmaf(p[i], s, acc[i]);
  return acc;
}
// Whether an element of Y is below 2^-80 or no finite number, in the bits as they are stored:
// twice the magnitude's bits less twice 2^-80's, which a smaller magnitude makes wrap.
struct Seen {
  uint32_t f32 = 0;
  u16x2_t bf16 = {0, 0};
  template <bool BF16>
  __device__ __forceinline__ void take(uint32_t v) {
    if constexpr (BF16) {
      const u16x2_t t = __builtin_bit_cast(u16x2_t, v) * (uint16_t)2 - (uint16_t)(2 * 0x1780);
      bf16 = __builtin_elementwise_max(bf16, t);
    } else {
      f32 = max(f32, (v << 1) - 2u * 0x17800000u);
    }
  }
  __device__ __forceinline__ bool odd() const {
    return __any(f32 >= 0xFF000000u - 2u * 0x17800000u ||
                 max(bf16[0], bf16[1]) >= 0xFF00 - 2 * 0x1780);
  }
};

// Two 16-byte chunks of a row, 64 bytes apart (p 16-byte aligned); in a row's last,
// short block the chunks past the `left` bytes from p on are zero (K % 16 == 0).
__device__ __forceinline__ i32x8_t frag(const uint8_t* p) {
  const i32x4_t a = reinterpret_cast<const i32x4_t*>(p)[0];
  const i32x4_t b = reinterpret_cast<const i32x4_t*>(p)[4];
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ i32x8_t frag_tail(const uint8_t* p, int left) {
  i32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  if (left > 0) a = reinterpret_cast<const i32x4_t*>(p)[0];
  if (left > 64) b = reinterpret_cast<const i32x4_t*>(p)[4];
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Row of X behind row r of Y; -1 when row_index names none (its row of Y is zero).
__device__ __forceinline__ int64_t x_row(const Args& a, int64_t r) {
  if (!a.idx) return r;
  const int i = a.idx[r];
  return i >= 0 && i < a.T ? i : -1;
}

// The part of Y of rows r0 + r1 .. (16·MB of them, `rows` in the tile from r0 on) and columns n1 ..
// (16·NA): whether the product of two scales is out of range.
__device__ __forceinline__ bool far_scales(const Args& a, int64_t r0, int r1, int MB, int rows,
                                           const float* wsp) {
  const int lane = threadIdx.x & 63;
  bool far = false;
#pragma unroll 1
  for (int b = 0; b < MB; ++b) {
    const int r = r1 + b * 16 + (lane & 15);
    const int64_t xr = r < rows ? x_row(a, r0 + r) : -1;
    if (xr < 0) continue;
#pragma unroll 4
    for (int k = lane >> 4; k < a.KB; k += 4) {
      const float sw = wsp[k], sx = a.xs[k * a.T + xr];
      // (a zero, infinite or NaN scale gives the same either way)
      far |= out_of_range(sw * sx) && !__builtin_amdgcn_classf(sw, 0x267) &&
             !__builtin_amdgcn_classf(sx, 0x267);
    }
  }
  return __any(far);
}
// The same part summed again straight from memory, 16 x 16 at a time, by add_block. K is
// summed in `sets` parts and these are added in order, as in the kernel that calls, so that other
// rows and columns keep their bits: set g takes the blocks from g·first on, `stride` apart,
// up to `count` of them. What the wave stored there before has arrived first: other lanes did.
template <bool WIDE>
__device__ __forceinline__ void sum_again(const Args& a, int e, int64_t r0, int r1, int MB, int rows,
                                          int64_t n1, int NA, const float* wsp, int sets, int first,
                                          int stride, int count) {
  typedef FragOf<WIDE> Op;
  const int lane = threadIdx.x & 63, l16 = lane & 15, kc = 16 * (lane >> 4);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll 1
  for (int u = 0; u < MB * NA; ++u) {
    const int r = r1 + u % MB * 16 + l16;
    const int64_t n = n1 + u / MB * 16;
    const int64_t xr = x_row(a, r0 + min(r, rows - 1));
    const uint8_t* wp = a.W + ((int64_t)e * a.N + min(n + l16, a.N - 1)) * a.K + kc;
    const uint8_t* xp = a.X + max(xr, (int64_t)0) * a.K + kc;
    const float* xsp = a.xs + max(xr, (int64_t)0);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int g = 0; g < sets; ++g) {
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const int k = g * first + i * stride;
        if (k >= a.KB) break;
        const int left = (int)(a.K - (int64_t)k * BLK) - kc;
        const f32x4_t p = Op::mul(Op::of(frag_tail(wp + (int64_t)k * BLK, left)),
                                  Op::of(frag_tail(xp + (int64_t)k * BLK, left)));
        acc = add_block(acc, p, wsp[k], xsp[(int64_t)k * a.T]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += acc[i];
    }
    if (xr < 0) v[0] = v[1] = v[2] = v[3] = 0.0f;
    if (r < rows) store_y(a, r0 + r, n + 4 * (lane >> 4), v);
  }
}

// ------------------------------------------------------------------ few rows
// Operands straight from memory to registers. A workgroup of 8 waves makes a
// tile of 16 columns by 16 rows (rows past the tile's repeat its last one, and
// are not stored); the waves take the blocks of K in turn (wave w: blocks w,
// w + 8, ...; four of them requested at a time) and their sums are added
// through LDS in wave order.
constexpr int DW = 8;

template <bool WIDE>
__global__ __launch_bounds__(64 * DW) void k_fp8_rows(Args a) {
  typedef FragOf<WIDE> Op;
  __shared__ float red[DW][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e, rows;
  int64_t r0;
  find_tile<16>(a, blockIdx.y, e, r0, rows);
  if (rows <= 0) return;
  const int l16 = lane & 15, kc = 16 * (lane >> 4);
  const int64_t n0 = (int64_t)xcd_range(blockIdx.x, gridDim.x) * 16;
  const int64_t n = n0 + l16 < a.N ? n0 + l16 : a.N - 1;
  const uint8_t* wp = a.W + ((int64_t)e * a.N + n) * a.K + kc;
  const float* wsp = a.ws + ((int64_t)e * a.NB + n0 / BLK) * a.KB;
  const int64_t xr = x_row(a, r0 + (l16 < rows ? l16 : rows - 1));
  const uint8_t* xp = a.X + (xr < 0 ? 0 : xr) * a.K + kc;
  const float* xsp = a.xs + (xr < 0 ? 0 : xr);
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const int full = (int)(a.K / BLK);
  auto add = [&](const i32x8_t& w, const i32x8_t& x, float s) {
    const f32x4_t p = Op::mul(Op::of(w), Op::of(x));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
  };
  auto batch = [&](int j, auto count) {
    constexpr int U = decltype(count)::value;
    i32x8_t w[U], x[U];
    float sw[U], sx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = j + u * DW;
      w[u] = frag(wp + k * BLK);
      x[u] = frag(xp + k * BLK);
      sw[u] = wsp[k];
      sx[u] = xsp[k * a.T];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) add(w[u], x[u], sw[u] * sx[u]);
    return j + U * DW;
  };
  int j = wave;
  while (j + 3 * DW < full) j = batch(j, std::integral_constant<int, 4>());
  if (j + DW < full) j = batch(j, std::integral_constant<int, 2>());
  if (j < full) j = batch(j, std::integral_constant<int, 1>());
  if (j < a.KB) {   // j = full: the short block
    const int left = (int)(a.K - (int64_t)full * BLK) - kc;
    add(frag_tail(wp + (int64_t)full * BLK, left), frag_tail(xp + (int64_t)full * BLK, left),
        wsp[full] * xsp[(int64_t)full * a.T]);
  }
  *reinterpret_cast<f32x4_t*>(red[wave][lane]) = acc;
  __syncthreads();
  if (wave == 0) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < DW; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += red[w][lane][i];
    if (xr < 0) v[0] = v[1] = v[2] = v[3] = 0.0f;
    Seen seen;
    if (l16 < rows) {
      store_y(a, r0 + l16, n0 + 4 * (lane >> 4), v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + 4 * (lane >> 4) + i < a.N) seen.take<false>(__float_as_uint(v[i]));
    }
    if (seen.odd() && far_scales(a, r0, 0, 1, rows, wsp))
      sum_again<WIDE>(a, e, r0, 0, 1, rows, n0, 1, wsp, DW, 1, DW, (a.KB + DW - 1) / DW);
  }
}

// ------------------------------------------------------------------ many rows
// Tiles of TM = 16·MB·WM rows by TN = 16·NA·WN columns, one wave per 16·MB x 16·NA
// part. A step is one block of 128 k: W's and X's rows of the tile (128 bytes
// each) and X's scales go straight from memory to LDS, NS stages of them. In
// LDS, 16-byte chunk c of row r sits at chunk c ^ ((r >> 1) & 7), so that the 16
// rows a fragment read touches with one chunk number lie in 16 different
// 16-byte slots of a 256-byte LDS cycle.
//
// A wave keeps its MB X fragments of the step and streams its NA W fragments
// past them, two ahead. When the last H of them are in registers, the wave waits
// for the next stage's loads and the workgroup meets; while the products of those
// H run, the stage just left is filled for NS steps ahead and the next step's
// fragments are read, each X fragment as the old one is done with. H = 3 spreads
// these reads, half of all, over more products, where registers allow it and a
// step is long: 256x256 tiles, 234 -> 231 us at 16384 x 4096 x 4096;
// 64x128 tiles are 2% slower with it.
//
// With KG > 1 a workgroup has KG such sets of waves and stages, each on its own
// contiguous part of the blocks of K (steps past the end add zeros); the sums of
// sets 1 .. KG - 1 join those of set 0 through LDS, in order. It shortens the
// chain of steps where there are too few tiles to keep several workgroups on
// each CU.
template <int WM, int WN, int MB, int NA, int NS, int KG>
struct Tile {
  static constexpr int TM = 16 * MB * WM, TN = 16 * NA * WN, NW = WM * WN;
  static constexpr int W_BYTES = TN * BLK, X_BYTES = TM * BLK;
  static constexpr int SROWS = TM < 64 ? 64 : TM;            // rows of scales loaded, 64 at a time
  static constexpr int STAGE = W_BYTES + X_BYTES + SROWS * 4;
  static constexpr int RING = NS * STAGE, LDS = KG * RING, THREADS = 64 * NW * KG;
  static constexpr int IW = TN / 8 / NW, IX = TM / 8 / NW;   // 1 KiB loads per wave and operand
  static constexpr int LOADS = IW + IX + 1;                  // of one wave and step
  static constexpr int H = NA >= 8 ? 3 : 2;                  // W fragments held at a step's end
  static_assert(IW * NW * 8 == TN && IX * NW * 8 == TM, "whole loads");
  static_assert(LDS <= 160 * 1024 && (NS - 1) * LOADS < 64, "LDS of a workgroup, vmcnt's range");
};

// Waits until at most n of the wave's vector-memory operations and none of its LDS
// operations are outstanding.
template <int n>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
}
constexpr uint32_t kNone = 0xFFFFFFF0u;   // past every buffer: the load writes zeros

// Workgroup -> (m tile, n tile). The tile sequence walks groups of GI tile rows,
// column by column; of each 256 tiles in a row (one for every CU) an XCD gets 32
// neighbours, which share operands in its L2, and all XCDs stay near one place
// of the sequence, so that what they stream (an expert's W above all) is in the
// last-level cache when the second one asks. Measured on 8192 tokens, 2 of 8
// experts, 11008 x 4096: 722 us against 768 with an eighth of the whole sequence
// per XCD. With one tile row nothing is read twice, and an eighth of W each is
// faster: 16 x 29568 x 8192, 46 us against 51.
__device__ __forceinline__ void tile_of(int w, int n, int tilesM, int tilesN, int& tm, int& tn) {
  constexpr int GI = 4, WINDOW = 256;
  const int base = tilesM == 1 ? 0 : w & ~(WINDOW - 1);
  const int L = base + xcd_range(w - base, tilesM == 1 ? n : min(n - base, WINDOW));
  const int g = L / (GI * tilesN), first = g * GI;
  const int size = min(tilesM - first, GI), in = L - g * GI * tilesN;
  tm = first + in % size;
  tn = in / size;
}

// Tiles of TM rows in all ranges (the dense product: of all rows).
template <int TM>
__device__ __forceinline__ int count_tiles(const Args& a) {
  if (!a.off) return (int)((a.R + TM - 1) / TM);
  int n = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int e = base + (threadIdx.x & 63);
    if (e < a.E) {
      const int R = (int)a.R, lo = min(max(a.off[e], 0), R);
      n += (min(max(a.off[e + 1], lo), R) - lo + TM - 1) / TM;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  return __builtin_amdgcn_readfirstlane(n);
}

template <int WM, int WN, int MB, int NA, int NS, int KG, bool WIDE, class O>   // O: Y's type
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void k_fp8_tile(Args a, int mostM, int tilesN) {
  typedef Tile<WM, WN, MB, NA, NS, KG> C;
  typedef FragOf<WIDE> Op;
  constexpr int H = C::H;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[C::LDS];
  const int lane = threadIdx.x & 63;
  const int gwave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = gwave / C::NW, wave = gwave % C::NW;
  uint8_t* lds = lds_all + set * C::RING;
  const int wm = wave % WM, wn = wave / WM;
  const int tilesM = min(count_tiles<C::TM>(a), mostM);
  if ((int)blockIdx.x >= tilesM * tilesN) return;   // more workgroups than tiles: ragged ranges
  int tm, tn, e, rows;
  int64_t r0;
  tile_of(blockIdx.x, tilesM * tilesN, tilesM, tilesN, tm, tn);
  find_tile<C::TM>(a, tm, e, r0, rows);
  if (rows <= 0) return;
  const int64_t n0 = (int64_t)tn * C::TN;
  const uint32_t K = (uint32_t)a.K;
  const int steps = (a.KB + KG - 1) / KG;                  // of every set
  const int kb0 = set * steps, kb1 = min(kb0 + steps, a.KB);
  const uint32_t kend = min((uint32_t)kb1 * BLK, K);

  // Loads: piece i of an operand is rows 8·(wave·I + i) .. + 7 of its tile, eight
  // lanes of 16 bytes a row; chunk[] is the lane's k offset within the block.
  const int cols = (int)(a.N - n0 < C::TN ? a.N - n0 : C::TN);
  const __amdgpu_buffer_rsrc_t bw =
      make_rsrc(a.W + ((int64_t)e * a.N + n0) * a.K, (uint32_t)cols * K);
  const __amdgpu_buffer_rsrc_t bx =
      a.idx ? make_rsrc(a.X, (uint32_t)((uint64_t)a.T * K))
            : make_rsrc(a.X + r0 * a.K, (uint32_t)rows * K);
  auto chunk = [&](int r) { return (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) * 16); };
  uint32_t vw[C::IW], vx[C::IX];
#pragma unroll
  for (int i = 0; i < C::IW; ++i) {
    const int r = 8 * (wave * C::IW + i) + (lane >> 3);
    vw[i] = r < cols ? (uint32_t)r * K + chunk(r) : kNone;
  }
#pragma unroll
  for (int i = 0; i < C::IX; ++i) {
    const int r = 8 * (wave * C::IX + i) + (lane >> 3);
    int64_t x = -1;
    if (r < rows) x = a.idx ? x_row(a, r0 + r) : r;
    vx[i] = x >= 0 ? (uint32_t)x * K + chunk(r) : kNone;
  }
  // scales: 64 rows per wave, four bytes a lane
  const int sw0 = 64 * (wave % (C::SROWS / 64)), sr = sw0 + lane;
  uint32_t vs = kNone;
  if (sr < rows) {
    const int64_t x = a.idx ? x_row(a, r0 + sr) : sr;
    if (x >= 0) vs = (uint32_t)x * 4u;
  }
  const float* xs = a.xs + (a.idx ? 0 : r0);
  const uint32_t xs_bytes = (uint32_t)(a.idx ? a.T : rows) * 4u;
#define AR_LDS(p) ((__attribute__((address_space(3))) void*)(p))
  // Past the last block (and in its missing chunks) the loads write zeros, so the
  // loop needs no branch around them.
  auto issue = [&](int kt, int stage, int piece) {
    uint8_t* st = lds + stage;
    const uint32_t so = (uint32_t)kt * BLK;
    const bool tail = so + BLK > kend;
    if (piece < C::IW) {
      const int i8 = wave * C::IW + piece, r = 8 * i8 + (lane >> 3);
      const uint32_t v = tail && so + chunk(r) >= kend ? kNone : vw[piece];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bw, AR_LDS(st + i8 * 1024), 16, v, so, 0, 0);
    } else if (piece < C::IW + C::IX) {
      const int i8 = wave * C::IX + piece - C::IW, r = 8 * i8 + (lane >> 3);
      const uint32_t v = tail && so + chunk(r) >= kend ? kNone : vx[piece - C::IW];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bx, AR_LDS(st + C::W_BYTES + i8 * 1024), 16, v, so,
                                               0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          make_rsrc(xs + (int64_t)kt * a.T, xs_bytes),
          AR_LDS(st + C::W_BYTES + C::X_BYTES + sw0 * 4), 4, kt < kb1 ? vs : kNone, 0, 0, 0);
    }
  };
#undef AR_LDS

  // Fragments: lane l reads row l % 16, chunks l / 16 and l / 16 + 4. An LDS cycle
  // serves 16 lanes of two neighbouring quarters of the wave, rows 0-3 and 12-15 of
  // one and 4-11 of the other (or the reverse): with chunk numbers that differ
  // in the last bit only, their slots are all different.
  const int l16 = lane & 15, q = lane >> 4;
  const uint32_t slot = (uint32_t)((q ^ (l16 >> 1)) * 16);
  const uint32_t aw = (uint32_t)(wn * NA * 16 + l16) * BLK + slot;
  const uint32_t ax = (uint32_t)C::W_BYTES + (uint32_t)(wm * MB * 16 + l16) * BLK + slot;
  const uint32_t as = (uint32_t)(C::W_BYTES + C::X_BYTES) + (uint32_t)(wm * MB * 16 + l16) * 4;
  auto rd = [&](int stage, uint32_t at) {
    const uint8_t* st = lds + stage;
    const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(st + at);
    const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(st + (at ^ 64u));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  // W's scales of this wave's columns (one block of 128), 64 blocks of K at a time
  const int64_t nb = (n0 + wn * NA * 16) / BLK;
  const float* wsp = a.ws + ((int64_t)e * a.NB + (nb < a.NB ? nb : a.NB - 1)) * a.KB;
  auto window = [&](int k0) { return k0 + lane < kb1 ? wsp[k0 + lane] : 0.0f; };
  float wsv = window(kb0);   // requested before the stages, so that it arrives first

  f32x4_t acc[NA][MB];
#pragma unroll
  for (int t = 0; t < NA; ++t)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[t][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  int cur = 0, nxt = C::STAGE;   // stages of steps kt and kt + 1
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) issue(kb0 + i, i * C::STAGE, j);
  wait_loads<(NS - 1) * C::LOADS>();
  meet();
  // W fragment t of a step is in fw[t % 4] (with NA = 2, where a step's last two
  // fragments are all it has, the next step's two come in through fw[2] and fw[3])
  // Fragments are kept as read, and widened (WIDE) where they are used: a conversion
  // at the read would wait for it.
  i32x8_t rx[MB], fw[4];
  float sx[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    rx[b] = rd(0, ax + b * 16 * BLK);
    sx[b] = *reinterpret_cast<const float*>(lds + as + b * 64);
  }
  fw[0] = rd(0, aw);
  fw[1] = rd(0, aw + 16 * BLK);

  auto step = [&](int kt) {
    const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv), (kt - kb0) & 63));
    float s[MB];
    typename Op::type fx[MB], w[H];   // w: the W fragments in use
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      s[b] = sw * sx[b];
      fx[b] = Op::of(rx[b]);
    }
    // Items: W fragment by W fragment up to the last H, those X fragment by X
    // fragment. Products join the accumulators three items behind the matrix
    // unit's issue.
    constexpr int ITEMS = NA * MB, LAST = (NA - H) * MB;
    auto tile = [](int u) { return u < LAST ? u / MB : NA - H + (u - LAST) % H; };
    auto part = [](int u) { return u < LAST ? u % MB : (u - LAST) / H; };
    f32x4_t p[4];
    auto join = [&](int u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[tile(u)][part(u)][i] = fmaf(p[u % 4][i], s[part(u)], acc[tile(u)][part(u)][i]);
    };
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
      const int t = tile(u), b = part(u);
      if (u == LAST) {
        // the next step's stage has landed, this one's reads are done; then everyone's
        wait_loads<(NS - 2) * C::LOADS>();
        meet();
      }
      const int h = u < LAST ? 0 : t - (NA - H);
      if (b == 0) w[h] = Op::of(fw[t % 4]);
      p[u % 4] = Op::mul(w[h], fx[b]);
      if (u < LAST) {
        if (b == 0) fw[(t + 2) % 4] = rd(cur, aw + (t + 2) * 16 * BLK);
        if (H == 3 && t == NA - 4 && b == MB / 2)
          fw[(NA - 1) % 4] = rd(cur, aw + (NA - 1) * 16 * BLK);
      } else {
        constexpr int EACH = (C::LOADS + H * MB - 1) / (H * MB);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
          if ((u - LAST) * EACH + i < C::LOADS) issue(kt + NS, cur, (u - LAST) * EACH + i);
        if (t == NA - 1) {   // the next step's fragments replace these
          rx[b] = rd(nxt, ax + b * 16 * BLK);
          sx[b] = *reinterpret_cast<const float*>(lds + nxt + as + b * 64);
          if (b == 0) fw[NA % 4] = rd(nxt, aw);
          if (b == MB - 1) fw[(NA + 1) % 4] = rd(nxt, aw + 16 * BLK);
        }
      }
      if (u >= 3) join(u - 3);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = ITEMS > 3 ? ITEMS - 3 : 0; u < ITEMS; ++u) join(u);
    if constexpr (NA == 2) {
      fw[0] = fw[2];
      fw[1] = fw[3];
    }
    cur = nxt;
    nxt = nxt + C::STAGE == C::RING ? 0 : nxt + C::STAGE;
  };
  for (int k0 = kb0; k0 < kb0 + steps; k0 += 64) {
    if (k0 > kb0) wsv = window(k0);
    asm volatile("" : "+v"(wsv));   // waits for it here, not in every step
    const int k1 = min(k0 + 64, kb0 + steps);
    for (int kt = k0; kt < k1; ++kt) step(kt);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no load may land in LDS after the end

  // The wave's part of Y goes through LDS (the stages are free once everyone is
  // here) so that rows leave as whole runs of 128 or 256 bytes, past the caches:
  // the tiles of all CUs end at about the same time. Measured at 16384 x 4096 x
  // 4096: 253 us instead of 267 from the accumulators, and 232 instead of 239 through the
  // caches. Rows of Y that are not 16-byte aligned leave in smaller units and through
  // the caches (12468 x 4831 x 256 on 256x256 tiles: 64 us, past them 78).
  __syncthreads();
  if constexpr (KG > 1) {
    static_assert((KG - 1) * C::TM * C::TN * 4 <= C::LDS, "the other sets' sums in LDS");
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds_all) + wave * (NA * MB * 64) + lane;
    if (set > 0)
#pragma unroll
      for (int u = 0; u < NA * MB; ++u)
        sums[((set - 1) * C::NW * NA * MB + u) * 64] = acc[u / MB][u % MB];
    __syncthreads();
    if (set > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int u = 0; u < NA * MB; ++u) {
        const f32x4_t v = sums[(g * C::NW * NA * MB + u) * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u / MB][u % MB][i] += v[i];
      }
    static_assert((KG - 1) * C::TM * C::TN * 4 + C::TM * C::TN * 4 <= C::LDS, "beside Y's tile");
    lds = lds_all + (KG - 1) * C::TM * C::TN * 4;
  }
  // A row that names none is zero even where W holds a NaN or an infinite scale.
  if (a.idx) {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int r = wm * MB * 16 + 16 * b + l16;
      if (r < rows && x_row(a, r0 + r) < 0)
#pragma unroll
        for (int t = 0; t < NA; ++t) acc[t][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
  Seen seen;
  constexpr int RB = NA * 16 * (int)sizeof(O);             // bytes of a row of the part
  static_assert(C::NW * MB * 16 * RB <= C::LDS, "the tile of Y in LDS");
  uint8_t* own = lds + wave * (MB * 16 * RB);
  auto at = [&](int r, int byte) {   // 16-byte chunks spread over the banks by row
    return own + r * RB + (byte ^ ((r & (RB / 16 - 1)) * 16));
  };
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      const f32x4_t v = acc[t][b];
      uint8_t* d = at(16 * b + l16, (16 * t + 4 * q) * (int)sizeof(O));
      if constexpr (sizeof(O) == 2)
        *reinterpret_cast<u32x2_t*>(d) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      else
        *reinterpret_cast<f32x4_t*>(d) = v;
    }
  O* Y = static_cast<O*>(a.Y) + (r0 + wm * MB * 16) * a.N + n0 + wn * NA * 16;
  const int nleft = (int)(a.N - n0) - wn * NA * 16, mleft = rows - wm * MB * 16;
  auto write = [&](auto unit) {      // rows in pieces of one unit, whole or absent
    typedef decltype(unit) V;
    constexpr int PER = sizeof(V) / sizeof(O), UPR = RB / (int)sizeof(V);
#pragma unroll 8
    for (int i = lane; i < MB * 16 * UPR; i += 64) {
      const int r = i / UPR, u = i % UPR;
      if (r < mleft && u * PER < nleft) {
        const V v = *reinterpret_cast<const V*>(at(r, u * (int)sizeof(V)));
        V* d = reinterpret_cast<V*>(Y + (int64_t)r * a.N) + u;
        if constexpr (sizeof(V) == 16) __builtin_nontemporal_store(v, d);
        else *d = v;   // runs that end inside a line are joined in L2
        if constexpr (sizeof(V) < 4) {
          seen.take<false>((uint32_t)v << 16);   // (a bf16's bits, as a float32's)
        } else {
#pragma unroll
          for (int w = 0; w < (int)sizeof(V) / 4; ++w) {
            if constexpr (sizeof(V) == 4) seen.take<sizeof(O) == 2>(v);
            else seen.take<sizeof(O) == 2>(v[w]);
          }
        }
      }
    }
  };
  const int64_t pitch = a.N * (int64_t)sizeof(O);
  if (pitch % 16 == 0) write(u32x4_t{});
  else if (pitch % 8 == 0) write(u32x2_t{});
  else if (sizeof(O) == 4 || pitch % 4 == 0) write(uint32_t{});
  else write(uint16_t{});
  if (seen.odd() && far_scales(a, r0, wm * MB * 16, MB, rows, wsp))
    sum_again<WIDE>(a, e, r0, wm * MB * 16, MB, rows, n0 + wn * NA * 16, NA, wsp, KG, steps, 1,
                    steps);
}

}  // namespace

template <int WM, int WN, int MB, int NA, int NS, int KG, bool WIDE, class O>
static ar_status tile_launch(const Args& a, const ArFp8Shape& g, hipStream_t st) {
  typedef Tile<WM, WN, MB, NA, NS, KG> C;
  const int64_t tilesM = ar_fp8_most_tiles(g, C::TM);
  const int64_t tilesN = (a.N + C::TN - 1) / C::TN;
  if (tilesM * tilesN * C::THREADS >= (int64_t(1) << 32)) return AR_ERR_SHAPE;   // HIP's limit
  hipLaunchKernelGGL((k_fp8_tile<WM, WN, MB, NA, NS, KG, WIDE, O>), dim3((unsigned)(tilesM * tilesN)),
                     dim3(C::THREADS), 0, st, a, (int)tilesM, (int)tilesN);
  return last_status();
}

static ar_status rows_launch(const Args& a, const ArFp8Shape& g, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)ar_fp8_most_tiles(g, 16));
  if (g.wide)
    hipLaunchKernelGGL((k_fp8_rows<true>), grid, dim3(64 * DW), 0, st, a);
  else
    hipLaunchKernelGGL((k_fp8_rows<false>), grid, dim3(64 * DW), 0, st, a);
  return last_status();
}

template <int WM, int WN, int MB, int NA, int NS, int KG>
static ar_status tile_sums(const Args& a, const ArFp8Shape& g, hipStream_t st) {
  if (!g.wide) return tile_launch<WM, WN, MB, NA, NS, KG, false, uint16_t>(a, g, st);
  return a.ydt == AR_BF16 ? tile_launch<WM, WN, MB, NA, NS, KG, true, uint16_t>(a, g, st)
                          : tile_launch<WM, WN, MB, NA, NS, KG, true, float>(a, g, st);
}
template <int WM, int WN, int MB, int NA, int NS>
static ar_status tile_pick(const Args& a, const ArFp8Shape& g, bool two, hipStream_t st) {
  return two ? tile_sums<WM, WN, MB, NA, NS, 2>(a, g, st)
             : tile_sums<WM, WN, MB, NA, NS, 1>(a, g, st);
}

ar_status ar_launch_fp8_gemm(const ArFp8Gemm& g, hipStream_t st) {
  const Args a{g.X, g.xs, g.W, g.ws, g.offsets, g.row_index, g.Y, g.ydt, g.T, g.R, g.N, g.K,
               (int)g.E, (int)((g.N + BLK - 1) / BLK), (int)((g.K + BLK - 1) / BLK)};
  const ArFp8Shape shape{g.offsets != nullptr, g.wide, g.R, g.N, g.K, g.E};
  const ArFp8Plan p = ar_fp8_plan(shape);
  switch (p.kind) {
    case kRows: return rows_launch(a, shape, st);
    case k32x64: return tile_pick<2, 2, 1, 2, 4>(a, shape, p.two, st);
    case k64x64: return tile_pick<2, 2, 2, 2, 4>(a, shape, p.two, st);
    case k64x128: return tile_pick<2, 2, 2, 4, 3>(a, shape, p.two, st);
    case k128x128: return tile_pick<2, 2, 4, 4, 2>(a, shape, p.two, st);
    default: return tile_launch<4, 2, 4, 8, 2, 1, false, uint16_t>(a, shape, st);
  }
}
