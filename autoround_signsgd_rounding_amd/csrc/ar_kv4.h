// Layout of the 4-bit key/value cache on the device (ar_kv4.hip writes and reads it,
// ar_kv4_attn.hip attends to it).
//
// codes [pages][2][heads][page][Dh/2]: of a page and head first the keys, then (the
// second index) the values. Two codes share a byte, the even channel in its low half.
//   keys    token after token, the bytes in order: a lane of the product takes
//           neighbouring channels of one token.
//   values  in octets of tokens: byte 32·b + 16·c + n of token t is at
//           [t/8][b][n][t%8][c] (b < Dh/64, n < 16, c < 2): a lane of the product takes
//           eight tokens of four channels in one 16-byte load, and the two halves of
//           each 32-bit word are neighbouring tokens, as the matrix unit wants them.
// scale [pages][2][heads][page][G] float32: its four lowest mantissa bits are the
// group's zero-point, and the whole word is the scale. A value is scale·(code - zp).
#pragma once

#include "ar_device.h"

struct ArKv4 {
  uint8_t* codes;
  float* scale;
  int64_t pages;
  int heads, page, shift;   // page = 1 << shift
  int64_t codes_page() const { return (int64_t)2 * heads * page; }   // token rows of a page
};

// The zero-point of a scale.
__device__ __forceinline__ uint32_t kv4_zero(float s) { return __float_as_uint(s) & 15u; }

// Offset of value byte 32·b + 16·c + n of token t within a page's and head's values.
__device__ __forceinline__ int kv4_value_at(int t, int b, int n, int c, int B) {
  return ((((t >> 3) * B + b) * 16 + n) * 8 + (t & 7)) * 2 + c;
}
