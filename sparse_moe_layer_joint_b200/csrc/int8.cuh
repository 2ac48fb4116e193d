// int8.cuh -- symmetric 8-bit codes of a row: with a = max |v| over the row,
//   scale = fl32(a / 127),  code = round-half-even(127 v / a),
// a row of zeros has scale 0 and codes 0, and a row that holds a NaN or an
// infinity has scale NaN and codes 0 (whatever it is multiplied with is NaN).
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {
namespace q8 {

struct RowScale {
  float pre;    // power of two that lifts tiny rows into fp32's normal range
  float inv;    // 127 / (a * pre)
  float scale;  // a / 127
  bool zero;    // every code is 0
};

__device__ __forceinline__ RowScale row_scale(float a) {
  RowScale r;
  const bool finite = a < INFINITY;  // false for NaN too
  r.zero = !finite || a == 0.0f;
  r.scale = finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fffffffu);
  r.pre = a < 0x1p-60f ? 0x1p66f : 1.0f;
  r.inv = r.zero ? 0.0f : __fdiv_rn(127.0f, a * r.pre);
  return r;
}

// Largest |v| of eight packed bf16 as a 16-bit pattern (NaN and infinity are 0x7f80 or above, so an
// integer maximum keeps them).
__device__ __forceinline__ uint32_t abs_max_bits(const uint4& v) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  return max(m & 0xffffu, m >> 16);
}

// Adding 1.5 * 2^23 rounds |q| <= 127 to the nearest integer, ties to even, and leaves its two's complement
// in the low byte.
__device__ __forceinline__ uint32_t to_code(float q) { return __float_as_uint(__fadd_rn(q, 12582912.0f)); }

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The exact code of a bf16 value without a division.  With 8-bit significands, 127 v / a is either exactly a
// half-integer or at least 1.5e-5 of its value away from one, and q = fl(v * fl(127 / a)) is within 2.4e-7 of
// it.  Rounding q to 17 significant bits (Veltkamp's splitting, within 3.9e-6) therefore lands on a
// half-integer exactly when the quotient is one, so the final rounding to even decides true ties only.
__device__ __forceinline__ uint32_t code_bf16(float v, const RowScale& r) {
  const float q = __fmul_rn(__fmul_rn(v, r.pre), r.inv);
  const float c = __fmul_rn(q, 129.0f);
  return to_code(__fsub_rn(c, __fsub_rn(c, q)));
}

__device__ __forceinline__ uint2 code8(const uint4& v, const RowScale& r) {
  if (r.zero) return make_uint2(0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = code_bf16(__uint_as_float(w[i] << 16), r);
    c[2 * i + 1] = code_bf16(__uint_as_float(w[i] & 0xffff0000u), r);
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// Codes of four fp32 values (within 2.4e-7 of the quotient before the rounding to an integer).
__device__ __forceinline__ uint32_t code4_f32(const float (&v)[4], const RowScale& r) {
  if (r.zero) return 0;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = to_code(__fmul_rn(__fmul_rn(v[i], r.pre), r.inv));
  return pack4(c[0], c[1], c[2], c[3]);
}

}  // namespace q8
}  // namespace moe
