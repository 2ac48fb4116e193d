// int8.cuh -- symmetric 8-bit codes of a row: with a = max |v| over the row,
//   scale = fl32(a / 127),  code = round-half-even(127 v / a)  (exact for bf16 values, see to_code for fp32),
// a row of zeros has scale 0 and codes 0, and a row that holds a NaN or an
// infinity has scale NaN and codes 0 (whatever it is multiplied with is NaN).
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {
namespace q8 {

struct RowScale {
  float inv;    // 127 / (a * pre), rounded up
  float scale;  // a / 127
  bool tiny;    // the row is lifted by `pre` = 2^66 so that inv does not overflow
  bool zero;    // every code is 0
};

constexpr float TINY_PRE = 0x1p66f;

__device__ __forceinline__ RowScale row_scale(float a) {
  RowScale r;
  const bool finite = a < INFINITY;  // false for NaN too
  r.zero = !finite || a == 0.0f;
  r.scale = finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fffffffu);
  r.tiny = a < 0x1p-60f;
  r.inv = r.zero ? 0.0f : __fdiv_ru(127.0f, r.tiny ? a * TINY_PRE : a);
  return r;
}

// Largest |v| of eight packed bf16 as a 16-bit pattern (NaN and infinity are 0x7f80 or above, so an
// integer maximum keeps them).
__device__ __forceinline__ uint32_t abs_max_bits(const uint4& v) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  return max(m & 0xffffu, m >> 16);
}

// The code of v in the low byte: v * inv rounded once to the nearest integer, ties to even, by adding 1.5 * 2^23 in the
// same fma (the sum's low byte is the integer's two's complement).
//
// For bf16 values this is the exact code of 127 v / a.  With 8-bit significands A of a and X of |v|, a half-integer
// quotient o / 2 means 254 X = o A 2^m, so the prime 127 divides A or o.  If it divides A, 127 / a is a power of two and
// inv and the product are exact.  If it divides o <= 253, then o = 127, |v| = a / 2, and inv rounded up makes the product
// 63.5 or just above: 64, the even neighbour, either way.  Every other quotient is at least 1.5e-5 of its value away
// from a half-integer, and inv is within 1.2e-7 of 127 / a.
// For fp32 values (the few-token layer's hidden rows) a quotient that lies below a half-integer by less than 2^-23 of itself
// may go to the code above; every other one is exact.
__device__ __forceinline__ uint32_t to_code(float v, float inv) { return __float_as_uint(__fmaf_rn(v, inv, 12582912.0f)); }

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <int N>
__device__ __forceinline__ void code_n(const float (&v)[N], const RowScale& r, uint32_t (&c)[N]) {
  if (r.tiny) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = to_code(v[i] * TINY_PRE, r.inv);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = to_code(v[i], r.inv);
  }
}

// Codes of eight packed bf16 values.
__device__ __forceinline__ uint2 code8(const uint4& v, const RowScale& r) {
  if (r.zero) return make_uint2(0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  uint32_t c[8];
  code_n(f, r, c);
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// Codes of four fp32 values.
__device__ __forceinline__ uint32_t code4_f32(const float (&v)[4], const RowScale& r) {
  if (r.zero) return 0;
  uint32_t c[4];
  code_n(v, r, c);
  return pack4(c[0], c[1], c[2], c[3]);
}

}  // namespace q8
}  // namespace moe
