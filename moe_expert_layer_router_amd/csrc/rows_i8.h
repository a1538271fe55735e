// Codes and scales of rows as 8-bit integers.
//
// A group of values v with the largest magnitude a:
//   scale = a / 127,  code = rint(v (127 / a))  (ties to even),  value = code * scale
// each quotient and product one correctly rounded fp32 operation, so the codes
// are defined bit for bit.  |v (127 / a)| rounds to 127 at most.  A group whose a
// is below 2^-100 (where 127 / a would leave fp32) has scale 0 and codes 0; a
// group with an infinity or a NaN has that as its scale, so that it comes back
// as NaN rather than as a number (whatever its codes: those next to a NaN are the
// low byte of its payload).  A group whose a is the largest fp32 number comes back with an
// infinity in a's place: a / 127 is rounded up.
#pragma once

#include "rows.h"

namespace moe {
namespace rows_i8 {

constexpr int kCols = 16;  // columns of a lane

// A lane's 16 values; chunks of 16 bytes, two of bf16 or four of fp32.
template <bool BF16>
__device__ __forceinline__ void load16(const void* base, size_t elem, float (&v)[kCols]) {
  using R = Row<BF16>;
#pragma unroll
  for (int i = 0; i < kCols / R::N; ++i) R::to_f32(R::ld_s(base, elem + i * R::N), v + i * R::N);
}

// The largest magnitude, as bits: the order of the magnitudes of floats is that
// of their bits, and NaN is above infinity.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[kCols], uint32_t top) {
#pragma unroll
  for (int i = 0; i < kCols; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}

struct Scale {
  float inv, scale;
  __device__ explicit Scale(uint32_t bits) {
    const float a = __uint_as_float(bits);
    const bool none = a < 0x1p-100f;  // (false for NaN)
    inv = none ? 0.f : 127.f / a;
    scale = none ? 0.f : a / 127.f;
  }
};

// Codes of four values: adding 1.5 * 2^23 rounds a product within +-127 to the
// nearest whole number, ties to even, and leaves it in the low byte; an infinity
// times 0 leaves 0 there.  The product is rounded by itself.
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = v[i] * inv;
    b[i] = __float_as_uint(p + 12582912.f);
  }
  // v_perm: selector 0..3 a byte of the second operand, 4..7 of the first, 12 zero
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return lo | hi;
}

__device__ __forceinline__ u32x4_t codes16(const float (&v)[kCols], float inv) {
  return u32x4_t{codes4(v, inv), codes4(v + 4, inv), codes4(v + 8, inv), codes4(v + 12, inv)};
}

}  // namespace rows_i8
}  // namespace moe
