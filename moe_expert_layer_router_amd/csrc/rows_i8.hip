// Rows as 8-bit integers with scales, for gfx950: operands of the int8 products
// (one scale a row) and activation checkpoints (one scale a group of columns).
//
// A group of values v with the largest magnitude a:
//   scale = a / 127,  code = rint(v (127 / a))  (ties to even),  value = code * scale
// each quotient and product one correctly rounded fp32 operation, so the codes
// are defined bit for bit.  |v (127 / a)| rounds to 127 at most.  A group whose a
// is below 2^-100 (where 127 / a would leave fp32) has scale 0 and codes 0; a
// group with an infinity or a NaN has that as its scale, so that it comes back
// as NaN rather than as a number.
//
// All kernels move their operands once; a lane quantizes 16 columns, whose codes
// are one 16-byte store, and restores as many as fill one.
#include "rows.h"

namespace moe {

namespace {

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
// nearest whole number, ties to even, and leaves it in the low byte; NaN
// (an infinity times 0) leaves 0 there.  The product is rounded by itself.
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

// Groups of G columns, 32 <= G <= 512 a power of two: G / 16 neighbouring lanes.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_groups_i8_kernel(const void* __restrict__ src, int rows,
                                                                 int cols, int lanes,
                                                                 const int32_t* __restrict__ nrows,
                                                                 int8_t* __restrict__ q,
                                                                 float* __restrict__ scale) {
  const int per_row = cols / kCols;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;  // chunk of 16 columns (below 2^32 in all)
  const uint32_t row = i / (uint32_t)per_row;
  if (row >= (uint32_t)rows || (nrows != nullptr && (int)row >= *nrows)) return;  // whole groups
  float v[kCols];
  load16<BF16>(src, (size_t)i * kCols, v);
  uint32_t top = top_bits(v, 0);
  for (int o = 1; o < lanes; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, kWave));
  const Scale s(top);
  __builtin_nontemporal_store(codes16(v, s.inv), reinterpret_cast<u32x4_t*>(q) + i);
  if (i % (uint32_t)lanes == 0) scale[i / (uint32_t)lanes] = s.scale;
}

// One scale a row, a wave for each row; rows of up to 64 * 16 * NC columns stay in
// registers, longer ones (NC = 0) are read twice.
template <bool BF16, int NC>
__global__ __launch_bounds__(256) void quantize_rows_i8_kernel(const void* __restrict__ src, int rows,
                                                               int cols, const int32_t* __restrict__ nrows,
                                                               int8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = lane_id();
  if (row >= rows || (nrows != nullptr && row >= *nrows)) return;
  const int per_row = cols / kCols;
  const size_t base = (size_t)row * cols;
  float v[NC == 0 ? 1 : NC][kCols];
  uint32_t top = 0;
  if constexpr (NC == 0) {
    for (int c = lane; c < per_row; c += kWave) {
      load16<BF16>(src, base + (size_t)c * kCols, v[0]);
      top = top_bits(v[0], top);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = lane + kWave * j;
      if (c < per_row) {
        load16<BF16>(src, base + (size_t)c * kCols, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) top = top_bits(v[j], top);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, kWave));
  const Scale s(top);
  if (lane == 0) scale[row] = s.scale;
  u32x4_t* out = reinterpret_cast<u32x4_t*>(q + base);
  if constexpr (NC == 0) {
    for (int c = lane; c < per_row; c += kWave) {
      load16<BF16>(src, base + (size_t)c * kCols, v[0]);
      out[c] = codes16(v[0], s.inv);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (lane + kWave * j < per_row) out[lane + kWave * j] = codes16(v[j], s.inv);
  }
}

// The codes of the columns whose values fill 16 bytes, so that a wave's stores
// are one run: 8 of bf16, 4 of fp32.  (With 16 columns a lane each store leaves
// every second 16 bytes to the next: 324 us for the gate and up of 131072 rows.)
template <bool BF16>
__device__ __forceinline__ void values(const int8_t* q, float scale, float (&v)[Row<BF16>::N]) {
  uint32_t w[Row<BF16>::N / 4];
  if constexpr (BF16) {
    const uint2 t = *reinterpret_cast<const uint2*>(q);
    w[0] = t.x;
    w[1] = t.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(q);
  }
#pragma unroll
  for (int i = 0; i < Row<BF16>::N; ++i) v[i] = (float)((int)(w[i / 4] << (24 - 8 * (i % 4))) >> 24) * scale;
}

// out[r] = values of code row src_row[r] (or r); 0 where src_row[r] names none.
template <bool BF16>
__global__ __launch_bounds__(256) void dequantize_i8_kernel(const int8_t* __restrict__ q,
                                                            const float* __restrict__ scale,
                                                            const int32_t* __restrict__ src_row, int rows,
                                                            int src_rows, int cols, int group,
                                                            const int32_t* __restrict__ nrows,
                                                            void* __restrict__ out) {
  using R = Row<BF16>;
  const uint32_t per_row = (uint32_t)cols / R::N;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = i / per_row, c = i % per_row;
  if (row >= (uint32_t)rows || (nrows != nullptr && (int)row >= *nrows)) return;
  const int from = src_row != nullptr ? src_row[row] : (int)row;
  float v[R::N] = {};
  if (from >= 0 && from < src_rows)
    values<BF16>(q + (size_t)from * cols + c * R::N,
                 scale[(size_t)from * (uint32_t)(cols / group) + c / (uint32_t)(group / R::N)], v);
  R::st_s(out, (size_t)i * R::N, R::from_f32(v));
}

// g and u from the codes of [g | u], and h = SiLU(g) u of the values as stored:
// what the backward reads of a forward whose gu and h were not kept.
template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_restore_i8_kernel(const int8_t* __restrict__ q,
                                                                const float* __restrict__ scale, int rows,
                                                                int I, int group,
                                                                const int32_t* __restrict__ nrows,
                                                                void* __restrict__ gu,
                                                                void* __restrict__ h) {
  using R = Row<BF16>;
  const uint32_t half = (uint32_t)I / R::N, per_group = (uint32_t)(group / R::N);
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = i / half, c = i % half;
  if (row >= (uint32_t)rows || (nrows != nullptr && (int)row >= *nrows)) return;
  const size_t e = (size_t)row * 2 * I + (size_t)c * R::N;
  const float* sr = scale + (size_t)row * (uint32_t)(2 * I / group);
  float g[R::N], u[R::N], o[R::N];
  values<BF16>(q + e, sr[c / per_group], g);
  values<BF16>(q + e + I, sr[(half + c) / per_group], u);
  const u32x4_t pg = R::from_f32(g), pu = R::from_f32(u);
  R::st_s(gu, e, pg);
  R::st_s(gu, e + I, pu);
  R::to_f32(pg, g);
  R::to_f32(pu, u);
#pragma unroll
  for (int n = 0; n < R::N; ++n) o[n] = g[n] * fast_rcp(1.f + __expf(-g[n])) * u[n];
  R::st_s(h, (size_t)i * R::N, R::from_f32(o));
}

// Workgroups of a launch with a thread for every `per` columns.
unsigned blocks_of(int rows, int cols, int per) {
  return (unsigned)(((uint64_t)rows * (uint64_t)(cols / per) + 255) / 256);
}

}  // namespace

uint64_t rows_i8_threads(int rows, int cols, int per) {
  return ((uint64_t)rows * (uint64_t)(cols / per) + 255) / 256 * 256;
}

hipError_t launch_quantize_i8(const void* src, int rows, int cols, int group, bool bf16,
                              const int32_t* nrows, int8_t* q, float* scale, hipStream_t s) {
  ProfScope ps(MOE_KERNEL_QUANTIZE_I8, s);
  if (group < cols) {
    const unsigned blocks = blocks_of(rows, cols, kCols);
    if (bf16)
      quantize_groups_i8_kernel<true><<<blocks, 256, 0, s>>>(src, rows, cols, group / kCols, nrows, q, scale);
    else
      quantize_groups_i8_kernel<false><<<blocks, 256, 0, s>>>(src, rows, cols, group / kCols, nrows, q, scale);
    return hipGetLastError();
  }
  const int blocks = (rows + 3) / 4, most = kWave * kCols;
#define MOE_Q(B, NC) quantize_rows_i8_kernel<B, NC><<<blocks, 256, 0, s>>>(src, rows, cols, nrows, q, scale)
#define MOE_QB(B) \
  if (cols <= most) MOE_Q(B, 1); else if (cols <= 2 * most) MOE_Q(B, 2); else if (cols <= 4 * most) MOE_Q(B, 4); else MOE_Q(B, 0)
  if (bf16) { MOE_QB(true); } else { MOE_QB(false); }
#undef MOE_QB
#undef MOE_Q
  return hipGetLastError();
}

hipError_t launch_dequantize_i8(const int8_t* q, const float* scale, const int32_t* src_row, int rows,
                                int src_rows, int cols, int group, bool bf16, const int32_t* nrows,
                                void* out, hipStream_t s) {
  const unsigned blocks = blocks_of(rows, cols, bf16 ? 8 : 4);
  if (bf16)
    dequantize_i8_kernel<true><<<blocks, 256, 0, s>>>(q, scale, src_row, rows, src_rows, cols, group, nrows, out);
  else
    dequantize_i8_kernel<false><<<blocks, 256, 0, s>>>(q, scale, src_row, rows, src_rows, cols, group, nrows, out);
  return hipGetLastError();
}

hipError_t launch_swiglu_restore_i8(const int8_t* q, const float* scale, int rows, int I, int group, bool bf16,
                                    const int32_t* nrows, void* gu, void* h, hipStream_t s) {
  ProfScope ps(MOE_KERNEL_RESTORE_I8, s);
  const unsigned blocks = blocks_of(rows, I, bf16 ? 8 : 4);
  if (bf16)
    swiglu_restore_i8_kernel<true><<<blocks, 256, 0, s>>>(q, scale, rows, I, group, nrows, gu, h);
  else
    swiglu_restore_i8_kernel<false><<<blocks, 256, 0, s>>>(q, scale, rows, I, group, nrows, gu, h);
  return hipGetLastError();
}

}  // namespace moe
