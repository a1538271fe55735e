// Rows as 8-bit integers with scales, for gfx950: operands of the int8 products
// (one scale a row) and activation checkpoints (one scale a group of columns).
//
// All kernels move their operands once; a lane quantizes 16 columns, whose codes
// are one 16-byte store, and restores as many as fill one.  Bound by the memory: the
// gate and up of 131072 rows, 2 x 768 bf16 columns in groups of 128, quantized in 101
// us (6.1 TB/s moved), restored together with h in 135 us (6.0 TB/s).
#include "rows_i8.h"

namespace moe {

namespace {

using namespace rows_i8;

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
// every second 16 bytes to the next: 324 us for 135 with the restored gate and up of
// 131072 rows.)
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
