// Combine with dropout and the residual, and its backward, for gfx950.
//
//   y[t,h] = r[t,h] + m[t,h] sum_j w[t,j] y_perm[dest[t,j],h],  m = keep / (1 - p)
// keep[t,h] is a comparison of one 32-bit word of a counter-based generator,
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy
// as 1, 2, 3; 2011): element i = t H + h is word i % 4 at counter
// (i / 4, offset) under the key seed, and is kept when the word is at least
// floor(p 2^32).  The backward computes the same words again, so no mask is
// stored, and the result does not depend on the launch shape.
#include "rows.h"

namespace moe {

namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t counter, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// Bit i: element elem + i of the N elements of one 16-byte chunk is kept
// (elem % 4 == 0: H is a multiple of the chunk).
template <int N>
__device__ __forceinline__ uint32_t keep_bits(uint64_t elem, uint64_t offset, uint64_t seed,
                                              uint32_t thr) {
  uint32_t bits = 0;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const Words r = philox(elem / 4 + q, offset, seed);
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= (uint32_t)(r.w[i] >= thr) << (4 * q + i);
  }
  return bits;
}

// The same as a mask over the chunk's bits.
template <bool BF16>
__device__ __forceinline__ u32x4_t keep_mask(uint32_t bits) {
  u32x4_t m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)
      m[i] = ((bits >> (2 * i) & 1) ? 0xffffu : 0u) | ((bits >> (2 * i + 1) & 1) ? 0xffff0000u : 0u);
    else
      m[i] = (bits >> i & 1) ? 0xffffffffu : 0u;
  }
  return m;
}

template <bool BF16, int CU, int SG>
__global__ __launch_bounds__(256) void combine_dropout_kernel(
    const void* __restrict__ y_perm, const float* __restrict__ topk_w,
    const int32_t* __restrict__ dest_row, const void* residual,
    const uint64_t* __restrict__ rng, uint32_t thr, float scale, int T, int H, int k, void* y) {
  using R = Row<BF16>;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = lane_id();
  const uint64_t seed = rng[0], offset = rng[1];
  int d = -1;
  float w = 1.f;
  if (lane < k) {
    d = dest_row[(size_t)t * k + lane];
    if (topk_w != nullptr) w = topk_w[(size_t)t * k + lane];
  }
  int dc, jc;
  float wc;
  const int n = pack_slots(d, w, dc, wc, jc);
  const int nch = H / R::N;
  for (int c0 = 0; c0 < nch; c0 += kWave * CU) {
    float acc[CU][R::N];
    u32x4_t res[CU];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int c = c0 + u * kWave + lane;
      res[u] = residual != nullptr && c < nch ? R::ld_s(residual, (size_t)t * H + (size_t)c * R::N)
                                              : u32x4_t{};
#pragma unroll
      for (int i = 0; i < R::N; ++i) acc[u][i] = 0.f;
    }
    gather_rows<BF16, true, CU, SG>(y_perm, H, nch, c0, n, dc, wc, acc);
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int c = c0 + u * kWave + lane;
      if (c0 + u * kWave >= nch) break;  // the whole wave
      if (c >= nch) continue;
      const size_t e = (size_t)t * H + (size_t)c * R::N;
      const uint32_t keep = n > 0 ? keep_bits<R::N>(e, offset, seed, thr) : 0;
      float r[R::N];
      R::to_f32(res[u], r);
#pragma unroll
      for (int i = 0; i < R::N; ++i) r[i] += (keep >> i & 1) ? scale * acc[u][i] : 0.f;
      R::st_s(y, e, R::from_f32(r));
    }
  }
}

// g = keep / (1 - p) dy;  dy_perm[dest_j] = w_j g[t];  d_topk_w[t,j] = <g[t], y_perm[dest_j]>
template <bool BF16, int CU, int SG>
__global__ __launch_bounds__(256) void combine_dropout_bwd_kernel(
    const void* __restrict__ dy, const void* __restrict__ y_perm, const float* __restrict__ topk_w,
    const int32_t* __restrict__ dest_row, const uint64_t* __restrict__ rng, uint32_t thr,
    float scale, int T, int H, int k, void* __restrict__ dy_perm, float* __restrict__ d_topk_w) {
  using R = Row<BF16>;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = lane_id();
  const uint64_t seed = rng[0], offset = rng[1];
  int d = -1;
  float w = 0.f;
  if (lane < k) {
    d = dest_row[(size_t)t * k + lane];
    w = topk_w[(size_t)t * k + lane];
    if (d < 0) d_topk_w[(size_t)t * k + lane] = 0.f;
  }
  int dc, jc;
  float wc;
  const int n = pack_slots(d, w, dc, wc, jc);
  const int nch = H / R::N;
  // this lane's kept elements, for the slots after the first ones (rows of up
  // to 64 elements a lane; longer ones compute them again)
  const bool keeps = nch <= kWave * (64 / R::N);
  uint64_t kept = 0;
  for (int j0 = 0; j0 < n; j0 += SG) {
    int dj[SG];
    float wj[SG], dot[SG];
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      dj[s] = __shfl(dc, j0 + s, kWave);
      wj[s] = __shfl(wc, j0 + s, kWave);
      dot[s] = 0.f;
    }
    for (int c0 = 0; c0 < nch; c0 += kWave * CU) {
      u32x4_t g[CU], raw[SG][CU];
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        const int c = c0 + u * kWave + lane;
        g[u] = c < nch ? R::ld_s(dy, (size_t)t * H + (size_t)c * R::N) : u32x4_t{};
#pragma unroll
        for (int s = 0; s < SG; ++s)
          raw[s][u] = (j0 + s < n && c < nch) ? R::ld_s(y_perm, (size_t)dj[s] * H + (size_t)c * R::N)
                                              : u32x4_t{};
      }
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        const int c = c0 + u * kWave + lane;
        if (c0 + u * kWave >= nch) break;  // the whole wave
        const int at = (c0 / kWave + u) * R::N;
        uint32_t bits;
        if (j0 == 0 || !keeps) {
          bits = keep_bits<R::N>((size_t)t * H + (size_t)c * R::N, offset, seed, thr);
          if (keeps) kept |= (uint64_t)bits << at;
        } else {
          bits = (uint32_t)(kept >> at);
        }
        // dropped elements leave both factors, so an infinity there is no NaN
        const u32x4_t m = keep_mask<BF16>(bits);
        float gf[R::N];
        R::to_f32(g[u] & m, gf);
#pragma unroll
        for (int i = 0; i < R::N; ++i) gf[i] *= scale;
#pragma unroll
        for (int s = 0; s < SG; ++s) {
          float v[R::N], o[R::N];
          R::to_f32(raw[s][u] & m, v);
#pragma unroll
          for (int i = 0; i < R::N; ++i) {
            dot[s] = fmaf(gf[i], v[i], dot[s]);
            o[i] = wj[s] * gf[i];
          }
          if (j0 + s < n && c < nch) R::st_s(dy_perm, (size_t)dj[s] * H + (size_t)c * R::N, R::from_f32(o));
        }
      }
    }
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      const float sum = wave_sum(dot[s]);
      const int js = __shfl(jc, j0 + s, kWave);
      if (lane == 0 && j0 + s < n) d_topk_w[(size_t)t * k + js] = sum;
    }
  }
}

// floor(p 2^32) and 1 / (1 - p), for 0 <= p < 1
struct Drop {
  uint32_t thr;
  float scale;
};
Drop drop_of(double p) { return {(uint32_t)(p * 4294967296.0), (float)(1.0 / (1.0 - p))}; }

}  // namespace

hipError_t launch_combine_dropout(const void* y_perm, const float* topk_w, const int32_t* dest_row,
                                  const void* residual, double p, const uint64_t* rng, int T, int H,
                                  int k, bool bf16, void* y, hipStream_t s) {
  const Drop d = drop_of(p);
  const int blocks = (T + 3) / 4;
  ProfScope ps(MOE_KERNEL_COMBINE_DROPOUT, s);
  // Two slots' rows in flight; four chunks of each for long rows (16384 tokens
  // of 2048, top-8: 112 us, 124 with two), two for short ones, whose chunks do
  // not fill four (of 512: 28 us, 33 with four).
#define MOE_DF(B, CU) \
  combine_dropout_kernel<B, CU, 2><<<blocks, 256, 0, s>>>(y_perm, topk_w, dest_row, residual, rng, d.thr, d.scale, T, H, k, y)
  if (bf16) {
    if (H > 2 * kWave * 8) MOE_DF(true, 4); else MOE_DF(true, 2);
  } else {
    if (H > 2 * kWave * 4) MOE_DF(false, 4); else MOE_DF(false, 2);
  }
#undef MOE_DF
  return hipGetLastError();
}

hipError_t launch_combine_dropout_bwd(const void* dy, const void* y_perm, const float* topk_w,
                                      const int32_t* dest_row, double p, const uint64_t* rng, int T,
                                      int H, int k, bool bf16, void* dy_perm, float* d_topk_w,
                                      hipStream_t s) {
  const Drop d = drop_of(p);
  const int blocks = (T + 3) / 4;
  ProfScope ps(MOE_KERNEL_COMBINE_DROPOUT_BWD, s);
  // Four slots, two chunks of each: enough in flight with more waves on a CU
  // than four chunks allow (8192 tokens with one local slot: 22 us for 24).
  if (bf16)
    combine_dropout_bwd_kernel<true, 2, 4><<<blocks, 256, 0, s>>>(
        dy, y_perm, topk_w, dest_row, rng, d.thr, d.scale, T, H, k, dy_perm, d_topk_w);
  else
    combine_dropout_bwd_kernel<false, 2, 4><<<blocks, 256, 0, s>>>(
        dy, y_perm, topk_w, dest_row, rng, d.thr, d.scale, T, H, k, dy_perm, d_topk_w);
  return hipGetLastError();
}

}  // namespace moe
