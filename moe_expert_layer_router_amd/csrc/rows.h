// Rows of 16-byte chunks and the per-token gather-reduce that the combine
// kernels share (one wave per token).
#pragma once

#include "common.h"

namespace moe {

// 16 bytes of a row: 8 bf16 or 4 fp32 elements, held as a native vector.
template <bool BF16>
struct Row {
  static constexpr int N = BF16 ? 8 : 4;
  static constexpr int EB = BF16 ? 2 : 4;
  __device__ static u32x4_t ld(const void* base, size_t elem) {
    return *reinterpret_cast<const u32x4_t*>((const char*)base + elem * EB);
  }
  __device__ static void st(void* base, size_t elem, u32x4_t v) {
    *reinterpret_cast<u32x4_t*>((char*)base + elem * EB) = v;
  }
  // Streaming (non-temporal) forms for rows touched once per call: grouped
  // rows, token rows and the outputs.  They keep the caches for what is
  // re-read (the router weight rows); on the full 128-expert layer they raise
  // the combine from 0.64 to 0.76 of HBM.
  __device__ static u32x4_t ld_s(const void* base, size_t elem) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>((const char*)base + elem * EB));
  }
  __device__ static void st_s(void* base, size_t elem, u32x4_t v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>((char*)base + elem * EB));
  }
  __device__ static void to_f32(u32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(v[i]);
      }
    }
  }
  __device__ static u32x4_t from_f32(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = BF16 ? pack_bf2(f[2 * i], f[2 * i + 1]) : __float_as_uint(f[i]);
    return v;
  }
};

// Chunks of 16 bytes per lane per pass and slots whose rows are loaded
// together: all CU x SG row loads of a pass are in flight at once.  Eight
// slots (a top-8 token in one round trip) double the load registers and halve
// the waves per SIMD, which costs more on an EP share (about one local slot
// per token) than it gains on the full layer.
constexpr int kCU = 4;
constexpr int kSG = 4;

// Moves the lanes holding a local slot (d >= 0; lanes >= k hold d = -1) to
// lanes 0..n-1, keeping slot order; returns n.  Lane i then holds that slot's
// row d, weight w and slot index j.  Lanes without a slot all send to lane
// 63, which is never read (n <= k <= 32).
__device__ __forceinline__ int pack_slots(int d, float w, int& dc, float& wc, int& jc) {
  const int lane = lane_id();
  const uint64_t m = __ballot(d >= 0);
  const int rank = __popcll(m & ((1ull << lane) - 1ull));
  const int to = (d >= 0 ? rank : 63) << 2;
  dc = __builtin_amdgcn_ds_permute(to, d);
  wc = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(w)));
  jc = __builtin_amdgcn_ds_permute(to, lane);
  return __popcll(m);
}

// out[c] = sum over packed slots j < n (ascending) of wc_j * rows[dc_j][c] for
// this lane's chunks c0 + u * 64 + lane; fp32 accumulation.  STREAM: the rows
// are read once (streaming loads).  n <= 64: groups of SG slots that divide the
// wave never ask a lane behind its last.
template <bool BF16, bool STREAM, int CU = kCU, int SG = kSG>
__device__ __forceinline__ void gather_rows(const void* __restrict__ rows, int H, int nch, int c0,
                                            int n, int dc, float wc,
                                            float (&acc)[CU][Row<BF16>::N]) {
  using R = Row<BF16>;
  static_assert(kWave % SG == 0, "a group of slots ends inside the wave");
  const int lane = lane_id();
  for (int j0 = 0; j0 < n; j0 += SG) {
    u32x4_t raw[SG][CU];
    float wj[SG];
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      const int j = j0 + s;  // < 64: a valid lane index
      const int dj = __shfl(dc, j, kWave);
      wj[s] = (j < n) ? __shfl(wc, j, kWave) : 0.f;
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        const int c = c0 + u * kWave + lane;
        const size_t e = (size_t)dj * H + (size_t)c * R::N;
        raw[s][u] = (j < n && c < nch) ? (STREAM ? R::ld_s(rows, e) : R::ld(rows, e)) : u32x4_t{};
      }
    }
#pragma unroll
    for (int s = 0; s < SG; ++s)
#pragma unroll
      for (int u = 0; u < CU; ++u) {
        float v[R::N];
        R::to_f32(raw[s][u], v);
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[u][i] = fmaf(wj[s], v[i], acc[u][i]);
      }
  }
}

}  // namespace moe
