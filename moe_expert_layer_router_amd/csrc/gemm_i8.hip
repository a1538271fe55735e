// Products of int8 rows with int8 expert weights, grouped by expert, for gfx950:
//   y[r,n] = xs[src r] ws[e,n] sum_k x[src r,k] w[e,n,k],  rows r of expert e,
// and the SwiGLU pair of them, h[r,n] = SiLU(g) u with the gate's and the up
// weight's products.  The sums are whole numbers, exact in the matrix core's
// int32, so every variant and every split of K gives the same bits; the two
// scales are applied in fp32 and the result is rounded once.
//
// Two kernels share the experts out by their number of rows, which only the
// device knows:
//   few rows (skinny_i8_kernel): bound by the read of the weights.  A workgroup
//     owns 32 columns of one expert; its four waves split K and take the weights
//     straight from memory into MFMA operands, each byte once for up to 64 rows,
//     and add their sums through LDS.
//   many rows (tile_i8_kernel): bound by the matrix cores and what feeds them.
//     Tiles of 256 rows x 128 weight rows in a workgroup of four waves, operands
//     through a ring of LDS stages filled by DMA, two workgroups on a CU so that
//     one's epilogue, barriers and first loads lie under the other's products.
// Weights are the first operand of the MFMA, so that a lane's results are
// neighbouring columns of one row; which weight row takes which place in the
// operand is chosen so that they are 16 or 32 in a run.
#include <algorithm>

#include "common.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float swiglu(float g, float u) { return g * fast_rcp(1.f + __expf(-g)) * u; }

// Operands of one product or of the gate and up pair (w1, s1 of the up weight).
struct ProductI8 {
  const int8_t* x;
  const float* xs;
  const int32_t* src;  // row r is x[src[r]]; null: x[r]
  int x_rows;
  const int32_t* offsets;
  int E_l, K, N;
  const int8_t *w0, *w1;
  const float *s0, *s1;
  bf16_t* out;  // [rows][N]
};

__device__ __forceinline__ int source_row(const ProductI8& p, int r) {
  const int x = p.src != nullptr ? p.src[r] : r;
  return min(max(x, 0), p.x_rows - 1);
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int kFew = 64;  // rows of one pass over an expert's weights

// The i-th expert that has between 1 and `most` rows; false if there are fewer.
__device__ __forceinline__ bool nth_expert(const int32_t* __restrict__ offsets, int E_l, int i, int most,
                                           int& e, int& lo, int& hi) {
  const int lane = lane_id();
  for (int e0 = 0; e0 < E_l; e0 += kWave) {
    const int at = min(e0 + lane, E_l - 1);
    const int a = offsets[at], b = offsets[at + 1];
    const bool has = e0 + lane < E_l && b > a && b - a <= most;
    const uint64_t m = __ballot(has);
    const int n = __popcll(m);
    if (i < n) {
      const uint64_t mine = __ballot(has && __popcll(m & ((1ull << lane) - 1ull)) == i);
      const int l = __ffsll((unsigned long long)mine) - 1;
      e = e0 + l;
      lo = __builtin_amdgcn_readlane(a, l);
      hi = __builtin_amdgcn_readlane(b, l);
      return true;
    }
    i -= n;
  }
  return false;
}

// NB blocks of 16 rows from row r0 on.  Columns: GU: 16 of gate and the same of
// up; else 32, a lane's 4 + 4 in a run of 8.
template <bool GU, int NB>
__device__ __forceinline__ void skinny_rows(const ProductI8& p, int e, int n0, int r0, int hi,
                                            i32x4_t (*red)[2 * 4][kWave]) {
  constexpr int U = NB == 1 ? 8 : 4;  // K steps of 64 in flight
  const int lane = lane_id(), wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int steps = (p.K + 63) / 64;
  const int8_t* wr[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int n = GU ? n0 + l16 : n0 + (l16 >> 2) * 8 + b * 4 + (l16 & 3);
    wr[b] = (GU && b == 1 ? p.w1 : p.w0) + ((size_t)e * p.N + min(n, p.N - 1)) * p.K + g * 16;
  }
  const int8_t* xr[NB];
#pragma unroll
  for (int m = 0; m < NB; ++m)
    xr[m] = p.x + (size_t)source_row(p, min(r0 + m * 16 + l16, hi - 1)) * p.K + g * 16;
  i32x4_t acc[2][NB] = {};
  for (int s0 = wave; s0 < steps; s0 += 4 * U) {
    i32x4_t a[U][2], b[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + 4 * u) * 64;
      const bool in = k + g * 16 < p.K;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[u][i] = in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(wr[i] + k)) : i32x4_t{};
#pragma unroll
      for (int m = 0; m < NB; ++m)
        b[u][m] = in ? *reinterpret_cast<const i32x4_t*>(xr[m] + k) : i32x4_t{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < NB; ++m)
          acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][i], b[u][m], acc[i][m], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < NB; ++m) red[wave][i * NB + m][lane] = acc[i][m];
  __syncthreads();
  if (wave < NB) {
    i32x4_t sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = red[0][i * NB + wave][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum[i] += red[w][i * NB + wave][lane];
    }
    const int r = r0 + wave * 16 + l16;
    if (r < hi) {
      const float xs = p.xs[source_row(p, r)];
      if constexpr (GU) {
        const int n = n0 + g * 4;
        if (n < p.N) {
          const f32x4_t sg = *reinterpret_cast<const f32x4_t*>(p.s0 + (size_t)e * p.N + n);
          const f32x4_t su = *reinterpret_cast<const f32x4_t*>(p.s1 + (size_t)e * p.N + n);
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = swiglu((float)sum[0][i] * xs * sg[i], (float)sum[1][i] * xs * su[i]);
          *reinterpret_cast<uint2*>(p.out + (size_t)r * p.N + n) =
              make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
        }
      } else {
        const int n = n0 + g * 8;
        if (n < p.N) {
          const f32x4_t* ws = reinterpret_cast<const f32x4_t*>(p.s0 + (size_t)e * p.N + n);
          const f32x4_t wa = ws[0], wb = ws[1];
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i] = (float)sum[0][i] * xs * wa[i];
            o[4 + i] = (float)sum[1][i] * xs * wb[i];
          }
          *reinterpret_cast<uint4*>(p.out + (size_t)r * p.N + n) = pack8(o);
        }
      }
    }
  }
}

template <bool GU>
__global__ __launch_bounds__(256) void skinny_i8_kernel(ProductI8 p, int most) {
  __shared__ i32x4_t red[4][2 * 4][kWave];
  int e, lo, hi;
  if (!nth_expert(p.offsets, p.E_l, (int)blockIdx.y, most, e, lo, hi)) return;
  const int n0 = (int)blockIdx.x * (GU ? 16 : 32);
  for (int r0 = lo; r0 < hi; r0 += kFew) {
    if (r0 > lo) __syncthreads();  // the last sums have been read
    const int left = hi - r0;
    if (left <= 16) skinny_rows<GU, 1>(p, e, n0, r0, hi, red);
    else if (left <= 32) skinny_rows<GU, 2>(p, e, n0, r0, hi, red);
    else skinny_rows<GU, 4>(p, e, n0, r0, hi, red);
  }
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kTileM = 256;   // rows of a tile
constexpr int kTileW = 128;   // weight rows of a tile (64 of gate and 64 of up in the pair)
constexpr int kStageK = 64;   // bytes of K a stage
constexpr int kStages = 3;
constexpr int kStageBytes = (kTileM + kTileW) * kStageK;
constexpr int kDmas = kStageBytes / 1024 / 4;  // of a wave, a stage: 2 of weights, 4 of rows

__device__ __forceinline__ uint32_t lds_byte_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)p);
}

// Chunks of 16 bytes of a 64-byte LDS row are stored at place c ^ swizzle(row),
// so that the eight neighbouring lanes of an operand read (eight rows in the
// order of the operand) touch eight different places of 128 bytes.
__device__ __forceinline__ int swizzle_row(int row) { return (row >> 1) & 3; }
template <bool GU>
__device__ __forceinline__ int swizzle_w(int row) {
  return ((row >> 1) & 1) | (((row >> (GU ? 4 : 5)) & 1) << 1);
}

template <bool GU>
struct Tile {
  const ProductI8& p;
  char* lds;
  int e, n0, r0, rows;  // rows of this tile, 1..256
  uint32_t wv[2], xv[4];  // byte offsets of this lane's DMA chunks at K = 0
  rsrc_t wd[2], xd;
  int chunk[2], xchunk[4];  // 16-byte chunk of the stage that each DMA takes
  uint32_t lds0;

  __device__ Tile(const ProductI8& p_, char* lds_, int e_, int n0_, int r0_, int rows_)
      : p(p_), lds(lds_), e(e_), n0(n0_), r0(r0_), rows(rows_) {
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wbytes = (uint32_t)p.N * (uint32_t)p.K;
    lds0 = lds_byte_addr(lds);
    // weights: DMA i of a wave fills LDS rows i * 64 + wave * 16 + lane / 4
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = i * 64 + wave * 16 + (lane >> 2);
      const int n = GU ? n0 + (row & 63) : n0 + row;
      const int8_t* base = (GU && i == 1 ? p.w1 : p.w0) + (size_t)e * p.N * p.K;
      wd[i] = make_rsrc(base, wbytes);
      chunk[i] = (lane & 3) ^ swizzle_w<GU>(row);
      wv[i] = n < p.N ? (uint32_t)n * (uint32_t)p.K + chunk[i] * 16 : kDmaKill;
    }
    xd = make_rsrc(p.x, (uint32_t)p.x_rows * (uint32_t)p.K);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 64 + wave * 16 + (lane >> 2);
      xchunk[i] = (lane & 3) ^ swizzle_row(row);
      xv[i] = row < rows ? (uint32_t)source_row(p, r0 + row) * (uint32_t)p.K + xchunk[i] * 16 : kDmaKill;
    }
  }

  // K step s into its ring stage; chunks past K (and whole steps past the last)
  // are dropped and leave zeros.
  __device__ __forceinline__ void issue(int s, int stage) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = s * kStageK;
    const uint32_t to = lds0 + stage * kStageBytes + wave * 1024;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = k + chunk[i] * 16 < p.K && wv[i] != kDmaKill;
      dma16(wd[i], in ? wv[i] + k : kDmaKill, to + i * 4096);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = k + xchunk[i] * 16 < p.K && xv[i] != kDmaKill;
      dma16(xd, in ? xv[i] + k : kDmaKill, to + kTileW * kStageK + i * 4096);
    }
  }

  // The products of a wave's 64 weight rows with NB blocks of 32 rows.
  template <int NB>
  __device__ __forceinline__ void run(int wm, int wn) const {
    const int lane = lane_id(), half = lane >> 5, l = lane & 31;
    const int a = l >> 3, h = (l >> 2) & 1, j = l & 3;
    const int wrow = GU ? wn * 32 + h * 16 + 4 * a + j : wn * 64 + h * 32 + 4 * a + j;
    constexpr int kBlk = (GU ? 64 : 16) * kStageK;  // from the first block of 32 weight rows to the second
    int aw[2], ax[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      aw[ks] = wrow * kStageK + (((ks * 2 + half) ^ swizzle_w<GU>(wrow)) * 16);
      ax[ks] = kTileW * kStageK + (wm * 128 + l) * kStageK + (((ks * 2 + half) ^ swizzle_row(l)) * 16);
    }
    i32x16_t acc[2][NB == 0 ? 1 : NB];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][m][i] = 0;
    const int steps = (p.K + kStageK - 1) / kStageK;
    issue(0, 0);
    issue(1, 1);
    int stage = 0;
    for (int s = 0; s < steps; ++s) {
      wait_vm<kDmas>();  // this wave's part of step s (step s + 1 may be on its way)
      lds_barrier();     // everybody's, and everybody has read step s - 1
      issue(s + 2, stage >= 1 ? stage - 1 : kStages - 1);
      const char* at = lds + stage * kStageBytes;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (NB > 0) {
          i32x4_t fa[2], fx[NB];
#pragma unroll
          for (int b = 0; b < 2; ++b) fa[b] = *reinterpret_cast<const i32x4_t*>(at + aw[ks] + b * kBlk);
#pragma unroll
          for (int m = 0; m < NB; ++m)
            fx[m] = *reinterpret_cast<const i32x4_t*>(at + ax[ks] + m * 32 * kStageK);
#pragma unroll
          for (int m = 0; m < NB; ++m)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              acc[b][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[b], fx[m], acc[b][m], 0, 0, 0);
        }
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    wait_vm<0>();  // the dropped steps' DMAs, before the LDS can be another workgroup's
    if constexpr (NB > 0) store<NB>(acc, wm, wn, half, l);
  }

  template <int NB>
  __device__ __forceinline__ void store(const i32x16_t (&acc)[2][NB], int wm, int wn, int half, int l) const {
    const int n = GU ? n0 + wn * 32 + half * 16 : n0 + wn * 64 + half * 32;
    f32x4_t ws[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float* s = (GU && b == 1 ? p.s1 : p.s0) + (size_t)e * p.N;
      const int c = GU ? n : n + b * 16;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ws[b][q] = c < p.N ? *reinterpret_cast<const f32x4_t*>(s + c + 4 * q) : f32x4_t{};
    }
#pragma unroll
    for (int m = 0; m < NB; ++m) {
      const int row = wm * 128 + m * 32 + l;
      if (row >= rows) continue;
      const int r = r0 + row;
      const float xs = p.xs[source_row(p, r)];
      bf16_t* out = p.out + (size_t)r * p.N;
      if constexpr (GU) {
        if (n >= p.N) continue;
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = swiglu((float)acc[0][m][i] * xs * ws[0][i / 4][i % 4],
                        (float)acc[1][m][i] * xs * ws[1][i / 4][i % 4]);
        *reinterpret_cast<uint4*>(out + n) = pack8(o);
        *reinterpret_cast<uint4*>(out + n + 8) = pack8(o + 8);
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int c = n + b * 16;
          if (c >= p.N) continue;
          float o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = (float)acc[b][m][i] * xs * ws[b][i / 4][i % 4];
          *reinterpret_cast<uint4*>(out + c) = pack8(o);
          *reinterpret_cast<uint4*>(out + c + 8) = pack8(o + 8);
        }
      }
    }
  }
};

// Experts with more than `few` rows, in tiles: (expert, column tile, row tile) in
// that order, the row tiles of one column tile next to each other on one XCD.
template <bool GU>
__global__ __launch_bounds__(256, 2) void tile_i8_kernel(ProductI8 p, int few) {
  __shared__ __align__(16) char lds[kStages * kStageBytes];
  __shared__ int scan[4], found[4];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int cols = (p.N + (GU ? 63 : 127)) / (GU ? 64 : 128);
  // row tiles before this thread's expert
  const int lo = tid < p.E_l ? p.offsets[tid] : 0, hi = tid < p.E_l ? p.offsets[tid + 1] : 0;
  const int mine = hi - lo > few ? (hi - lo + kTileM - 1) / kTileM : 0;
  int sum = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(sum, o, kWave);
    if (lane >= o) sum += up;
  }
  if (lane == 63) scan[wave] = sum;
  __syncthreads();
  int before = sum - mine;
  for (int w = 0; w < wave; ++w) before += scan[w];
  const int tiles = (scan[0] + scan[1] + scan[2] + scan[3]) * cols;
  if ((int)blockIdx.x >= tiles) return;
  const int id = xcd_remap((int)blockIdx.x, tiles);
  // expert by expert: its tiles are mine * cols in a run
  if (id >= before * cols && id < (before + mine) * cols) {
    const int at = id - before * cols;
    found[0] = tid;
    found[1] = at / mine;
    found[2] = lo + (at % mine) * kTileM;
    found[3] = hi;
  }
  __syncthreads();
  const int r0 = __builtin_amdgcn_readfirstlane(found[2]), end = __builtin_amdgcn_readfirstlane(found[3]);
  const int rows = min(kTileM, end - r0);
  const Tile<GU> t(p, lds, __builtin_amdgcn_readfirstlane(found[0]),
                   __builtin_amdgcn_readfirstlane(found[1]) * (GU ? 64 : 128), r0, rows);
  const int w = __builtin_amdgcn_readfirstlane(wave), wm = w >> 1, wn = w & 1;
  const int blocks = (rows - wm * 128 + 31) / 32;  // of this wave that have rows
  if (blocks > 2) t.template run<4>(wm, wn);
  else if (blocks > 0) t.template run<2>(wm, wn);
  else t.template run<0>(wm, wn);
}

// Up to this many rows for an expert on average go without the tiles: one launch
// then serves every expert, whatever its rows.
constexpr int kSkinnyOnly = 16;

template <bool GU>
hipError_t launch_product(const ProductI8& p, int R_cap, int kernel_id, hipStream_t s) {
  ProfScope ps(kernel_id, s);
  const int few_cols = GU ? 16 : 32, cols = GU ? 64 : 128;
  const bool tiles = R_cap > kSkinnyOnly * p.E_l;
  const dim3 grid((p.N + few_cols - 1) / few_cols, std::min(p.E_l, R_cap));
  if (tiles) {
    const unsigned most = (unsigned)(R_cap / kTileM + p.E_l) * (unsigned)((p.N + cols - 1) / cols);
    tile_i8_kernel<GU><<<most, 256, 0, s>>>(p, kFew);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  skinny_i8_kernel<GU><<<grid, 256, 0, s>>>(p, tiles ? kFew : 0x7fffffff);
  return hipGetLastError();
}

}  // namespace

// Threads of the larger of the launches (below 2^32 as a caller has to check).
uint64_t gemm_i8_threads(int R_cap, int E_l, int N) {
  return ((uint64_t)R_cap / kTileM + (uint64_t)E_l) * (uint64_t)((N + 63) / 64) * 256;
}

hipError_t launch_gemm_i8(const int8_t* x, const float* xs, const int32_t* src, int x_rows,
                          const int32_t* offsets, int E_l, int R_cap, int K, int N, const int8_t* w,
                          const float* ws, bf16_t* y, hipStream_t s) {
  const ProductI8 p = {x, xs, src, x_rows, offsets, E_l, K, N, w, nullptr, ws, nullptr, y};
  return launch_product<false>(p, R_cap, MOE_KERNEL_GEMM_I8, s);
}

size_t ffn_fwd_i8_ws_bytes(int R_cap, int I) {
  const auto al = [](size_t b) { return (b + 255) & ~(size_t)255; };
  return al((size_t)R_cap * I) + al((size_t)R_cap * sizeof(float));
}

hipError_t launch_ffn_fwd_i8(const int8_t* x, const float* xs, const int32_t* src, int x_rows,
                             const int32_t* offsets, int E_l, int R_cap, int H, int I, const int8_t* wg,
                             const float* wgs, const int8_t* wu, const float* wus, const int8_t* wd,
                             const float* wds, bf16_t* h, bf16_t* y, void* ws, hipStream_t s) {
  int8_t* hq = (int8_t*)ws;
  float* hs = (float*)((char*)ws + (((size_t)R_cap * I + 255) & ~(size_t)255));
  const ProductI8 up = {x, xs, src, x_rows, offsets, E_l, H, I, wg, wu, wgs, wus, h};
  hipError_t e = launch_product<true>(up, R_cap, MOE_KERNEL_FFN_GATEUP_I8, s);
  if (e != hipSuccess) return e;
  e = launch_quantize_i8(h, R_cap, I, I, true, offsets + E_l, hq, hs, s);
  if (e != hipSuccess) return e;
  const ProductI8 down = {hq, hs, nullptr, R_cap, offsets, E_l, I, H, wd, nullptr, wds, nullptr, y};
  return launch_product<false>(down, R_cap, MOE_KERNEL_FFN_DOWN_I8, s);
}

}  // namespace moe
