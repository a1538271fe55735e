// Products of int8 rows with int8 expert weights, grouped by expert, for gfx950:
//   y[r,n] = xs[src r] ws[e,n] sum_k x[src r,k] w[e,n,k],  rows r of expert e,
// and the SwiGLU pair of them, h[r,n] = SiLU(g) u with the gate's and the up
// weight's products.  The sums are whole numbers, exact in the matrix core's
// int32, so every variant and every split of K gives the same bits; the two
// scales are applied in fp32 and the result is rounded once.
//
// Two kernels share the experts out by their number of rows, which only the
// device knows:
//   few rows (skinny_expert): bound by the read of the weights.  A workgroup
//     owns 32 columns of one expert; its four waves split K and take the weights
//     straight from memory into MFMA operands, each byte once for up to 64 rows,
//     and add their sums through LDS.
//   many rows (tile_i8_kernel): bound by the matrix cores and what feeds them.
//     Tiles of 256 rows x 256 weight rows in a workgroup of eight waves that stays
//     on its CU and takes tile after tile; operands through two LDS stages of 128
//     bytes of K (whole cache lines) filled by DMA, the next tile's first stages on
//     their way while the results of the last are written.
// Weights are the first operand of the MFMA, so that a lane's results are
// neighbouring columns of one row; which weight row takes which place in the
// operand is chosen so that they are 16 or 32 in a run.
#include <algorithm>
#include <type_traits>

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

// The i-th expert that has rows; false if there are fewer.
__device__ __forceinline__ bool nth_expert(const int32_t* __restrict__ offsets, int E_l, int i, int& e,
                                           int& lo, int& hi) {
  const int lane = lane_id();
  int a[kMaxE / kWave], b[kMaxE / kWave];
#pragma unroll
  for (int c = 0; c < kMaxE / kWave; ++c) {  // one round trip for all of them
    const int at = c * kWave + lane;
    a[c] = at < E_l ? offsets[at] : 0;
    b[c] = at < E_l ? offsets[at + 1] : 0;
  }
#pragma unroll
  for (int c = 0; c < kMaxE / kWave; ++c) {
    const bool has = b[c] > a[c];
    const uint64_t m = __ballot(has);
    const int n = __popcll(m);
    if (i < n) {
      const uint64_t mine = __ballot(has && __popcll(m & ((1ull << lane) - 1ull)) == i);
      const int l = __ffsll((unsigned long long)mine) - 1;
      e = c * kWave + l;
      lo = __builtin_amdgcn_readlane(a[c], l);
      hi = __builtin_amdgcn_readlane(b[c], l);
      return true;
    }
    i -= n;
  }
  return false;
}

// NB blocks of 16 rows from row r0 on.  Columns: GU: 16 of gate and the same of
// up; else 32, a lane's 4 + 4 in a run of 8.
template <bool GU, int NB, int WAVES>
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
  for (int s0 = wave; s0 < steps; s0 += WAVES * U) {
    i32x4_t a[U][2], b[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + WAVES * u) * 64;
      const bool in = k + g * 16 < p.K;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[u][i] = in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(wr[i] + k)) : i32x4_t{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + WAVES * u) * 64;
      const bool in = k + g * 16 < p.K;
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
      for (int w = 1; w < WAVES; ++w) sum[i] += red[w][i * NB + wave][lane];
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

// All rows [lo, hi) of expert e for the columns from n0 on.
template <bool GU, int WAVES>
__device__ __forceinline__ void skinny_expert(const ProductI8& p, int e, int n0, int lo, int hi,
                                              i32x4_t (*red)[2 * 4][kWave]) {
  for (int r0 = lo; r0 < hi; r0 += kFew) {
    if (r0 > lo) __syncthreads();  // the last sums have been read
    const int left = hi - r0;
    if (left <= 16) skinny_rows<GU, 1, WAVES>(p, e, n0, r0, hi, red);
    else if (left <= 32) skinny_rows<GU, 2, WAVES>(p, e, n0, r0, hi, red);
    else skinny_rows<GU, 4, WAVES>(p, e, n0, r0, hi, red);
  }
}

template <bool GU>
__global__ __launch_bounds__(256) void skinny_i8_kernel(ProductI8 p) {
  __shared__ i32x4_t red[4][2 * 4][kWave];
  int e, lo, hi;
  if (!nth_expert(p.offsets, p.E_l, (int)blockIdx.y, e, lo, hi)) return;
  skinny_expert<GU, 4>(p, e, (int)blockIdx.x * (GU ? 16 : 32), lo, hi, red);
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kTileM = 256;    // most rows of a tile
constexpr int kTileW = 256;    // weight rows of a tile (128 of gate and 128 of up in the pair)
constexpr int kTileWaves = 8;  // 2 along the rows, 4 along the weight rows
constexpr int kStageK = 128;    // bytes of K a stage
constexpr int kStages = 256 / kStageK;
constexpr int kStageBytes = (kTileM + kTileW) * kStageK;
constexpr int kRowChunks = kStageK / 16;            // 16-byte chunks of an LDS row
constexpr int kDmaRows = kWave / kRowChunks;        // LDS rows that one DMA fills
constexpr int kDmas = kTileM / kDmaRows / kTileWaves;  // of a wave, a step, for each operand
constexpr int kOutBytes = 32 * 64;  // of a wave: 32 rows of 32 columns on their way out
constexpr int kOutAt = kStages * kStageBytes;
constexpr int kTileLds = kOutAt + kTileWaves * kOutBytes;

template <bool GU>
constexpr int tile_cols() { return GU ? 128 : 256; }

__device__ __forceinline__ uint32_t lds_byte_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)p);
}

// Chunks of 16 bytes of an LDS row are stored at place c ^ swizzle(row), so that
// neighbouring lanes of an operand read (rows in the order of the operand, one
// chunk) touch different banks: 8 of them different places of 128 bytes, 16 of them
// of 256.  For rows of 128 and of 64 bytes:
template <int CHUNKS>
__device__ __forceinline__ int swizzle_row(int row) {
  return CHUNKS == 8 ? ((row >> 1) & 3) << 1 | ((row ^ (row >> 3)) & 1)
                     : ((row >> 2) & 1) << 1 | (((row >> 1) ^ (row >> 3)) & 1);
}
__device__ __forceinline__ int swizzle_w(int row) {
  const int h = (row >> 4) & 1;
  return kRowChunks == 8 ? ((row >> 1) & 1) << 2 | h << 1 | ((row ^ (row >> 2)) & 1)
                         : h << 1 | (((row >> 1) ^ (row >> 2)) & 1);
}

// Where a tile lies.
struct At {
  int e, n0, r0, rows;  // expert, first column, first row, rows (1 .. tile height)
};

// What every workgroup finds out from the offsets, and what it keeps of a tile.
struct TileLds {
  int start[kMaxE + 1];  // row tiles before expert e
  int row0[kMaxE], row1[kMaxE];
  int list[kMaxE];       // experts with few rows
  int scan[4], few[4], tall[4];
  int row[kTileM];       // rows of x of the next tile
  float xs[kTileM], ws[kTileW];  // scales of the tile in work
};

// What a workgroup's DMA reads of a tile.
template <bool GU>
struct Feed {
  uint32_t wv[kDmas], xv[kDmas];  // byte offsets of this lane's chunks at K = 0, or kDmaKill
  rsrc_t wd[2], xd;
  int K;

  // DMA i of a wave fills LDS rows i * 8 kDmaRows + wave * kDmaRows + lane / kRowChunks.
  static __device__ __forceinline__ int lds_row(int i, int wave) {
    return (i * kTileWaves + wave) * kDmaRows + lane_id() / kRowChunks;
  }
  static __device__ __forceinline__ int chunk_w(int i, int wave) {
    return (lane_id() & (kRowChunks - 1)) ^ swizzle_w(lds_row(i, wave));
  }
  static __device__ __forceinline__ int chunk_x(int i, int wave) {
    return (lane_id() & (kRowChunks - 1)) ^ swizzle_row<kRowChunks>(lds_row(i, wave));
  }

  __device__ __forceinline__ void set(const ProductI8& p, const At& t, const int* rows, int wave) {
    const uint32_t wbytes = (uint32_t)p.N * (uint32_t)p.K;
    K = p.K;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      wd[i] = make_rsrc((GU && i == 1 ? p.w1 : p.w0) + (size_t)t.e * p.N * p.K, wbytes);
    xd = make_rsrc(p.x, (uint32_t)p.x_rows * (uint32_t)p.K);
#pragma unroll
    for (int i = 0; i < kDmas; ++i) {
      const int row = lds_row(i, wave);
      const int n = GU ? t.n0 + (row & 127) : t.n0 + row;
      wv[i] = n < p.N ? (uint32_t)n * (uint32_t)p.K + chunk_w(i, wave) * 16 : kDmaKill;
      xv[i] = row < t.rows ? (uint32_t)rows[row] * (uint32_t)p.K + chunk_x(i, wave) * 16 : kDmaKill;
    }
  }

  // The first steps of a tile, into all stages.
  __device__ __forceinline__ void start(uint32_t to, int wave) const {
#pragma unroll
    for (int i = 0; i < kStages; ++i) issue(i, to + i * kStageBytes, wave);
  }

  // K step s into its ring stage; chunks past K (and whole steps past the last)
  // are dropped and leave zeros.
  __device__ __forceinline__ void issue(int s, uint32_t to, int wave) const {
    const int k = s * kStageK;
#pragma unroll
    for (int i = 0; i < kDmas; ++i) {
      const bool in = k + chunk_w(i, wave) * 16 < K && wv[i] != kDmaKill;
      dma16(wd[GU ? i / (kDmas / 2) : 0], in ? wv[i] + k : kDmaKill, to + i * (kTileWaves * 1024));
    }
#pragma unroll
    for (int i = 0; i < kDmas; ++i) {
      const bool in = k + chunk_x(i, wave) * 16 < K && xv[i] != kDmaKill;
      dma16(xd, in ? xv[i] + k : kDmaKill, to + kTileW * kStageK + i * (kTileWaves * 1024));
    }
  }
};

__device__ __forceinline__ void store16(u32x4_t v, u32x4_t* to) {
#ifdef NTS
  __builtin_nontemporal_store(v, to);
#else
  *to = v;
#endif
}

template <bool GU>
struct Wave {
  const ProductI8& p;
  char* lds;
  TileLds& c;
  uint32_t lds0;  // where this wave's DMA goes in the first stage
  int wave, wm, wn, half, l;

  __device__ Wave(const ProductI8& p_, char* lds_, TileLds& c_) : p(p_), lds(lds_), c(c_) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lds0 = lds_byte_addr(lds) + wave * 1024;
    wm = wave >> 2;
    wn = wave & 3;
    half = lane_id() >> 5;
    l = lane_id() & 31;
  }

  // Operands of 32 bytes of K, read from a stage while the products of the last
  // ones run.
  template <int NB>
  struct Operands {
    i32x4_t w[2], x[NB];
    __device__ __forceinline__ void load(const char* w_at, const char* x_at) {
      constexpr int kBlk = (GU ? 128 : 32) * kStageK;  // from the first block of 32 weight rows to the second
#pragma unroll
      for (int b = 0; b < 2; ++b) w[b] = *reinterpret_cast<const i32x4_t*>(w_at + b * kBlk);
#pragma unroll
      for (int m = 0; m < NB; ++m) x[m] = *reinterpret_cast<const i32x4_t*>(x_at + m * 32 * kStageK);
    }
  };
  template <int NB, bool FIRST>
  static __device__ __forceinline__ void multiply(const Operands<NB>& o, i32x16_t (&acc)[2][NB]) {
    const i32x16_t zero = {};
#pragma unroll
    for (int m = 0; m < NB; ++m)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[b][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[b], o.x[m], FIRST ? zero : acc[b][m], 0, 0, 0);
  }
  // Order for the scheduler: the 2 + NB operand reads spread over the 2 NB products
  // before them, one after each.
  template <int NB>
  static __device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);    // a product
      if (i < 2 + NB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
    }
    if constexpr (2 + NB > 2 * NB) __builtin_amdgcn_sched_group_barrier(0x100, 2 + NB - 2 * NB, 0);
  }

  // One tile, whose first steps have landed in the stages (every wave has waited for
  // its part of them).  The products of 64 weight rows with NB blocks of 32 rows,
  // from row `first` of the tile on; `begin` fetches what the next tile and the
  // results need; `next` starts the next tile's first steps; then the results.
  template <int NB, class Begin, class Next>
  __device__ __forceinline__ void run(const At& t, const Feed<GU>& feed, int first, const Begin& begin,
                                      const Next& next) const {
    constexpr int N1 = NB == 0 ? 1 : NB;
    constexpr int kSub = kStageK / 32;  // operands of a stage
    const int a = l >> 3, h = (l >> 2) & 1, j = l & 3;
    const int wrow = wn * (GU ? 32 : 64) + h * 16 + 4 * a + j;
    const int sw = swizzle_w(wrow), sx = swizzle_row<kRowChunks>(l);
    int aw[kSub], ax[kSub];
#pragma unroll
    for (int ks = 0; ks < kSub; ++ks) {
      aw[ks] = wrow * kStageK + (((ks * 2 + half) ^ sw) * 16);
      ax[ks] = kTileW * kStageK + (first + l) * kStageK + (((ks * 2 + half) ^ sx) * 16);
    }
    i32x16_t acc[2][N1];
    const int steps = (p.K + kStageK - 1) / kStageK;
    lds_barrier();  // everybody's part of the first steps
    begin();
    Operands<N1> o[2];
    if constexpr (NB > 0) o[0].load(lds + aw[0], lds + ax[0]);
    const auto step = [&](auto first_step, int s) {
      constexpr bool kFirst = decltype(first_step)::value;
      const char* at = lds + (s & (kStages - 1)) * kStageBytes;
      const char* after = lds + ((s + 1) & (kStages - 1)) * kStageBytes;
#pragma unroll
      for (int ks = 0; ks < kSub - 1; ++ks) {
        if constexpr (NB > 0) {
          o[(ks + 1) & 1].load(at + aw[ks + 1], at + ax[ks + 1]);
          if constexpr (kFirst) {
            if (ks == 0) multiply<N1, true>(o[0], acc);
            else multiply<N1, false>(o[ks & 1], acc);
          } else {
            multiply<N1, false>(o[ks & 1], acc);
          }
          interleave<N1>();
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (s >= kStages - 1) wait_vm<2 * kDmas*(kStages - 2)>();  // this wave's part of step s + 1
      lds_barrier();  // everybody's, and everybody has read step s
      feed.issue(s + kStages, lds0 + (s & (kStages - 1)) * kStageBytes, wave);  // (dropped past K)
      if constexpr (NB > 0) {
        o[0].load(after + aw[0], after + ax[0]);  // (of no use after the last step)
        multiply<N1, false>(o[(kSub - 1) & 1], acc);
        interleave<N1>();
      }
    };
    step(std::true_type{}, 0);
    for (int s = 1; s < steps; ++s) step(std::false_type{}, s);
    wait_vm<0>();  // the dropped steps
    next.publish();
    lds_barrier();  // nobody reads the ring any more, and what `begin` fetched is in the LDS
    next();
    if constexpr (NB > 0) store<NB>(t, acc, first);
    else wait_vm<0>();  // the next tile's first steps
  }

  // The results of a wave go through its own part of the LDS, 32 rows of 32 columns
  // at a time, so that a store writes 64 bytes in a run.
  template <int NB>
  __device__ __forceinline__ void store(const At& t, const i32x16_t (&acc)[2][NB], int first) const {
    const int lane = lane_id(), chunk = lane & 3;
    char* mine = lds + kOutAt + wave * kOutBytes;
    f32x4_t ws[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ws[b][q] = *reinterpret_cast<const f32x4_t*>(c.ws + (GU ? b * 128 + wn * 32 : wn * 64 + b * 32) + half * 16 + 4 * q);
#pragma unroll
    for (int m = 0; m < NB; ++m) {
      const float xs = c.xs[first + m * 32 + l];
#pragma unroll
      for (int b = 0; b < (GU ? 1 : 2); ++b) {
        const int col = t.n0 + wn * (GU ? 32 : 64) + b * 32;
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = (float)acc[b][m][i] * xs * ws[b][i / 4][i % 4];
          o[i] = GU ? swiglu(v, (float)acc[1][m][i] * xs * ws[1][i / 4][i % 4]) : v;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<uint4*>(mine + (l * 4 + ((half * 2 + q) ^ swizzle_row<4>(l))) * 16) = pack8(o + 8 * q);
        // The next tile's first steps, before the first store: a wait for them later
        // would wait for the stores as well.
        if (m == 0 && b == 0) wait_vm<0>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = i * 16 + lane / 4;
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + (row * 4 + (chunk ^ swizzle_row<4>(row))) * 16);
          if (first + m * 32 + row < t.rows && col + chunk * 8 < p.N)
            store16(v, reinterpret_cast<u32x4_t*>(p.out + (size_t)(t.r0 + first + m * 32 + row) * p.N + col + chunk * 8));
        }
      }
    }
  }
};

// Experts with more than kFew rows in tiles, in the order (expert, column tile, row
// tile); then the other experts, a few columns at a time.  Every workgroup counts
// the tiles from the offsets and takes its share of them: an XCD a run of the
// order, in rounds of one tile a workgroup, so that neighbouring tiles (of the same
// weights, of the same rows) are in work at the same time on one L2.
template <bool GU>
__global__ __launch_bounds__(64 * kTileWaves, 2) void tile_i8_kernel(ProductI8 p) {
  extern __shared__ __align__(16) char lds[];
  __shared__ __align__(16) TileLds c;
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int cols = (p.N + tile_cols<GU>() - 1) / tile_cols<GU>();
  int height = kTileM;
  {
    const bool in = tid < p.E_l;
    const int lo = in ? p.offsets[tid] : 0, hi = in ? p.offsets[tid + 1] : 0, n = hi - lo;
    const bool is_few = n > 0 && n <= kFew;
    const uint64_t small = __ballot(is_few);
    // row tiles of the full height: with fewer of them than two for a workgroup,
    // tiles of half the height keep more CUs at work
    int full = n > kFew ? (n + kTileM - 1) / kTileM : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) full += __shfl_xor(full, o, kWave);
    if (lane == 0 && wave < 4) {
      c.tall[wave] = full;
      c.few[wave] = __popcll(small);
    }
    __syncthreads();
    if ((c.tall[0] + c.tall[1] + c.tall[2] + c.tall[3]) * cols < 2 * (int)gridDim.x) height = kTileM / 2;
    const int mine = n > kFew ? (n + height - 1) / height : 0;
    int sum = mine;  // row tiles up to this thread's expert
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int up = __shfl_up(sum, o, kWave);
      if (lane >= o) sum += up;
    }
    if (lane == 63 && wave < 4) c.scan[wave] = sum;
    __syncthreads();
    if (tid < kMaxE) {
      int at = __popcll(small & ((1ull << lane) - 1ull)), before = sum - mine;
      for (int w = 0; w < wave; ++w) {
        at += c.few[w];
        before += c.scan[w];
      }
      if (is_few) c.list[at] = tid;
      c.start[tid] = before;
      c.row0[tid] = lo;
      c.row1[tid] = hi;
    }
    if (tid == 0) c.start[kMaxE] = c.scan[0] + c.scan[1] + c.scan[2] + c.scan[3];
    __syncthreads();
  }
  const int tiles = c.start[kMaxE] * cols;
  // this XCD's run of the tiles
  const int xcds = min(8, (int)gridDim.x), xcd = (int)blockIdx.x % xcds, nth = (int)blockIdx.x / xcds;
  const int share = ((int)gridDim.x - xcd + xcds - 1) / xcds;  // workgroups of this XCD
  const int from = (int)((long)tiles * xcd / xcds), to = (int)((long)tiles * (xcd + 1) / xcds);
  const auto place = [&](int id) {
    // the last expert whose tiles begin at or before id (experts without tiles begin
    // where the next one does)
    const int* s = c.start + 4 * lane;
    int a = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) a += __popcll(__ballot(s[i] * cols <= id));
    const int n = c.start[a + 1] - c.start[a], at = id - c.start[a] * cols;
    const int r0 = c.row0[a] + at % n * height;
    At t;
    t.e = __builtin_amdgcn_readfirstlane(a);
    t.n0 = __builtin_amdgcn_readfirstlane(at / n) * tile_cols<GU>();
    t.r0 = __builtin_amdgcn_readfirstlane(r0);
    t.rows = __builtin_amdgcn_readfirstlane(min(height, c.row1[a] - r0));
    return t;
  };
  const Wave<GU> w(p, lds, c);
  int id = from + nth;
  if (id < to) {
    At t = place(id);
    Feed<GU> feed;
    // thread i < 256 keeps the row of x that row i of a tile is, the others the scale
    // of a weight row
    int row = tid < t.rows ? source_row(p, t.r0 + tid) : 0;
    if (tid < kTileM) c.row[tid] = row;
    __syncthreads();
    feed.set(p, t, c.row, w.wave);
    feed.start(w.lds0, w.wave);
    wait_vm<0>();
    while (id < to) {
      const At now = t;
      const Feed<GU> f = feed;
      float scale = 0.f;
      id += share;
      if (id < to) t = place(id);
      const auto begin = [&]() {
        if (tid < kTileM) {
          if (tid < now.rows) scale = p.xs[row];
          if (id < to && tid < t.rows) row = source_row(p, t.r0 + tid);
        } else {
          const int i = tid - kTileM, n = now.n0 + (GU ? i & 127 : i);
          if (n < p.N) scale = (GU && i >= 128 ? p.s1 : p.s0)[(size_t)now.e * p.N + n];
        }
      };
      struct {
        const ProductI8& p;
        const At& t;
        Feed<GU>& feed;
        TileLds& c;
        const Wave<GU>& w;
        const bool more;
        const int tid;
        const int& row;
        const float& scale;
        __device__ void publish() const {
          if (tid < kTileM) {
            c.row[tid] = row;
            c.xs[tid] = scale;
          } else {
            c.ws[tid - kTileM] = scale;
          }
        }
        __device__ void operator()() const {
          if (!more) return;
          feed.set(p, t, c.row, w.wave);
          feed.start(w.lds0, w.wave);
        }
      } next = {p, t, feed, c, w, id < to, tid, row, scale};
      const int first = w.wm * (height / 2);
      const int blocks = min((now.rows - first + 31) / 32, height / 64);  // of this wave that have rows
      if (blocks > 2) w.template run<4>(now, f, first, begin, next);
      else if (blocks > 0) w.template run<2>(now, f, first, begin, next);
      else w.template run<0>(now, f, first, begin, next);
    }
  }
  const int per = (p.N + (GU ? 15 : 31)) / (GU ? 16 : 32);
  const int items = (c.few[0] + c.few[1] + c.few[2] + c.few[3]) * per;
  for (int i = (int)blockIdx.x; i < items; i += (int)gridDim.x) {
    const int e = __builtin_amdgcn_readfirstlane(c.list[i / per]);
    __syncthreads();  // the LDS of the last tile or item has been read
    skinny_expert<GU, kTileWaves>(p, e, (i % per) * (GU ? 16 : 32), c.row0[e], c.row1[e],
                                  reinterpret_cast<i32x4_t(*)[2 * 4][kWave]>(lds));
  }
}

// Up to this many rows for an expert on average go without the tiles: the
// workgroups then need less LDS and stream the weights with more waves a CU.
constexpr int kSkinnyOnly = 32;

template <bool GU>
hipError_t launch_product(const ProductI8& p, int R_cap, int kernel_id, hipStream_t s) {
  ProfScope ps(kernel_id, s);
  if ((long)R_cap <= (long)kSkinnyOnly * p.E_l) {
    const int cols = (p.N + (GU ? 15 : 31)) / (GU ? 16 : 32);
    skinny_i8_kernel<GU><<<dim3(cols, std::min(p.E_l, R_cap)), 256, 0, s>>>(p);
  } else {
    tile_i8_kernel<GU><<<kCUs, 64 * kTileWaves, kTileLds, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

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
