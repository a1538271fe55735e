// Products of int8 rows with int8 expert weights, grouped by expert, for gfx950:
//   y[r,n] = xs[src r] ws[e,n] sum_k x[src r,k] w[e,n,k],  rows r of expert e,
// and the SwiGLU pair of them, h[r,n] = SiLU(g) u with the gate's and the up
// weight's products.  The sums are whole numbers, exact in the matrix core's
// int32, so every variant and every split of K gives the same bits; the two
// scales are applied in fp32 and the result is rounded once.
//
// Two kernels, chosen by the rows for an expert on average and by the size of the whole:
//   few rows (skinny_i8_kernel): bound by the read of the weights.  A workgroup
//     owns 32 columns of one expert (64 where K is short); its waves split K and
//     take the weights straight from memory into MFMA operands, each byte once for
//     up to 64 rows, and add their sums through LDS.  64 tokens of the whole layer
//     (128 experts of 2048 x 768, top-8): gate and up 56 us, down 32, 598 MB together
//     at 6.8 TB/s.
//   many rows (tile_i8_kernel): bound by the matrix cores and what feeds them.
//     Tiles of 256 rows x 256 weight rows in a workgroup of eight waves that stays
//     on its CU and takes tile after tile; operands through two LDS stages of 128
//     bytes of K (whole cache lines) filled by DMA, the next tile's first stages
//     issued between the stores of the last one's results.  16384 tokens of the whole
//     layer: gate and up 400 to 417 us (2000 TOP/s), down 320 (1290).  The steps are bound by
//     what fills the LDS: by the clocks of a step some 20 bytes a clock and CU arrive,
//     1.5 to 1.75 us for the 64 KB of a step, 2450 TOP/s and more in the steady state;
//     the products alone would take 1.15 us (3740 TOP/s on random operands).  The rest
//     are the ends of the tiles, for the down product with its 6 steps a tile a third.
//     Two waits that the compiler adds there make them longer than the counted ones ask:
//     before a tile's first products one for everything (the clamp of the next tile's row map uses
//     the loaded rows at once), which waits for the second step and the last tile's
//     stores as well; and in the down product seven reloads of spilled registers, each with one,
//     between the last stores of a tile.
// Weights are the first operand of the MFMA, so that a lane's results are
// neighbouring columns of one row; which weight row takes which place in the
// operand is chosen so that they are 16 or 32 in a run.
#include <algorithm>
#include <type_traits>

#include "rows_i8.h"

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
  bf16_t* out;      // [rows][N]
  const bf16_t* h;  // rows before their quantization (skinny_quantize_i8_kernel)
};

__device__ __forceinline__ int source_row(const ProductI8& p, int r) {
  const int x = p.src != nullptr ? p.src[r] : r;
  return min(max(x, 0), p.x_rows - 1);
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int kFew = 64;      // rows of one pass over an expert's weights
constexpr int kFewWaves = 4;  // of a workgroup

// Waves that share K: where it is short, two, and twice the columns, so that a wave
// has enough loads in flight (768: 64 tokens of the whole layer 51 -> 39 us).
constexpr int split_of(int K) { return K > 1024 ? 4 : 2; }

// The down product quantizes h itself up to this many rows for an expert on average
// and this many columns: one launch less, but every workgroup of an expert quantizes
// all of its rows.  The FFN, a launch more and so: 128 experts of 2048 x 768, 1/16 of
// a row on average 19.4 and 17.7 us, 1: 67.6 and 66.4, 4: 93.7 and 98.1; 64 experts of
// 2048 x 1536, 1/2 of a row 52.4 and 55.4.
constexpr int kFusedRows = 1, kFusedCols = 1024;
constexpr int kFusedSplit = split_of(kFusedCols);
static_assert(kFusedCols <= kWave * rows_i8::kCols, "a chunk of a row for each lane");

// Codes of up to 16 rows of p.h from r0 on, as moe_quantize_i8 makes them, a wave a
// row (of up to 64 * 16 columns).  Ends with a barrier.
__device__ __forceinline__ void quantize_rows(const ProductI8& p, int r0, int hi, int8_t* codes, float* scales) {
  using namespace rows_i8;
  const int lane = lane_id(), per_row = p.K / kCols;
  for (int r = threadIdx.x >> 6; r0 + r < hi; r += kFewWaves) {
    const size_t base = (size_t)(r0 + r) * p.K;
    float v[kCols];
    uint32_t top = 0;
    if (lane < per_row) {
      load16<true>(p.h, base + (size_t)lane * kCols, v);
      top = top_bits(v, top);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, kWave));
    const Scale s(top);
    if (lane == 0) scales[r] = s.scale;
    if (lane < per_row) *reinterpret_cast<u32x4_t*>(codes + r * p.K + lane * kCols) = codes16(v, s.inv);
  }
  __syncthreads();
}

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

// Columns of a wave: 16 of gate and the same of up, or 32, a lane's 4 + 4 in a run of 8.
template <bool GU>
constexpr int few_cols() { return GU ? 16 : 32; }

// NB blocks of 16 rows from row r0 on; every SPLIT waves share K for one wave's
// columns.  QUANT: the rows are bf16 (p.h), and their codes are made here, in LDS,
// while the weights are on their way.
template <bool GU, int NB, int SPLIT, bool QUANT = false>
__device__ __forceinline__ void skinny_rows(const ProductI8& p, int e, int n_first, int r0, int hi,
                                            i32x4_t (*red)[2 * 4][kWave], int8_t* codes = nullptr,
                                            float* scales = nullptr) {
  static_assert(!QUANT || NB == 1, "codes of one block of rows");
  constexpr int kCols = few_cols<GU>();
  constexpr int U = 8 / NB;  // K steps of 64 in flight
  const int lane = lane_id(), wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int steps = (p.K + 63) / 64, n0 = n_first + wave / SPLIT * kCols;
  int xi[NB];  // rows of x, needed after the weights' loads have been issued
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    const int r = min(r0 + m * 16 + l16, hi - 1);
    xi[m] = p.src != nullptr ? p.src[r] : r;
  }
  const int8_t* wr[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int n = GU ? n0 + l16 : n0 + (l16 >> 2) * 8 + b * 4 + (l16 & 3);
    wr[b] = (GU && b == 1 ? p.w1 : p.w0) + ((size_t)e * p.N + min(n, p.N - 1)) * p.K + g * 16;
  }
  i32x4_t acc[2][NB] = {};
  bool first = true;
  for (int s0 = wave % SPLIT; s0 < steps || (QUANT && first); s0 += SPLIT * U) {
    i32x4_t a[U][2], b[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + SPLIT * u) * 64;
      const bool in = k + g * 16 < p.K;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[u][i] = in ? *reinterpret_cast<const i32x4_t*>(wr[i] + k) : i32x4_t{};
    }
    const int8_t* xr[NB];
    if constexpr (QUANT) {
      if (first) quantize_rows(p, r0, hi, codes, scales);
      xr[0] = codes + min(l16, hi - 1 - r0) * p.K + g * 16;
    } else {
#pragma unroll
      for (int m = 0; m < NB; ++m) {
        asm volatile("" : "+v"(xi[m]));  // not before the weights' loads
        xr[m] = p.x + (size_t)min(max(xi[m], 0), p.x_rows - 1) * p.K + g * 16;
      }
    }
    first = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + SPLIT * u) * 64;
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
  for (int q = wave; q < NB * (kFewWaves / SPLIT); q += kFewWaves) {  // (block of rows, wave's columns)
    const int m = q % NB, cg = q / NB;
    i32x4_t sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = red[cg * SPLIT][i * NB + m][lane];
#pragma unroll
      for (int w = 1; w < SPLIT; ++w) sum[i] += red[cg * SPLIT + w][i * NB + m][lane];
    }
    const int r = r0 + m * 16 + l16, n = n_first + cg * kCols + g * (GU ? 4 : 8);
    if (r >= hi || n >= p.N) continue;
    const float xs = QUANT ? scales[l16] : p.xs[source_row(p, r)];
    const f32x4_t* ws = reinterpret_cast<const f32x4_t*>(p.s0 + (size_t)e * p.N + n);
    const f32x4_t wa = ws[0], wb = GU ? *reinterpret_cast<const f32x4_t*>(p.s1 + (size_t)e * p.N + n) : ws[1];
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float va = (float)sum[0][i] * xs * wa[i], vb = (float)sum[1][i] * xs * wb[i];
      o[i] = GU ? swiglu(va, vb) : va;
      o[4 + i] = vb;
    }
    bf16_t* to = p.out + (size_t)r * p.N + n;
    if constexpr (GU) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
    else *reinterpret_cast<uint4*>(to) = pack8(o);
  }
}

// Two waves a SIMD at the least: with registers for four the loads in flight spill
// (64 tokens of the whole layer: 88 us, 63 with these bounds, for 403 MB).
template <bool GU, int SPLIT>
__global__ __launch_bounds__(256, 2) void skinny_i8_kernel(ProductI8 p) {
  __shared__ i32x4_t red[4][2 * 4][kWave];
  int e, lo, hi;
  if (!nth_expert(p.offsets, p.E_l, (int)blockIdx.y, e, lo, hi)) return;
  const int n0 = (int)blockIdx.x * (kFewWaves / SPLIT * few_cols<GU>());
  const int from = lo + (int)blockIdx.z * kFew, by = (int)gridDim.z * kFew;
  for (int r0 = from; r0 < hi; r0 += by) {
    if (r0 > from) __syncthreads();  // the last sums have been read
    const int left = hi - r0;
    if (left <= 16) skinny_rows<GU, 1, SPLIT>(p, e, n0, r0, hi, red);
    else if (left <= 32) skinny_rows<GU, 2, SPLIT>(p, e, n0, r0, hi, red);
    else skinny_rows<GU, 4, SPLIT>(p, e, n0, r0, hi, red);
  }
}

// The product of bf16 rows, each workgroup quantizing those of its expert itself,
// 16 at a time: for few rows one launch less, and the rows' reads lie under the
// weights'.
__global__ __launch_bounds__(256, 2) void skinny_quantize_i8_kernel(ProductI8 p) {
  extern __shared__ __align__(16) char lds[];  // codes of 16 rows
  __shared__ i32x4_t red[4][2 * 4][kWave];
  __shared__ float scales[16];
  int e, lo, hi;
  if (!nth_expert(p.offsets, p.E_l, (int)blockIdx.y, e, lo, hi)) return;
  for (int r0 = lo; r0 < hi; r0 += 16) {
    if (r0 > lo) __syncthreads();  // the last sums and codes have been read
    skinny_rows<false, 1, kFusedSplit, true>(p, e, (int)blockIdx.x * (kFewWaves / kFusedSplit * few_cols<false>()),
                                             r0, min(hi, r0 + 16), red, (int8_t*)lds, scales);
  }
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kTileM = 256;    // most rows of a tile
constexpr int kTileW = 256;    // weight rows of a tile (128 of gate and 128 of up in the pair)
constexpr int kTileWaves = 8;  // 2 along the rows, 4 along the weight rows
constexpr int kStageK = 128;   // bytes of K a stage
constexpr int kStages = 2;
constexpr int kStageBytes = (kTileM + kTileW) * kStageK;
constexpr int kRowChunks = kStageK / 16;            // 16-byte chunks of an LDS row
constexpr int kDmaRows = kWave / kRowChunks;        // LDS rows that one DMA fills
constexpr int kDmas = kTileM / kDmaRows / kTileWaves;  // of a wave, a step, for each operand
constexpr int kOutBytes = 32 * 64;  // of a wave: 32 rows of 32 columns on their way out
constexpr int kOutAt = kStages * kStageBytes;
constexpr int kTileLds = kOutAt + kTileWaves * kOutBytes;

// Streaming stores for a product's rows, in whole cache lines: 131072 rows of 768 by
// 2048 columns 316 -> 260 us, inside the FFN 355 -> 351.  (h, in half lines and read
// again at once, is stored plainly: 493 us, 503 streamed.)
constexpr int kStreamed = 2;

template <bool GU>
constexpr int tile_cols() { return GU ? 128 : 256; }

// Between the LDS accesses of a wave's lanes to each other's values: the hardware
// keeps them in order, and the compiler, which looks at one lane, is kept from
// changing it.
__device__ __forceinline__ void lanes_meet() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_byte_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)p);
}

// Chunks of 16 bytes of an LDS row are stored at place c ^ swizzle(row), so that
// neighbouring lanes of an operand read (rows in the order of the operand, one
// chunk) touch different banks: 8 of them different places of 128 bytes, 16 of them
// of 256.  For rows of 8 chunks, and of 4 (results on their way out):
template <int CHUNKS>
__device__ __forceinline__ int swizzle_row(int row) {
  return CHUNKS == 8 ? ((row >> 1) & 3) << 1 | ((row ^ (row >> 3)) & 1)
                     : ((row >> 2) & 1) << 1 | (((row >> 1) ^ (row >> 3)) & 1);
}
__device__ __forceinline__ int swizzle_w(int row) {
  return ((row >> 1) & 1) << 2 | ((row >> 4) & 1) << 1 | ((row ^ (row >> 2)) & 1);
}

// Where a tile lies.
struct At {
  int e, n0, r0, rows;  // expert, first column, first row, rows (1 .. tile height)
};

// What every workgroup finds out from the offsets, and what it keeps of a tile.
struct TileLds {
  int start[kMaxE + 4];  // row tiles before expert e; start[kMaxE]: of all
  int off[kMaxE + 4];    // the offsets (experts past E_l have no rows)
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

  // DMA i of K step s (the weights' first) into its ring stage; chunks past K (and
  // whole steps past the last) are dropped and leave zeros.
  __device__ __forceinline__ void issue(int i, int s, uint32_t to, int wave) const {
    const int k = s * kStageK, j = i % kDmas;
    if (i < kDmas) {
      const bool in = k + chunk_w(j, wave) * 16 < K && wv[j] != kDmaKill;
      dma16(wd[GU ? j / (kDmas / 2) : 0], in ? wv[j] + k : kDmaKill, to + j * (kTileWaves * 1024));
    } else {
      const bool in = k + chunk_x(j, wave) * 16 < K && xv[j] != kDmaKill;
      dma16(xd, in ? xv[j] + k : kDmaKill, to + kTileW * kStageK + j * (kTileWaves * 1024));
    }
  }
  // DMA i of the first two steps, into the first two stages.
  __device__ __forceinline__ void start(int i, uint32_t to, int wave) const {
    issue(i % (2 * kDmas), i / (2 * kDmas), to + i / (2 * kDmas) * kStageBytes, wave);
  }
};

// The results of a wave with NB blocks of 32 rows leave in blocks of 32 columns, two
// stores each, and the DMAs of the next tile's first two steps are issued in the
// first (up to four) of them: the memory counter of a wait for one of the steps has
// to leave room for what was issued after it, a fixed number of operations.
template <bool GU, int NB>
struct Order {
  static constexpr int kBlocks = NB * (GU ? 1 : 2);
  static constexpr int kFront = kBlocks < 4 ? kBlocks : 4;
  static constexpr int kPer = kFront == 0 ? 0 : 4 * kDmas / kFront;  // DMAs in each of the first blocks
  // operations behind the first step's last DMA, and behind the second's
  static constexpr int stores_from(int block) { return GU ? 2 * (kBlocks - block) : 4 * ((kBlocks - block + 1) / 2); }
  static constexpr int kAfter0 = 2 * kDmas + (kFront == 0 ? 0 : stores_from((2 * kDmas - 1) / kPer));
  static constexpr int kAfter1 = kFront == 0 ? 0 : stores_from(kFront - 1);
};

// A wait for the second step of a tile, with this many operations behind it.
__device__ __forceinline__ void wait_second(int after) {
  if (after == 12) wait_vm<12>();
  else if (after == 4) wait_vm<4>();
  else if (after == 2) wait_vm<2>();
  else wait_vm<0>();
}
static_assert(Order<false, 4>::kAfter1 == 12 && Order<false, 2>::kAfter1 == 4 && Order<true, 4>::kAfter1 == 2 &&
              Order<true, 2>::kAfter1 == 2 && Order<true, 0>::kAfter1 == 0, "the counts that wait_second knows");

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

  // One tile, whose first step has landed in the first stage and whose second is on
  // its way, `after` operations behind it.  The products of 64 weight rows with NB
  // blocks of 32 rows, from row `first` of the tile on; `begin` fetches what the next
  // tile and the results need; then the results, and the next tile's first steps
  // between them.  Returns what is behind its second step.
  template <int NB, class Begin, class Next>
  __device__ __forceinline__ int run(const At& t, const Feed<GU>& feed, int first, int after,
                                     const Begin& begin, const Next& next) const {
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
    lds_barrier();  // everybody's part of the first step
    begin();
    Operands<N1> o[2];
    if constexpr (NB > 0) o[0].load(lds + aw[0], lds + ax[0]);
    const auto step = [&](auto first_step, int s) {
      constexpr bool kFirst = decltype(first_step)::value;
      const char* at = lds + (s & 1) * kStageBytes;
      const char* behind = lds + ((s + 1) & 1) * kStageBytes;
#pragma unroll
      for (int ks = 0; ks < kSub - 1; ++ks) {
        // A step's DMAs are spread over the products: a wave whose DMAs wait for the
        // memory pipeline issues no products.  These are the rest of step s + 1.
        if (!kFirst && ks < 2) {
#pragma unroll
          for (int i = 3 + 3 * ks; i < 6 + 2 * ks; ++i)
            feed.issue(i, s + 1, lds0 + ((s + 1) & 1) * kStageBytes, wave);
        }
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
      if (kFirst) wait_second(after);  // this wave's part of step s + 1
      else wait_vm<0>();
      lds_barrier();  // everybody's, and everybody has read step s
#pragma unroll
      for (int i = 0; i < 3; ++i) feed.issue(i, s + 2, lds0 + (s & 1) * kStageBytes, wave);  // (dropped past K)
      if constexpr (NB > 0) {
        o[0].load(behind + aw[0], behind + ax[0]);  // (of no use after the last step)
        multiply<N1, false>(o[(kSub - 1) & 1], acc);
        interleave<N1>();
      }
    };
    step(std::true_type{}, 0);
    for (int s = 1; s < steps; ++s) step(std::false_type{}, s);
    wait_vm<0>();  // the dropped steps
    next.publish();
    lds_barrier();  // nobody reads the ring any more, and what `begin` fetched is in the LDS
    next.set();
    store<NB>(t, acc, first, next);
    wait_vm<Order<GU, NB>::kAfter0>();  // the next tile's first step
    return Order<GU, NB>::kAfter1;
  }

  // The results of a wave go through its own part of the LDS, 32 rows of 32 columns
  // at a time, so that a store writes 64 bytes in a run.
  template <int NB, class Next, int N1>
  __device__ __forceinline__ void store(const At& t, const i32x16_t (&acc)[2][N1], int first,
                                        const Next& next) const {
    if constexpr (NB == 0) {
#pragma unroll
      for (int i = 0; i < 4 * kDmas; ++i) next.start(i);
      return;
    }
    using O = Order<GU, NB>;
    const int lane = lane_id(), chunk = lane & 3;
    char* mine = lds + kOutAt + wave * kOutBytes;
    const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(
        p.out + (size_t)t.r0 * p.N, 0, t.rows * p.N * 2, 0x00020000);
    uint4 held[4];
    f32x4_t ws[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ws[b][q] = *reinterpret_cast<const f32x4_t*>(c.ws + (GU ? b * 128 + wn * 32 : wn * 64 + b * 32) + half * 16 + 4 * q);
#pragma unroll
    for (int n = 0; n < O::kBlocks; ++n) {
      const int m = GU ? n : n / 2, b = GU ? 0 : n % 2;
      if (n < O::kFront) {
#pragma unroll
        for (int i = 0; i < O::kPer; ++i) next.start(n * O::kPer + i);
      }
      const float xs = c.xs[first + m * 32 + l];
      const int col = t.n0 + wn * (GU ? 32 : 64) + b * 32;
      float o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = (float)acc[b][m][i] * xs * ws[b][i / 4][i % 4];
        o[i] = GU ? swiglu(v, (float)acc[1][m][i] * xs * ws[1][i / 4][i % 4]) : v;
      }
      if constexpr (GU) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<uint4*>(mine + (l * 4 + ((half * 2 + q) ^ swizzle_row<4>(l))) * 16) = pack8(o + 8 * q);
        lanes_meet();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = i * 16 + lane / 4, at = first + m * 32 + row;
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + (row * 4 + (chunk ^ swizzle_row<4>(row))) * 16);
          const bool in = at < t.rows && col + chunk * 8 < p.N;  // (the others are dropped by the descriptor's range)
          __builtin_amdgcn_raw_buffer_store_b128(v, to, in ? (at * p.N + col + chunk * 8) * 2 : (int)kDmaKill, 0, 0);
        }
        lanes_meet();
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) held[b * 2 + q] = pack8(o + 8 * q);
        if (b == 1) {  // 16 rows of 64 columns at a time
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if ((l >> 4) == g) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int ch = (q >> 1) * 4 + half * 2 + (q & 1);
                *reinterpret_cast<uint4*>(mine + ((l & 15) * 8 + (ch ^ swizzle_row<8>(l & 15))) * 16) = held[q];
              }
            }
            lanes_meet();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = i * 8 + lane / 8, at = first + m * 32 + g * 16 + row, ch = lane & 7;
              const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + (row * 8 + (ch ^ swizzle_row<8>(row))) * 16);
              const int c0 = t.n0 + wn * 64 + ch * 8;
              const bool in = at < t.rows && c0 < p.N;
              __builtin_amdgcn_raw_buffer_store_b128(v, to, in ? (at * p.N + c0) * 2 : (int)kDmaKill, 0, kStreamed);
            }
            lanes_meet();
          }
        }
      }
    }
  }
};

// Sums of the lanes up to each (inclusive), by row shifts and broadcasts.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of a row to the next
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return v;
}

// Tiles in the order (expert, column tile, row tile).  Every workgroup counts them
// from the offsets and takes its share: an XCD a run of the order, in rounds of one
// tile a workgroup, so that neighbouring tiles (of the same weights, of the same
// rows) are in work at the same time on one L2.
template <bool GU>
__global__ __launch_bounds__(64 * kTileWaves, 2) void tile_i8_kernel(ProductI8 p) {
  extern __shared__ __align__(16) char lds[];
  __shared__ __align__(16) TileLds c;
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int cols = (p.N + tile_cols<GU>() - 1) / tile_cols<GU>();
  // Every wave counts for itself, a lane for four experts, and writes what the others
  // write: nobody waits for anybody.
  int height = kTileM;
  {
    int off[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) off[i] = p.offsets[min(4 * lane + i, p.E_l)];
    const auto tiles_of = [&](int h, int i) { return (max(off[i + 1] - off[i], 0) + h - 1) / h; };
    int full = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) full += tiles_of(kTileM, i);
    // tiles of the full height: with fewer of them than two for a workgroup, tiles of
    // half the height keep more CUs at work (FFN of 16 experts, 64 rows each: 53.6 -> 42.2
    // us; with more tiles half of them are slower: 1024 rows for each of 128, 840 ->
    // 1039 us)
    if (__builtin_amdgcn_readlane(wave_scan(full), 63) * cols < 2 * (int)gridDim.x) height = kTileM / 2;
    int mine = 0, n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mine += n[i] = height == kTileM ? tiles_of(kTileM, i) : tiles_of(kTileM / 2, i);
    const int upto = wave_scan(mine);
    int before = upto - mine;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c.start[4 * lane + i] = before;
      c.off[4 * lane + i] = off[i];
      before += n[i];
    }
    if (lane == 63) {
      c.start[kMaxE] = upto;
      c.off[kMaxE] = off[4];
    }
    lanes_meet();
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
    const uint32_t n = c.start[a + 1] - c.start[a], at = id - c.start[a] * cols;
    const uint32_t col = at / n;
    const int r0 = c.off[a] + (int)(at - col * n) * height;
    At t;
    t.e = __builtin_amdgcn_readfirstlane(a);
    t.n0 = __builtin_amdgcn_readfirstlane((int)col) * tile_cols<GU>();
    t.r0 = __builtin_amdgcn_readfirstlane(r0);
    t.rows = __builtin_amdgcn_readfirstlane(min(height, c.off[a + 1] - r0));
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
#pragma unroll
    for (int i = 0; i < 4 * kDmas; ++i) feed.start(i, w.lds0, w.wave);
    wait_vm<2 * kDmas>();
    int after = 0;  // operations behind the second step
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
        // After the last tile every chunk is dropped: the DMAs have to be there for the
        // waits' counts, and move nothing.
        __device__ void set() const {
          feed.set(p, t, c.row, w.wave);
          if (more) return;
#pragma unroll
          for (int i = 0; i < kDmas; ++i) feed.wv[i] = feed.xv[i] = kDmaKill;
        }
        __device__ void start(int i) const { feed.start(i, w.lds0, w.wave); }
      } next = {p, t, feed, c, w, id < to, tid, row, scale};
      const int first = w.wm * (height / 2);
      const int blocks = min((now.rows - first + 31) / 32, height / 64);  // of this wave that have rows
      if (blocks > 2) after = w.template run<4>(now, f, first, after, begin, next);
      else if (blocks > 0) after = w.template run<2>(now, f, first, after, begin, next);
      else after = w.template run<0>(now, f, first, after, begin, next);
    }
    wait_vm<0>();  // the last "next tile", before the LDS is another workgroup's
  }
}

// Up to this many rows for an expert on average (of the capacity: the host does not
// know more) go without the tiles.  The FFN, without and with them: 128 experts of
// 2048 x 768, 8 rows on average 115 and 130 us, 12: 129 and 133, 16: 141 and 134; 64
// experts of 2048 x 2048, 8 rows 164 and 173, 16: 198 and 179.
constexpr int kSkinnyRows = 12;

// Small products go without the tiles too, which would leave most CUs idle, with several
// workgroups for the rows of an expert, 64 at a time.  What then counts are the rows of
// K that the workgroups read: each weight row once for every block of rows, each row once
// for every 32 weight rows (as many as there may be: the host knows the capacity).  Products with and without tiles: 777
// rows of 5 experts, 1040 x 528 (23 thousand) 12.8 and 6.4 us; 2000 of 8, 1024 x 512 (53)
// 11.9 and 9.1; 512 of one, 2048 x 2048 (52) 16.7 and 13.9; 700 of one (68) 16.8 and
// 19.2; 777 of 5 (87) 17.3 and 23.1.
constexpr long kSkinnyReads = 60000;
constexpr int kFewBlocks = 1024;  // (expert, block) pairs of a launch, as far as experts allow

template <bool GU>
hipError_t launch_product(const ProductI8& p, int R_cap, int kernel_id, hipStream_t s) {
  ProfScope ps(kernel_id, s);
  const long experts = std::min(p.E_l, R_cap), wrows = (long)p.N * (GU ? 2 : 1);
  const bool few = R_cap <= kSkinnyRows * experts;
  if (few || wrows * (experts + R_cap / kFew + (R_cap + 8 * experts) / 32) <= kSkinnyReads) {
    const int split = split_of(p.K), cols = kFewWaves / split * few_cols<GU>();
    const int blocks = few ? 1 : std::min((R_cap + kFew - 1) / kFew, kFewBlocks / (int)experts);
    const dim3 grid((p.N + cols - 1) / cols, (int)experts, blocks);
    if (split == 4) skinny_i8_kernel<GU, 4><<<grid, 256, 0, s>>>(p);
    else skinny_i8_kernel<GU, 2><<<grid, 256, 0, s>>>(p);
  } else {
    tile_i8_kernel<GU><<<kCUs, 64 * kTileWaves, kTileLds, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const int8_t* x, const float* xs, const int32_t* src, int x_rows,
                          const int32_t* offsets, int E_l, int R_cap, int K, int N, const int8_t* w,
                          const float* ws, bf16_t* y, hipStream_t s) {
  const ProductI8 p = {x, xs, src, x_rows, offsets, E_l, K, N, w, nullptr, ws, nullptr, y, nullptr};
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
  const ProductI8 up = {x, xs, src, x_rows, offsets, E_l, H, I, wg, wu, wgs, wus, h, nullptr};
  hipError_t e = launch_product<true>(up, R_cap, MOE_KERNEL_FFN_GATEUP_I8, s);
  if (e != hipSuccess) return e;
  const ProductI8 down = {hq, hs, nullptr, R_cap, offsets, E_l, I, H, wd, nullptr, wds, nullptr, y, h};
  if ((long)R_cap <= (long)kFusedRows * E_l && I <= kFusedCols) {
    ProfScope ps(MOE_KERNEL_FFN_DOWN_I8, s);
    const int cols = kFewWaves / kFusedSplit * few_cols<false>();
    const dim3 grid((H + cols - 1) / cols, std::min(E_l, R_cap));
    skinny_quantize_i8_kernel<<<grid, 256, 16 * I, s>>>(down);
    return hipGetLastError();
  }
  e = launch_quantize_i8(h, R_cap, I, I, true, offsets + E_l, hq, hs, s);
  if (e != hipSuccess) return e;
  return launch_product<false>(down, R_cap, MOE_KERNEL_FFN_DOWN_I8, s);
}

}  // namespace moe
