// Low-rank adapters of many requests beside a shared projection, for gfx950.
//
// Row r with adapter a = row_id[r] (rows without one are left alone):
//   forward   v_r = s_a A_a x_r,  y_r += B_a v_r
//   backward  w_r = s_a B_a^T dy_r,  dx_r += A_a^T w_r,
//             dA_a = sum_r w_r x_r^T,  dB_a = sum_r dy_r v_r^T
// The backward's data part is the forward on transposed weights (B_a^T in the
// place of A_a, A_a^T in the place of B_a), so one kernel does both.
//
// A fragment of the matrix instruction is 16 bytes per lane in both types: row
// (or column) lane % 16, 16-byte chunk lane / 16 of the summed axis.  bf16
// takes 8 values and one 16x16x32 instruction, fp32 4 values and four 16x16x4
// instructions (instruction i sums element i of every chunk).  Any order of
// the summed axis is right as long as both operands share it.
#include "common.h"

#include <algorithm>

namespace moe {

namespace {

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

template <bool BF16>
struct Elem {
  static constexpr int EB = BF16 ? 2 : 4;
  static constexpr int CE = BF16 ? 8 : 4;  // values of one 16-byte chunk
  static constexpr int KE = 4 * CE;        // summed values of one fragment step
};

__device__ __forceinline__ u32x4_t load16(const char* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}

// d += a b^T over one fragment step.
template <bool BF16>
__device__ __forceinline__ f32x4_t step(u32x4_t a, u32x4_t b, f32x4_t d) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), d, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), d, 0,
                                               0, 0);
    return d;
  }
}

// ---------------------------------------------------------------------------
// rows in adapter order (for the weight gradients)
// ---------------------------------------------------------------------------

// Rows of one adapter in row order, cut into chunks of `chunk`: an adapter of
// one chunk (or no row) writes its gradient whole, one of more writes fp32
// partials that a second pass adds in chunk order.  count = chunks in all, each
// {id, begin, end, slot}.
struct ChunkPlan {
  int32_t* count;
  int32_t* chunks;   // [upper][4]
  int32_t* first;    // [n_ids] first slot of an id of several chunks
  int32_t* offsets;  // [n_ids + 1] rows of an id in the order list
};

// The adapter of row r, or -1, by the forward's rule.
struct RowIds {
  const int32_t* row_id;
  const int32_t* src_row;
  int R, x_rows, n_ids;
  __device__ __forceinline__ int operator()(int r) const {
    const int a = row_id[r], s = src_row != nullptr ? src_row[r] : r;
    return a >= 0 && a < n_ids && s >= 0 && s < x_rows ? a : -1;
  }
};

constexpr int kSortBlocks = 128;  // at most, so that a block adds few counts
int sort_rows(int R) {
  return R <= 2048 ? (R + 255) / 256 * 256 + 256 * (R == 0) : max(1024, ((R + kSortBlocks - 1) / kSortBlocks + 255) / 256 * 256);
}

// Inclusive prefix sum over the first 256 threads of a workgroup (s: a word per
// wave).
__device__ __forceinline__ int block_scan(int v, int* s) {
  const int lane = lane_id(), wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int x = __shfl_up(v, o, kWave);
    v += lane >= o ? x : 0;
  }
  if (lane == kWave - 1) s[wave] = v;
  lds_barrier();
#pragma unroll
  for (int w = 0; w < 3; ++w) v += w < wave ? s[w] : 0;
  return v;
}

// What the backward needs to order the rows by adapter.
struct RowOrder {
  RowIds ids;
  int per, nblk;    // rows of a block, blocks
  int32_t* counts;  // [nblk][n_ids] rows of each adapter (more than one block)
  int chunk;
  ChunkPlan plan;
  int32_t* order;   // out
};

// The rows in adapter order, rows of one adapter in row order: every block adds
// the counts of the blocks before it (and all, for the adapters' offsets), its
// four waves take a quarter of its rows each, 64 at a time, and a row's place
// is its wave's cursor for the adapter plus the lanes before it that have the
// same.  The first block also writes the chunks.  Waves after the fourth only
// keep the barriers; mem: kOrderLds bytes of LDS.
constexpr int kOrderLds = 4 * (4 * kMaxE + 3 * 8);
static_assert(kMaxE == 256, "a thread per adapter");
__device__ __forceinline__ void order_block(const RowOrder& o, int b, char* mem) {
  int(*s_cur)[kMaxE] = reinterpret_cast<int(*)[kMaxE]>(mem);
  int *s_t = reinterpret_cast<int*>(mem) + 4 * kMaxE, *s_n = s_t + 8, *s_m = s_n + 8;
  const RowIds& ids = o.ids;
  const ChunkPlan& plan = o.plan;
  const int per = o.per, nblk = o.nblk, chunk = o.chunk;
  const int32_t* counts = o.counts;
  int32_t* order = o.order;
  const int tid = threadIdx.x, wave = tid >> 6, lane = lane_id();
  int before = 0, all = 0;
  if (nblk > 1 && tid < ids.n_ids) {
#pragma unroll 8
    for (int i = 0; i < nblk; ++i) {
      const int c = counts[(size_t)i * ids.n_ids + tid];
      before += i < b ? c : 0;
      all += c;
    }
  }
  const bool key = tid < kMaxE;  // this thread's adapter is tid
  if (key)
#pragma unroll
    for (int w = 0; w < 4; ++w) s_cur[w][tid] = 0;
  __syncthreads();
  const int q = (per + 3) / 4;  // rows of a wave
  const int r0 = b * per + wave * q, r1 = wave < 4 ? min(min(ids.R, (b + 1) * per), r0 + q) : r0;
  constexpr int KR = 8;  // 64-row steps of a wave whose adapters stay in registers
  int keep[KR];
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int r = r0 + j * kWave + lane;
    keep[j] = r < r1 ? ids(r) : -1;
  }
#pragma unroll
  for (int j = 0; j < KR; ++j)
    if (keep[j] >= 0) atomicAdd(&s_cur[wave][keep[j]], 1);
  for (int r = r0 + KR * kWave + lane; r < r1; r += kWave) {
    const int a = ids(r);
    if (a >= 0) atomicAdd(&s_cur[wave][a], 1);
  }
  if (nblk <= 1) {
    lds_barrier();
    if (key)
#pragma unroll
      for (int w = 0; w < 4; ++w) all += s_cur[w][tid];
  }
  const int end = block_scan(all, s_t), begin = end - all;
  int at = begin + before;
  if (key)
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // counts of the waves to their cursors
      const int n = s_cur[w][tid];
      s_cur[w][tid] = at;
      at += n;
    }
  __syncthreads();
  auto place = [&](int r, int a) {
    int rank = 0, same_n = 0;
    for (uint64_t todo = __ballot(a >= 0); todo != 0;) {
      const int cur = __builtin_amdgcn_readlane(a, __builtin_ctzll(todo));
      const uint64_t same = __ballot(a == cur);
      todo &= ~same;
      if (a == cur) {
        rank = __popcll(same & ((1ull << lane) - 1ull));
        same_n = __popcll(same);
      }
    }
    const int from = a >= 0 ? s_cur[wave][a] : 0;
    asm volatile("" ::: "memory");  // a wave's LDS accesses complete in order
    if (a >= 0) {
      order[from + rank] = r;
      if (rank == 0) s_cur[wave][a] = from + same_n;
    }
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j < KR; ++j)
    if (r0 + j * kWave < r1) place(r0 + j * kWave + lane, keep[j]);
  for (int rb = r0 + KR * kWave; rb < r1; rb += kWave)
    place(rb + lane, rb + lane < r1 ? ids(rb + lane) : -1);
  if (b != 0) return;
  // the chunks, and the slots of adapters of several
  const int n = tid < ids.n_ids ? max(1, (all + chunk - 1) / chunk) : 0;
  const int m = n > 1 ? n : 0;
  const int n_end = block_scan(n, s_n), m_end = block_scan(m, s_m);
  if (tid == kMaxE - 1) *plan.count = n_end;
  if (tid >= ids.n_ids) return;
  plan.offsets[tid] = begin;
  if (tid == ids.n_ids - 1) plan.offsets[tid + 1] = end;
  const int slot = m_end - m;
  plan.first[tid] = slot;
  for (int c = 0; c < n; ++c) {
    int32_t* e = plan.chunks + 4 * (size_t)(n_end - n + c);
    e[0] = tid;
    e[1] = begin + c * chunk;
    e[2] = min(end, begin + (c + 1) * chunk);
    e[3] = n > 1 ? slot + c : -1;
  }
}

__global__ __launch_bounds__(256) void adapter_order_kernel(RowOrder o) {
  __shared__ __align__(16) char mem[kOrderLds];
  order_block(o, blockIdx.x, mem);
}

// ---------------------------------------------------------------------------
// forward and data gradients
// ---------------------------------------------------------------------------

struct AdapterArgs {
  const char* x;            // [x_rows][ldx]
  const int32_t* src_row;   // token row of row r, or null: r
  int gather;               // x holds token rows: row r is x[src_row[r]]
  const int32_t* row_id;    // [R]
  const char* a;            // [n_ids][rank][K]
  const char* b;            // [n_ids][N][rank]
  const float* scale;       // [n_ids] or null: 1
  char* y;                  // [R][ldy], added to (null: v alone)
  float* v;                 // [R][rank] or null
  long ldx, ldy;
  int x_rows, R, K, N, n_ids, rank;
  int rows, splits;         // rows of a workgroup, column ranges per row tile
  int window;               // whether mixed rows are regrouped by adapter
};

// 64 lanes x 16 bytes from per-lane global addresses to LDS at lds + 16 * lane.
// Inline asm, as in the grouped GEMMs: the compiler keeps no count of these
// loads; the explicit vmcnt waits below order every access.
__device__ __forceinline__ void dma16g(const char* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// LDS of one wave of adapter_kernel, in bytes: two stages of the first
// product's operands, whose place the partial sums, the second product's
// results and a set of B's columns take afterwards.  For small ranks another
// set of B's columns behind them, loaded before the first product and then in
// turn with the other (TWO).
template <bool BF16, int RT, int MT>
struct AdapterLds {
  static constexpr int ST = 2048 * (MT + RT);               // a stage: 128 bytes of every row
  static constexpr int RL = 16 * RT + 4;                    // pitch of the rank values (floats)
  static constexpr int RED = 16 * MT * RL * 4;              // partial sums
  static constexpr int DL = 68;                             // pitch of the results (floats)
  static constexpr int DELTA = 16 * DL * 4;                 // 16 rows x 64 columns
  static constexpr int JB = (BF16 ? 2 : 4) * RT;            // KB of 64 columns of B at most
  static constexpr bool TWO = BF16 && RT <= 2;
  static constexpr int B1 = RED + DELTA;
  static constexpr int FIRST = 2 * ST > B1 + 1024 * JB ? 2 * ST : B1 + 1024 * JB;
  static constexpr int B0 = TWO ? FIRST : B1;
  static constexpr int WAVE = FIRST + (TWO ? 1024 * JB : 0);
};

constexpr int kWindow = 512;      // rows regrouped together
constexpr int kWindowKeys = 256;  // adapters (at most 255) and the rows without one

// Rows in mixed order: every adapter among a workgroup's rows is a pass of its
// own, so 16 rows of 16 adapters cost 16 passes.  Where 64 neighbours sampled
// from a window of rows say that runs of one adapter are shorter than 8 rows on
// average (mixed_rows: every wave asks the same 128 rows, so all workgroups of
// the window agree), the window's workgroups share its rows out sorted by
// adapter, by a stable counting sort in LDS that each of them does alike.
// Which workgroup takes a row changes no bit of its result.  8191 rows of 64
// adapters, mixed: 39 us, 75 without.
__device__ __forceinline__ bool mixed_rows(const AdapterArgs& p, int row0) {
  const int r = min(row0 / kWindow * kWindow + kWindow / kWave * lane_id(), p.R - 1);
  return __popcll(__ballot(p.row_id[r] != p.row_id[min(r + 1, p.R - 1)])) > kWave / 8;
}

template <int NW>
__device__ __forceinline__ void regroup(const AdapterArgs& p, int row0, char* lds, int& row) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int base = row0 / kWindow * kWindow;
  constexpr int Q = kWindow / NW;  // rows of a wave
  uint16_t* s_ord = reinterpret_cast<uint16_t*>(lds);
  int* s_cur = reinterpret_cast<int*>(lds + 2 * kWindow);  // [NW][kWindowKeys]
  int key[Q / kWave];
#pragma unroll
  for (int j = 0; j < Q / kWave; ++j) {
    const int r = base + wave * Q + j * kWave + lane;
    const int a = r < p.R ? p.row_id[r] : -1;
    key[j] = a >= 0 && a < p.n_ids ? a : kWindowKeys - 1;
  }
  for (int i = threadIdx.x; i < NW * kWindowKeys; i += NW * kWave) s_cur[i] = 0;
  lds_barrier();
#pragma unroll
  for (int j = 0; j < Q / kWave; ++j) atomicAdd(&s_cur[wave * kWindowKeys + key[j]], 1);
  lds_barrier();
  if (wave == 0) {  // counts to cursors, by key and then by wave
    constexpr int KL = kWindowKeys / kWave;
    int n[KL], sum = 0;
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      n[i] = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) n[i] += s_cur[w * kWindowKeys + KL * lane + i];
      sum += n[i];
    }
    int end = sum;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int x = __shfl_up(end, o, kWave);
      end += lane >= o ? x : 0;
    }
    int at = end - sum;
#pragma unroll
    for (int i = 0; i < KL; ++i)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        int* c = &s_cur[w * kWindowKeys + KL * lane + i];
        const int m = *c;
        *c = at;
        at += m;
      }
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < Q / kWave; ++j) {
    int rank = 0, same_n = 0;
    for (uint64_t todo = ~0ull; todo != 0;) {
      const int cur = __builtin_amdgcn_readlane(key[j], __builtin_ctzll(todo));
      const uint64_t same = __ballot(key[j] == cur);
      todo &= ~same;
      if (key[j] == cur) {
        rank = __popcll(same & ((1ull << lane) - 1ull));
        same_n = __popcll(same);
      }
    }
    int* c = &s_cur[wave * kWindowKeys + key[j]];
    const int from = *c;
    asm volatile("" ::: "memory");  // a wave's LDS accesses complete in order
    s_ord[from + rank] = (uint16_t)(wave * Q + j * kWave + lane);
    if (rank == 0) *c = from + same_n;
    asm volatile("" ::: "memory");
  }
  lds_barrier();
  if (lane < p.rows) row = base + s_ord[row0 - base + lane];
  lds_barrier();  // read by all before the LDS is used otherwise
}

// A workgroup of NW waves takes `rows` <= 16 MT rows and one of `splits`
// column ranges of y.  First A_a x for its rows, the summed axis cut over the
// waves and added through LDS in wave order; then the waves go over the
// columns 64 at a time.  Every distinct adapter among the rows is a pass over
// the rows that have it: lanes of other rows compute on a row of this adapter
// and are not used, so nothing of one request's adapter or activations reaches
// another's row.
//
// Bound by the reads of x, the read and write of y and, for few rows per
// adapter, the weights.  A fragment wants 16 rows in neighbouring lanes, and
// loaded like that every lane quad touches four cache lines, which the L1's
// tag lookups serve at a quarter of their rate (8191 rows, rank 64: 40 us).  So
// everything is loaded with a row's 128 bytes in eight neighbouring lanes: x,
// A and B straight into the wave's own LDS (16-byte chunk c of row r at place
// c ^ (r % 8): fragment reads hit all banks), y into registers, where the
// second product's results meet it through LDS.  No barrier: only the wave
// that loaded reads.
//
// ORDER, in a backward with weight gradients: the first `oblocks` workgroups (a
// multiple of 8, the XCDs) order the rows by adapter instead, for the launches
// after this one (8285 rows: one launch of 5 us less; 1003 rows: 2.7 us less than
// in the launch before).
template <bool BF16, int RT, int MT, int NW, bool ORDER>
__global__ __launch_bounds__(NW* kWave) void adapter_kernel(AdapterArgs p, int oblocks, RowOrder o) {
  using E = Elem<BF16>;
  using S = AdapterLds<BF16, RT, MT>;
  constexpr int RL = S::RL;
  extern __shared__ __align__(16) char lds[];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15, g = lane >> 4;
  if constexpr (ORDER) {
    if ((int)blockIdx.x < oblocks) {
      if ((int)blockIdx.x < o.nblk) order_block(o, blockIdx.x, lds);
      return;
    }
  }
  const int nob = ORDER ? oblocks : 0;
  const int bid = xcd_remap(blockIdx.x - nob, gridDim.x - nob);
  const int tile = bid / p.splits, split = bid % p.splits;
  const int row0 = tile * p.rows;

  // lane i: the workgroup's row i, its adapter, scale and x row
  int row = row0 + lane, id = -1, xr = 0;
  float scale = 1.f;
  auto look = [&]() {
    id = -1;
    if (lane >= p.rows || row >= p.R) return;
    id = p.row_id[row];
    xr = p.src_row != nullptr ? p.src_row[row] : row;
  };
  look();
  if (p.window && mixed_rows(p, row0)) {
    regroup<NW>(p, row0, lds, row);
    look();
  }
  if (id < 0 || id >= p.n_ids || xr < 0 || xr >= p.x_rows) id = -1;
  if (!p.gather) xr = row;
  if (id >= 0 && p.scale != nullptr) scale = p.scale[id];
  const uint64_t live = __ballot(id >= 0);
  if (live == 0) {
    if (p.v != nullptr && split == 0)
      for (int i = 0; i < p.rows; ++i) {
        const int r = __builtin_amdgcn_readlane(row, i);
        if (r >= p.R) continue;
        for (int j = threadIdx.x; j < p.rank; j += NW * kWave) p.v[(size_t)r * p.rank + j] = 0.f;
      }
    return;
  }
  int idm[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) idm[m] = __shfl(id, 16 * m + l, kWave);
  char* my = lds + wave * S::WAVE;
  const uint32_t my_lds = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t*)my);

  // ---- operands of the second product: 64 columns of y and of an adapter's B
  constexpr int YR = 64 / (64 / E::CE);  // rows of y in one load: 64 columns are 64 / CE lanes
  constexpr int YL = 64 / E::CE;
  constexpr int NYI = 16 * MT / YR;      // loads of y
  const int per = ((p.N + 63) / 64 + p.splits - 1) / p.splits * 64;
  const int n1 = p.y != nullptr ? min(p.N, (split + 1) * per) : 0;
  char* yrow[NYI];
  bool yon[NYI];
#pragma unroll
  for (int j = 0; j < NYI; ++j) {
    const int r = YR * j + lane / YL;
    yon[j] = __shfl(id, r, kWave) >= 0;
    // a row without an adapter reads one that has, and is not written
    yrow[j] = p.y + (size_t)__shfl(row, yon[j] ? r : __builtin_ctzll(live), kWave) * p.ldy * E::EB;
  }
  const int yc = lane % YL * E::CE;  // this lane's first column of the 64
  auto load_y = [&](u32x4_t (&y)[NYI], int nb) {
#pragma unroll
    for (int j = 0; j < NYI; ++j)
      y[j] = load16(yrow[j] + (size_t)min(nb + yc, n1 - E::CE) * E::EB);
  };
  // B's 64 rows of rank values lie one after another: chunk p of the block is
  // chunk p % rc of row p / rc, at LDS place p with the chunk swizzled by the
  // row so that 16 rows' chunks spread over the banks
  const int rc = p.rank / E::CE;
  const int jb = p.rank / (BF16 ? 8 : 4);  // KB of the block
  const int sw = min(rc & -rc, 8);
  const int sh = __builtin_ctz(8 / sw);
  auto swz = [&](int n, int c) { return c ^ ((n >> sh) & (sw - 1)); };
  int boff[S::JB];
#pragma unroll
  for (int j = 0; j < S::JB; ++j) {
    const int q = 64 * j + lane, n = q / rc;
    boff[j] = (n * rc + swz(n, q - n * rc)) * 16;
  }
  auto load_b = [&](int at, int nb, int cur) {
    const char* base = p.b + (size_t)cur * p.N * p.rank * E::EB;
    const long first = (long)nb * p.rank * E::EB, last = (long)p.N * p.rank * E::EB - 16;
#pragma unroll
    for (int j = 0; j < S::JB; ++j)
      if (j < jb) dma16g(base + min(first + boff[j], last), my_lds + at + 1024 * j);
  };
  const int cur0 = __builtin_amdgcn_readlane(id, __builtin_ctzll(live));
  int nb = split * per + 64 * wave;
  u32x4_t y[NYI];
  if (nb < n1) {
    if (S::TWO) load_b(S::B0, nb, cur0);
    load_y(y, nb);
  }

  // ---- first product
  f32x4_t tot[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) tot[m][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // The wave's part of the summed axis in stages of 128 bytes a row (two
  // fragment steps), the next two in flight; the last wave also takes what is
  // behind the last whole stage.
  constexpr int GE = 2 * E::KE;
  constexpr int NI = 2 * (MT + RT);  // loads of a stage, 8 rows each
  const int stages = p.K / GE;
  const int s0 = wave * stages / NW, s1 = (wave + 1) * stages / NW;
  const bool tail = wave == NW - 1 && stages * GE < p.K;
  for (uint64_t todo = live; todo != 0;) {
    const int first = __builtin_ctzll(todo);
    const int cur = __builtin_amdgcn_readlane(id, first);
    const int xfirst = __builtin_amdgcn_readlane(xr, first);
    todo &= ~__ballot(id == cur);
    const int xs = id == cur ? xr : xfirst;
    const char* ab = p.a + (size_t)cur * p.rank * p.K * E::EB;
    f32x4_t acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[m][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    u32x4_t tx[2][MT], ta[2][RT];
    if (tail) {  // loaded before the stages, multiplied after them
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = min(stages * GE + u * E::KE + g * E::CE, p.K - E::CE);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          tx[u][m] = load16(p.x + ((size_t)__shfl(xs, 16 * m + l, kWave) * p.ldx + k) * E::EB);
#pragma unroll
        for (int r = 0; r < RT; ++r)
          ta[u][r] = load16(ab + ((size_t)min(16 * r + l, p.rank - 1) * p.K + k) * E::EB);
      }
    }
    if (s0 < s1) {
      const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
      const char* src[NI];
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j)
        src[j] = p.x + (size_t)__shfl(xs, 8 * j + (lane >> 3), kWave) * p.ldx * E::EB + chunk;
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j)  // rank values past the last are not used
        src[2 * MT + j] = ab + (size_t)(8 * min(j, p.rank / 8 - 1) + (lane >> 3)) * p.K * E::EB + chunk;
      auto issue = [&](int s) {
        const uint32_t dst = my_lds + (s & 1) * S::ST;
#pragma unroll
        for (int j = 0; j < NI; ++j) dma16g(src[j] + 128 * (size_t)s, dst + 1024 * j);
      };
      auto read = [&](int s, u32x4_t (&x)[2][MT], u32x4_t (&a)[2][RT]) {
        const char* st = my + (s & 1) * S::ST;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = l * 128 + ((4 * u + g) ^ (l & 7)) * 16;
#pragma unroll
          for (int m = 0; m < MT; ++m) x[u][m] = load16(st + 2048 * m + at);
#pragma unroll
          for (int r = 0; r < RT; ++r) a[u][r] = load16(st + 2048 * (MT + r) + at);
        }
      };
      auto multiply = [&](const u32x4_t (&x)[2][MT], const u32x4_t (&a)[2][RT]) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[m][r] = step<BF16>(a[u][r], x[u][m], acc[m][r]);
      };
      u32x4_t xf[2][MT], af[2][RT];
      wait_lds_reads();  // an earlier adapter's stages have been read
      issue(s0);
      if (s0 + 1 < s1) issue(s0 + 1);
      for (int s = s0; s + 1 < s1; ++s) {
        wait_vm<NI>();  // stage s has landed, s + 1 is in flight
        read(s, xf, af);
        wait_lds_reads();
        if (s + 2 < s1) issue(s + 2);
        multiply(xf, af);
      }
      wait_vm<0>();
      read(s1 - 1, xf, af);
      multiply(xf, af);
    }
    if (tail) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool in = stages * GE + u * E::KE + g * E::CE < p.K;  // behind the end: zeros on both sides
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[m][r] = step<BF16>(in ? ta[u][r] : u32x4_t{}, in ? tx[u][m] : u32x4_t{}, acc[m][r]);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[m][r][i] = idm[m] == cur ? acc[m][r][i] : tot[m][r][i];
  }
  // tot[m][r][i] = this wave's part of value 16 r + 4 g + i of row 16 m + l
  float* red = reinterpret_cast<float*>(my);
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if (16 * m + l < p.rows)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        *reinterpret_cast<f32x4_t*>(red + (16 * m + l) * RL + 16 * r + 4 * g) = tot[m][r];
  lds_barrier();
  for (int i0 = wave * kWave; i0 < p.rows * 4 * RT; i0 += NW * kWave) {
    const int i = i0 + lane;
    const int t = min(i / (4 * RT), p.rows - 1), j = 4 * (i % (4 * RT));
    const float f = __shfl(scale, t, kWave);
    const int r = __shfl(row, t, kWave);
    const bool on = (live >> t & 1) != 0;
    if (i >= p.rows * 4 * RT) continue;
    float* r0 = reinterpret_cast<float*>(lds) + t * RL + j;
    f32x4_t s = *reinterpret_cast<f32x4_t*>(r0);
#pragma unroll
    for (int w = 1; w < NW; ++w) s += *reinterpret_cast<f32x4_t*>(r0 + w * S::WAVE / 4);
    s = on ? s * f : f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (p.v != nullptr && split == 0 && r < p.R && j < p.rank)
      *reinterpret_cast<f32x4_t*>(p.v + (size_t)r * p.rank + j) = s;
    *reinterpret_cast<f32x4_t*>(r0) = s;
  }
  if (p.y == nullptr) return;
  lds_barrier();

  // The rank values (in the first wave's place) as fragments.  bf16 holds each
  // fp32 value whole as three bf16 parts (8 bits each), three instructions on the
  // same weights: the products are exact and the sums fp32, like those of the
  // fp32 path.  (Two parts, 16 of the 24 bits, gain 0 to 2 %: 8191 rows of rank 64
  // 27.6 us for 28.2.)
  constexpr int KF = BF16 ? (RT + 1) / 2 : RT;  // fragment steps of the rank values
  constexpr int NP = BF16 ? 3 : 1;
  u32x4_t vf[NP][MT][KF];
#pragma unroll
  for (int s = 0; s < KF; ++s)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool on = 4 * s + g < rc && idm[m] >= 0;
      const float* vr = reinterpret_cast<const float*>(lds) + min(16 * m + l, p.rows - 1) * RL +
                        min(4 * s + g, rc - 1) * E::CE;
      float v[E::CE];
#pragma unroll
      for (int i = 0; i < E::CE; i += 4)
        *reinterpret_cast<f32x4_t*>(v + i) = *reinterpret_cast<const f32x4_t*>(vr + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
          // an infinity is in the first part alone
          auto rest = [](float x, float part) {
            const float r = x - part;
            return __builtin_isfinite(r) ? r : 0.f;
          };
          float r0 = v[2 * i], r1 = v[2 * i + 1];
#pragma unroll
          for (int h = 0; h < NP; ++h) {
            const float p0 = bf2f(f2bf(r0)), p1 = bf2f(f2bf(r1));
            vf[h][m][s][i] = on ? pack_bf2(p0, p1) : 0u;
            r0 = rest(r0, p0);
            r1 = rest(r1, p1);
          }
        } else {
          vf[0][m][s][i] = on ? __float_as_uint(v[i]) : 0u;
        }
      }
    }

  // ---- second product
  int bfr[4][KF];  // this lane's chunk of row 16 q + l of B in step s
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int s = 0; s < KF; ++s) {
      const int n = 16 * q + l;
      bfr[q][s] = (n * rc + swz(n, min(4 * s + g, rc - 1))) * 16;
    }
  float* delta = reinterpret_cast<float*>(my + S::RED);
  int at = S::B0;
  for (; nb < n1; nb += 64 * NW) {
    if (!S::TWO) load_b(at, nb, cur0);
    wait_vm<0>();  // the block's B and y
    u32x4_t yn[NYI];
    const bool more = nb + 64 * NW < n1;
    const int atn = S::TWO && at == S::B0 ? S::B1 : S::B0;
    if (more) {  // the next block's, before this one's products
      if (S::TWO) load_b(atn, nb + 64 * NW, cur0);
      load_y(yn, nb + 64 * NW);
    }
    f32x4_t d[4][MT];
    bool loaded = true;
    for (uint64_t todo = live; todo != 0;) {
      const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      todo &= ~__ballot(id == cur);
      if (!loaded) {
        wait_lds_reads();
        load_b(at, nb, cur);
        wait_vm<0>();
      }
      loaded = false;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u32x4_t w[KF];
#pragma unroll
        for (int s = 0; s < KF; ++s) {
          w[s] = load16(my + at + bfr[q][s]);
          w[s] = 4 * s + g < rc ? w[s] : u32x4_t{};
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KF; ++s)
#pragma unroll
            for (int h = 0; h < NP; ++h) acc = step<BF16>(w[s], vf[h][m][s], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[q][m][i] = idm[m] == cur ? acc[i] : d[q][m][i];
        }
      }
    }
    // d[q][m][i]: column 16 q + 4 g + i of row 16 m + l, to y's lanes
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(delta + l * S::DL + 16 * q + 4 * g) = d[q][m];
      asm volatile("" ::: "memory");  // a wave's LDS accesses complete in order
#pragma unroll
      for (int j = m * (16 / YR); j < (m + 1) * (16 / YR); ++j) {
        const float* dr = delta + (YR * j + lane / YL - 16 * m) * S::DL + yc;
        u32x4_t v = y[j];
        if constexpr (BF16) {
          const f32x4_t d0 = *reinterpret_cast<const f32x4_t*>(dr);
          const f32x4_t d1 = *reinterpret_cast<const f32x4_t*>(dr + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4_t& t = i < 2 ? d0 : d1;
            const int k = 2 * (i % 2);
            v[i] = pack_bf2(__uint_as_float(v[i] << 16) + t[k],
                            __uint_as_float(v[i] & 0xffff0000u) + t[k + 1]);
          }
        } else {
          const f32x4_t d0 = *reinterpret_cast<const f32x4_t*>(dr);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + d0[i]);
        }
        if (yon[j] && nb + yc < n1)
          *reinterpret_cast<u32x4_t*>(yrow[j] + (size_t)(nb + yc) * E::EB) = v;
      }
      asm volatile("" ::: "memory");  // a wave's LDS accesses complete in order
    }
    wait_lds_reads();  // this block's B has been read before it is loaded over
    if (more)
#pragma unroll
      for (int j = 0; j < NYI; ++j) y[j] = yn[j];
    at = atn;
  }
}

template <bool BF16, int RT, int MT, int NW>
hipError_t launch_one(const AdapterArgs& p, const RowOrder& o, hipStream_t s) {
  constexpr int lds = NW * AdapterLds<BF16, RT, MT>::WAVE;
  static_assert(lds <= 160 * 1024, "the LDS of one CU");
  static_assert(NW < 4 || lds >= kOrderLds, "the order's LDS");
  const int tiles = (p.R + p.rows - 1) / p.rows;
  if (NW >= 4 && o.nblk > 0) {
    const int oblocks = (o.nblk + 7) / 8 * 8;
    adapter_kernel<BF16, RT, MT, NW, NW >= 4><<<oblocks + tiles * p.splits, NW * kWave, lds, s>>>(p, oblocks, o);
    return hipGetLastError();
  }
  adapter_kernel<BF16, RT, MT, NW, false><<<tiles * p.splits, NW * kWave, lds, s>>>(p, 0, o);
  if (o.nblk > 0) adapter_order_kernel<<<o.nblk, 256, 0, s>>>(o);
  return hipGetLastError();
}

// Rows of a workgroup and column ranges.  More rows share one read of an
// adapter's weights, more column ranges repeat the first product, and fewer
// than one workgroup per CU leaves CUs idle: the choice is the one whose
// busiest CU moves the fewest elements, with the adapters among `rows` rows
// taken as twice those of rows sorted by adapter (1 .. rows).  Up to 16 rows
// (one tile): 32 rows gain 2 % at 131072 sorted rows (217 us for 222) and lose
// on 8191 rows in mixed order (165 us for 73) and on 8285 sorted ones (24 for
// 21).  Above rank 64, where the weights are most of the traffic, 32 (8191 rows
// of rank 128: 44 us for 65).
// Eight waves where there are few workgroups (2048 rows: 10.6 us for 13.3 with
// four), four where a CU takes several in turn (131072 rows: 222 us for 243) or
// where two workgroups of eight do not fit its LDS (8191 rows of rank 64: 29 us
// for 34).
struct AdapterTiles {
  int rows, splits, waves;
  long wgs;
};
template <bool BF16, int RT>
struct AdapterWaves {
  static constexpr int MT = RT <= 4 ? 1 : 2;
  static constexpr int WAVE = AdapterLds<BF16, RT, MT>::WAVE;
  static constexpr bool EIGHT = 8 * WAVE <= 160 * 1024;
  static constexpr int FEW = 4 * WAVE <= 160 * 1024 ? 4 : 2;
  static int of(long wgs) { return EIGHT && wgs <= (8 * WAVE <= 80 * 1024 ? 4 : 1) * kCUs ? 8 : FEW; }
};
template <bool BF16>
AdapterTiles adapter_tiles(int R, int K, int N, int n_ids, int rank, bool y) {
  AdapterTiles t{};
  const int most = rank > 64 ? 32 : 16;
  double best = 0.0;
  for (int rows = 1; rows <= most; rows *= 2)
    for (int splits = 1; splits <= (y ? 8 : 1); splits *= 2) {
      if (splits > 1 && 256 * splits > N) break;
      const long tiles = ((long)R + rows - 1) / rows;
      const double ids = (double)std::clamp(2L * rows * n_ids / R, 1L, (long)rows) * rank;
      const double each = (rows + ids) * K + (ids + 2.0 * rows) * N / splits;
      const double cost = (double)((tiles * splits + kCUs - 1) / kCUs) * each;
      if (best > 0.0 && cost > best) continue;
      best = cost;
      t = {rows, splits, 0, tiles * splits};
    }
  const int rt = (rank + 15) / 16;
  t.waves = rt <= 1   ? AdapterWaves<BF16, 1>::of(t.wgs)
            : rt <= 2 ? AdapterWaves<BF16, 2>::of(t.wgs)
            : rt <= 4 ? AdapterWaves<BF16, 4>::of(t.wgs)
                      : AdapterWaves<BF16, 8>::of(t.wgs);
  return t;
}

template <bool BF16>
hipError_t launch_adapter(AdapterArgs p, const RowOrder& o, hipStream_t s) {
  const AdapterTiles t = adapter_tiles<BF16>(p.R, p.K, p.N, p.n_ids, p.rank, p.y != nullptr);
  p.rows = t.rows;
  p.splits = t.splits;
  p.window = p.rows > 1 && p.n_ids > 1 && p.n_ids < kWindowKeys;
  const int rt = (p.rank + 15) / 16;
#define MOE_AD(RT)                                                                     \
  do {                                                                                 \
    using W = AdapterWaves<BF16, RT>;                                                  \
    if constexpr (W::EIGHT)                                                            \
      if (t.waves == 8) return launch_one<BF16, RT, W::MT, 8>(p, o, s);                \
    return launch_one<BF16, RT, W::MT, W::FEW>(p, o, s);                               \
  } while (0)
  if (rt <= 1) MOE_AD(1);
  else if (rt <= 2) MOE_AD(2);
  else if (rt <= 4) MOE_AD(4);
  else MOE_AD(8);
#undef MOE_AD
}

// ---------------------------------------------------------------------------
// weight gradients
// ---------------------------------------------------------------------------

// First launch of the backward, two independent parts.
//  - Both transposed weights, A [ids][rank][K] -> [ids][K][rank] and
//    B [ids][N][rank] -> [ids][rank][N]: a thread turns a block of 16 bytes of
//    ranks x CW columns in registers, so both sides move whole lane-contiguous
//    words.
//  - Counts of the rows of each adapter in blocks of rows, for the order list
//    (where there are several).
template <bool BF16>
__global__ __launch_bounds__(256) void adapter_prepare_kernel(const char* __restrict__ A,
                                                              const char* __restrict__ B, int rank,
                                                              int K, int N, char* __restrict__ At,
                                                              char* __restrict__ Bt, int tblocks,
                                                              RowOrder o) {
  using E = Elem<BF16>;
  constexpr int CW = 4 / E::EB;  // columns of one 4-byte word
  const RowIds& ids = o.ids;
  if ((int)blockIdx.x >= tblocks) {
    __shared__ int s_n[kMaxE];
    for (int i = threadIdx.x; i < ids.n_ids; i += 256) s_n[i] = 0;
    __syncthreads();
    const int b = blockIdx.x - tblocks, r1 = min(ids.R, (b + 1) * o.per);
    for (int r = b * o.per + threadIdx.x; r < r1; r += 256) {
      const int a = ids(r);
      if (a >= 0) atomicAdd(&s_n[a], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ids.n_ids; i += 256) o.counts[(size_t)b * ids.n_ids + i] = s_n[i];
    return;
  }
  const int ka = K / CW, kn = N / CW, rc = rank / E::CE;  // words, chunks
  const long unit = (long)blockIdx.x * 256 + threadIdx.x;
  const long each = (long)(ka + kn) * rc;
  if (unit >= each * ids.n_ids) return;
  const long id = unit / each;
  int i = (int)(unit - id * each);
  const bool second = i >= ka * rc;
  if (second) i -= ka * rc;
  const int cols = second ? N : K, cw = second ? kn : ka;
  const int j = i / cw * E::CE, c = i % cw * CW;  // first rank value, first column
  const size_t base = (size_t)id * rank * cols * E::EB;
  // wide[c]: 16 bytes of ranks of column c (rows of B and of A^T);
  // word[j]: 4 bytes of columns of rank value j (rows of A and of B^T)
  u32x4_t wide[CW];
  uint32_t word[E::CE];
  const char* src = (second ? B : A) + base;
  char* dst = (second ? Bt : At) + base;
  if (second) {
#pragma unroll
    for (int u = 0; u < CW; ++u) wide[u] = load16(src + ((size_t)(c + u) * rank + j) * E::EB);
  } else {
#pragma unroll
    for (int u = 0; u < E::CE; ++u)
      word[u] = *reinterpret_cast<const uint32_t*>(src + ((size_t)(j + u) * cols + c) * E::EB);
  }
  if constexpr (BF16) {
    if (second) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t x = wide[0][u / 2] >> (16 * (u % 2)), y = wide[1][u / 2] >> (16 * (u % 2));
        word[u] = (x & 0xffffu) | (y << 16);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        wide[0][u] = (word[2 * u] & 0xffffu) | (word[2 * u + 1] << 16);
        wide[1][u] = (word[2 * u] >> 16) | (word[2 * u + 1] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (second) word[u] = wide[0][u]; else wide[0][u] = word[u];
    }
  }
  if (second) {
#pragma unroll
    for (int u = 0; u < E::CE; ++u)
      *reinterpret_cast<uint32_t*>(dst + ((size_t)(j + u) * cols + c) * E::EB) = word[u];
  } else {
#pragma unroll
    for (int u = 0; u < CW; ++u)
      *reinterpret_cast<u32x4_t*>(dst + ((size_t)(c + u) * rank + j) * E::EB) = wide[u];
  }
}

struct WgradArgs {
  const float* p[2];         // [R][rank]: w (for dA), v (for dB)
  const char* q[2];          // x rows (through src_row), dy rows
  const int32_t* src_row;    // of q[0]
  const int32_t* order;      // rows in adapter order
  float* out[2];             // dA [n_ids][rank][K], dB [n_ids][N][rank]
  float* part;               // [slots][rank (K + N)]
  ChunkPlan plan;
  long ldq[2];
  int C[2];                  // K, N
  int nb0;                   // 256-column blocks of the first product
  int rank, accumulate;
};

constexpr int kWgMaxChunk = 1024;

// G = sum over a chunk's rows of p_r q_r^T: the rows are the summed axis.
//
// The wide factor: a wave holds 64 columns, lane l the columns 4 l .. 4 l + 3
// of the rows of its 16-lane group g; loaded row by row (128 contiguous bytes
// of a bf16 row per group, the next step's while this one is multiplied), the
// eight rows of a lane are put together per column by 16-bit permutes.
// The narrow fp32 factor: SB rows at a time, turned to [value][row] in LDS
// once for the four waves.  bf16 takes it as three bf16 parts (24 bits), so the
// products are exact and the sums fp32 like those of the fp32 path.
// Bound by the reads of the wide factor (HBM, and the L2 for gathered rows).
//
// SPLIT (wgrad_split), for up to kWgMaxChunk rows in all (every adapter is one chunk) and rank
// up to 32: the four waves of a workgroup hold the same 64 columns and take the
// steps of a staged block in turn; their sums meet in LDS, in wave order.  As
// many waves as chunks of 128 rows give, without the second launch.
template <bool BF16, int RT>
struct WgradLds {
  static constexpr int SB = RT <= 2 ? 128 : RT == 4 ? 64 : 32;  // rows of a staged block
  static constexpr int NP = BF16 ? 3 : 1;
  static constexpr int PITCH = SB * (BF16 ? 2 : 4) + 16;        // bytes of one value's rows
  static constexpr int BYTES = NP * 16 * RT * PITCH;
};

template <bool BF16, int RT, bool SPLIT>
__global__ __launch_bounds__(256) void adapter_wgrad_kernel(WgradArgs a) {
  using S = WgradLds<BF16, RT>;
  constexpr int SR = BF16 ? 32 : 16;  // rows of one step
  constexpr int LR = SR / 4;          // rows of a lane
  constexpr int SB = S::SB;
  constexpr int IT = 16 * RT * SB / 8 / 256;  // (value, 8 rows) pairs of a thread
  typedef uint32_t word_t __attribute__((ext_vector_type(BF16 ? 2 : 4)));
  __shared__ __align__(16) int s_row[kWgMaxChunk], s_q[kWgMaxChunk];
  __shared__ __align__(16) char s_p[2][S::BYTES];
  if ((int)blockIdx.x >= *a.plan.count) return;
  const int32_t* e = a.plan.chunks + 4 * (size_t)blockIdx.x;
  const int id = e[0], begin = e[1], n = e[2] - e[1], slot = e[3];
  const int z = (int)blockIdx.y >= a.nb0 ? 1 : 0;
  const int C = a.C[z];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, l = lane & 15, g = lane >> 4;
  const int c0 = SPLIT ? 64 * ((int)blockIdx.y - z * a.nb0) + 4 * l
                       : 256 * ((int)blockIdx.y - z * a.nb0) + 64 * wave + 4 * l;
  const float* P = a.p[z];
  const char* Q = a.q[z] + (size_t)min(c0, C - 4) * (BF16 ? 2 : 4);
  const size_t ldq = (size_t)a.ldq[z] * (BF16 ? 2 : 4);
  f32x4_t acc[RT][4];  // tile q: columns 4 l' + q
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[r][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (n > 0) {
    // the list to a whole staged block, the last row again behind the end
    const int np = (n + SB - 1) / SB * SB;
    for (int i = tid; i < np; i += 256) {
      const int r = a.order[begin + min(i, n - 1)];
      s_row[i] = r;
      s_q[i] = z == 0 && a.src_row != nullptr ? a.src_row[r] : r;
    }
    __syncthreads();
    float pv[IT][8];
    auto load_p = [&](int i0) {
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int j = (tid + 256 * t) % (16 * RT), o = (tid + 256 * t) / (16 * RT) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          pv[t][i] = P[(size_t)s_row[i0 + o + i] * a.rank + min(j, a.rank - 1)];
      }
    };
    auto store_p = [&](int i0, char* to) {
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int j = (tid + 256 * t) % (16 * RT), o = (tid + 256 * t) / (16 * RT) * 8;
        float v[8], h[8], m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i0 + o + i < n ? pv[t][i] : 0.f;
        char* at = to + j * S::PITCH;
        if constexpr (BF16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[i] = bf2f(f2bf(v[i]));
            const float r = v[i] - h[i];
            m[i] = bf2f(f2bf(r));
            v[i] = r - m[i];
          }
          const float* parts[3] = {h, m, v};
#pragma unroll
          for (int p = 0; p < 3; ++p)
            *reinterpret_cast<u32x4_t*>(at + p * 16 * RT * S::PITCH + o * 2) =
                u32x4_t{pack_bf2(parts[p][0], parts[p][1]), pack_bf2(parts[p][2], parts[p][3]),
                        pack_bf2(parts[p][4], parts[p][5]), pack_bf2(parts[p][6], parts[p][7])};
        } else {
          *reinterpret_cast<f32x4_t*>(at + o * 4) = f32x4_t{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f32x4_t*>(at + o * 4 + 16) = f32x4_t{v[4], v[5], v[6], v[7]};
        }
      }
    };
    auto load_q = [&](word_t (&raw)[LR], int i0) {
#pragma unroll
      for (int i = 0; i < LR; ++i)
        raw[i] = *reinterpret_cast<const word_t*>(Q + (size_t)s_q[i0 + LR * g + i] * ldq);
    };
    auto multiply = [&](word_t (&raw)[LR], int i0, const char* sp) {
      if (i0 + SR > n)  // rows behind the end: zeros on both sides
#pragma unroll
        for (int i = 0; i < LR; ++i)
          if (i0 + LR * g + i >= n) raw[i] = word_t{};
      const char* at = sp + l * S::PITCH + (i0 % SB + LR * g) * (BF16 ? 2 : 4);
      if constexpr (BF16) {
        u32x4_t col[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = raw[2 * i][h], y = raw[2 * i + 1][h];
            col[2 * h][i] = __builtin_amdgcn_perm(y, x, 0x05040100u);      // the low halves
            col[2 * h + 1][i] = __builtin_amdgcn_perm(y, x, 0x07060302u);  // the high halves
          }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const u32x4_t f = load16(at + (p * RT + r) * 16 * S::PITCH);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[r][q] = step<true>(f, col[q], acc[r][q]);
          }
      } else {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const f32x4_t f = *reinterpret_cast<const f32x4_t*>(at + r * 16 * S::PITCH);
#pragma unroll
          for (int i = 0; i < LR; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[r][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[i], __uint_as_float(raw[i][q]),
                                                               acc[r][q], 0, 0, 0);
        }
      }
    };
    if constexpr (SPLIT) {
      constexpr int NS = SB / SR / 4;  // a wave's steps of a staged block
      static_assert(NS * SR * 4 == SB, "the waves share a block's steps out evenly");
      word_t q0[NS][LR], q1[NS][LR];
      auto load = [&](word_t (&q)[NS][LR], int b0) {
#pragma unroll
        for (int i = 0; i < NS; ++i) load_q(q[i], b0 + (wave + 4 * i) * SR);
      };
      auto block = [&](word_t (&q)[NS][LR], word_t (&next)[NS][LR], int b0) {
        const bool more = b0 + SB < np;
        if (more) {
          load_p(b0 + SB);
          load(next, b0 + SB);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NS; ++i) multiply(q[i], b0 + (wave + 4 * i) * SR, s_p[b0 / SB & 1]);
        if (more) store_p(b0 + SB, s_p[(b0 / SB + 1) & 1]);
        __syncthreads();
      };
      load_p(0);
      load(q0, 0);
      store_p(0, s_p[0]);
      __syncthreads();
      for (int b0 = 0; b0 < np; b0 += 2 * SB) {
        block(q0, q1, b0);
        if (b0 + SB < np) block(q1, q0, b0 + SB);
      }
    } else {
      word_t q0[LR], q1[LR];
      load_p(0);
      load_q(q0, 0);
      store_p(0, s_p[0]);
      __syncthreads();
      for (int b0 = 0; b0 < np; b0 += SB) {
        const char* sp = s_p[b0 / SB & 1];
        const bool more = b0 + SB < np;
        if (more) load_p(b0 + SB);
#pragma unroll
        for (int u = 0; u < SB / SR; u += 2) {
          const int i0 = b0 + u * SR;
          if (SB / SR > 1) {
            load_q(q1, i0 + SR);
            __builtin_amdgcn_sched_barrier(0);
            multiply(q0, i0, sp);
            if (u + 2 < SB / SR || more) load_q(q0, i0 + 2 * SR);
            __builtin_amdgcn_sched_barrier(0);
            multiply(q1, i0 + SR, sp);
          } else {
            if (more) load_q(q1, i0 + SR);
            multiply(q0, i0, sp);
#pragma unroll
            for (int i = 0; i < LR; ++i) q0[i] = q1[i];
          }
        }
        if (more) {
          store_p(b0 + SB, s_p[(b0 / SB + 1) & 1]);
          __syncthreads();
        }
      }
    }
  }
  if constexpr (SPLIT) {
    // acc of wave w: [w][r][q][i][lane], of which each wave adds a quarter
    static_assert(4 * 16 * RT * kWave * 4 <= sizeof(s_p), "the sums of four waves");
    float* sum = reinterpret_cast<float*>(s_p) + lane;
    auto at = [&](int w, int r, int q, int i) -> float& {
      return sum[(((w * RT + r) * 4 + q) * 4 + i) * kWave];
    };
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) at(wave, r, q, i) = acc[r][q][i];
    lds_barrier();
    if (c0 >= C) return;
    float* out = a.out[z] + (size_t)id * a.rank * C;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int j = 16 * r + 4 * g;
      if (j >= a.rank) continue;
      // z = 0, [rank][K]: four columns of rank value j + wave
      // z = 1, [N][rank]: four rank values of column c0 + wave
      float* o = z == 0 ? out + (size_t)(j + wave) * C + c0 : out + (size_t)(c0 + wave) * a.rank + j;
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += z == 0 ? at(w, r, i, wave) : at(w, r, wave, i);
      if (a.accumulate) v += *reinterpret_cast<const f32x4_t*>(o);
      *reinterpret_cast<f32x4_t*>(o) = v;
    }
    return;
  }
  if (c0 >= C) return;
  // acc[r][q][i]: rank value 16 r + 4 g + i, column c0 + q
  float* out;
  const bool add = slot < 0 && a.accumulate;
  if (slot >= 0)
    out = a.part + (size_t)slot * a.rank * (a.C[0] + a.C[1]) + (z ? (size_t)a.rank * a.C[0] : 0);
  else
    out = a.out[z] + (size_t)id * a.rank * C;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int j = 16 * r + 4 * g;
    if (j >= a.rank) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x4_t v;
      float* o;
      if (z == 0) {  // [rank][K]: four columns of one rank value
        v = f32x4_t{acc[r][0][i], acc[r][1][i], acc[r][2][i], acc[r][3][i]};
        o = out + (size_t)(j + i) * C + c0;
      } else {  // [N][rank]: four rank values of one column
        v = acc[r][i];
        o = out + (size_t)(c0 + i) * a.rank + j;
      }
      if (add) v += *reinterpret_cast<const f32x4_t*>(o);
      *reinterpret_cast<f32x4_t*>(o) = v;
    }
  }
}

// Gradients of the adapters of several chunks: their partials in chunk order.
__global__ __launch_bounds__(256) void adapter_wgrad_sum_kernel(
    int chunk, ChunkPlan plan, const f32x4_t* __restrict__ part, int rank, int K, int N,
    int accumulate, f32x4_t* __restrict__ dA, f32x4_t* __restrict__ dB) {
  const int id = blockIdx.y;
  const int n = (plan.offsets[id + 1] - plan.offsets[id] + chunk - 1) / chunk;
  if (n <= 1) return;
  const int ka = rank * K / 4, all = rank * (K + N) / 4;  // 16-byte groups
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  f32x4_t* o = i < ka ? dA + (size_t)id * ka + i : dB + (size_t)id * (all - ka) + (i - ka);
  f32x4_t v = accumulate ? *o : f32x4_t{0.f, 0.f, 0.f, 0.f};
  const f32x4_t* q = part + (size_t)plan.first[id] * all + i;
  constexpr int U = 8;  // partials in flight
  for (int c0 = 0; c0 < n; c0 += U) {
    f32x4_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = q[(size_t)min(c0 + u, n - 1) * all];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < n) v += t[u];
  }
  *o = v;
}

// Adapter of grouped row r: that of its token, of its expert.
__global__ __launch_bounds__(256) void adapter_rows_kernel(const int32_t* __restrict__ offsets,
                                                           const int32_t* __restrict__ src_row,
                                                           const int32_t* __restrict__ token_adapter,
                                                           int E_l, int T, int n_adapters, int R_cap,
                                                           int32_t* __restrict__ row_id) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= R_cap) return;
  int id = -1;
  if (r < offsets[E_l]) {
    const int t = src_row[r];
    const int a = t >= 0 && t < T ? token_adapter[t] : -1;
    if (a >= 0 && a < n_adapters) {
      int lo = 0, hi = E_l - 1;  // the last expert whose rows begin at or before r
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (offsets[mid] <= r) lo = mid; else hi = mid - 1;
      }
      id = a * E_l + lo;
    }
  }
  row_id[r] = id;
}

// h[r] = SiLU(g[r]) u[r] from the g, u that the adapters changed (bf16: the
// stored, rounded ones); rows without an adapter keep the product's h.
template <bool BF16>
__global__ __launch_bounds__(256) void adapter_swiglu_kernel(const char* __restrict__ gu, RowIds ids,
                                                             int I, char* __restrict__ h) {
  using E = Elem<BF16>;
  const int r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= ids.R || ids(r) < 0) return;
  const char* g = gu + (size_t)r * 2 * I * E::EB;
  const char* u = g + (size_t)I * E::EB;
  char* o = h + (size_t)r * I * E::EB;
  auto act = [](float a, float b) { return a / (1.f + expf(-a)) * b; };
  for (int c = lane_id() * 16; c < I * E::EB; c += kWave * 16) {
    const u32x4_t a = load16(g + c), b = load16(u + c);
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16)
        v[i] = pack_bf2(act(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16)),
                        act(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u)));
      else
        v[i] = __float_as_uint(act(__uint_as_float(a[i]), __uint_as_float(b[i])));
    }
    *reinterpret_cast<u32x4_t*>(o + c) = v;
  }
}

// Workgroups of the weight gradients with one chunk for every adapter.
long wgrad_units(int K, int N, int n_ids) { return (long)n_ids * ((K + 255) / 256 + (N + 255) / 256); }

// Few rows and too few workgroups: the waves of a workgroup share an adapter's
// rows out.  (Backward of 1024 rows of 5 adapters, 2048 x 2048, rank 16: 20 us,
// 23 in chunks; 600 rows of rank 8, 512 x 256: 14.4 for 16.8.  With one adapter of
// 1024 rows 21 for 18.6, with 64 adapters, whose workgroups are many, 43 for 38.)
bool wgrad_split(int R, int K, int N, int n_ids, int rank) {
  return R <= kWgMaxChunk && R <= 512L * n_ids && rank <= 32 && wgrad_units(K, N, n_ids) < 256;
}

// Rows of a chunk, whole staged blocks: about 700 workgroups of the weight
// gradients, so that a CU has a few and the partial sums stay few (32768 rows
// of one adapter: 159 us for the backward, 204 with a third of the rows).  Up to
// 512 rows of enough adapters are not cut, which spares the second launch (512
// rows of 32 adapters, 2048 x 2048: 27 us for 29).
int wgrad_chunk(int R, int K, int N, int n_ids, int rank) {
  if (wgrad_split(R, K, N, n_ids, rank)) return kWgMaxChunk;
  if (R <= 512 && wgrad_units(K, N, n_ids) >= 256) return 512;
  const long blocks = (K + 255) / 256 + (N + 255) / 256;
  const long c = (R * blocks / 700 + 127) / 128 * 128;
  return (int)std::clamp(c, 128L, (long)kWgMaxChunk);
}

// Threads of the transposes.
uint64_t transpose_units(int n_ids, int rank, int K, int N, int eb) {
  return (uint64_t)n_ids * (rank * eb / 16) * ((K + N) * (long)eb / 4);
}

struct BwdLayout {
  size_t at, bt, w, counts, order, count, chunks, first, offsets, part, total;
  int chunk, upper;
};

BwdLayout bwd_layout(int R, int K, int N, int n_ids, int rank, int eb) {
  BwdLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t was = at; at += up256(bytes); return was; };
  l.chunk = wgrad_chunk(R, K, N, n_ids, rank);
  l.upper = R / l.chunk + n_ids;
  l.at = take((size_t)n_ids * rank * K * eb);
  l.bt = take((size_t)n_ids * rank * N * eb);
  l.w = take((size_t)R * rank * 4);
  l.counts = take((size_t)((R + sort_rows(R) - 1) / sort_rows(R)) * n_ids * 4);
  l.order = take((size_t)R * 4);
  l.count = take(4);
  l.chunks = take((size_t)l.upper * 16);
  l.first = take((size_t)n_ids * 4);
  l.offsets = take((size_t)(n_ids + 1) * 4);
  l.part = take((size_t)(2 * (R / l.chunk)) * rank * (K + N) * 4);
  l.total = at;
  return l;
}

}  // namespace

uint64_t adapter_fwd_threads(bool bf16, int R, int K, int N, int n_ids, int rank, bool y) {
  if (R < 1 << 19) return (uint64_t)R * 8 * 512;  // at most a workgroup for each row and column range
  const AdapterTiles t = bf16 ? adapter_tiles<true>(R, K, N, n_ids, rank, y)
                              : adapter_tiles<false>(R, K, N, n_ids, rank, y);
  return (uint64_t)t.wgs * t.waves * kWave;
}

uint64_t adapter_bwd_threads(bool bf16, int R, int K, int N, int n_ids, int rank, bool dx) {
  const uint64_t data = adapter_fwd_threads(bf16, R, N, K, n_ids, rank, dx) + kSortBlocks * 512;
  const uint64_t prepare = transpose_units(n_ids, rank, K, N, bf16 ? 2 : 4) + 256 * (kSortBlocks + 1);
  return std::max(data, prepare);  // (HIP's own max takes int)
}

size_t adapter_bwd_ws_bytes(int R, int K, int N, int n_ids, int rank, int elem_bytes) {
  return bwd_layout(R, K, N, n_ids, rank, elem_bytes).total;
}

hipError_t launch_adapter_rows(const int32_t* offsets, const int32_t* src_row,
                               const int32_t* token_adapter, int E_l, int T, int n_adapters,
                               int R_cap, int32_t* row_id, hipStream_t s) {
  adapter_rows_kernel<<<(R_cap + 255) / 256, 256, 0, s>>>(offsets, src_row, token_adapter, E_l, T,
                                                          n_adapters, R_cap, row_id);
  return hipGetLastError();
}

hipError_t launch_adapter_swiglu(const void* gu, const int32_t* row_id, const int32_t* src_row,
                                 int R, int x_rows, int n_ids, int I, bool bf16, void* h,
                                 hipStream_t s) {
  const RowIds ids = {row_id, src_row, R, x_rows, n_ids};
  if (bf16)
    adapter_swiglu_kernel<true><<<(R + 3) / 4, 256, 0, s>>>((const char*)gu, ids, I, (char*)h);
  else
    adapter_swiglu_kernel<false><<<(R + 3) / 4, 256, 0, s>>>((const char*)gu, ids, I, (char*)h);
  return hipGetLastError();
}

hipError_t launch_adapter_fwd(const AdapterShape& d, const void* x, const int32_t* src_row,
                              const int32_t* row_id, const void* A, const void* B,
                              const float* scale, void* y, float* v, hipStream_t s) {
  AdapterArgs p{};
  p.x = (const char*)x;
  p.src_row = src_row;
  p.gather = src_row != nullptr;
  p.row_id = row_id;
  p.a = (const char*)A;
  p.b = (const char*)B;
  p.scale = scale;
  p.y = (char*)y;
  p.v = v;
  p.ldx = d.ldx;
  p.ldy = d.ldy;
  p.x_rows = d.x_rows;
  p.R = d.R;
  p.K = d.K;
  p.N = d.N;
  p.n_ids = d.n_ids;
  p.rank = d.rank;
  ProfScope ps(MOE_KERNEL_ADAPTER, s);
  const RowOrder none{};
  return d.bf16 ? launch_adapter<true>(p, none, s) : launch_adapter<false>(p, none, s);
}

hipError_t launch_adapter_bwd(const AdapterShape& d, const void* dy, const void* x,
                              const int32_t* src_row, const int32_t* row_id, const void* A,
                              const void* B, const float* v, const float* scale, void* dx,
                              long lddx, float* dA, float* dB, bool accumulate, void* ws,
                              hipStream_t s) {
  const int eb = d.bf16 ? 2 : 4;
  const BwdLayout l = bwd_layout(d.R, d.K, d.N, d.n_ids, d.rank, eb);
  char* w = (char*)ws;
  const int per = sort_rows(d.R);
  const RowOrder o = {{row_id, src_row, d.R, d.x_rows, d.n_ids},
                      per,
                      dA != nullptr ? (d.R + per - 1) / per : 0,
                      (int32_t*)(w + l.counts),
                      l.chunk,
                      {(int32_t*)(w + l.count), (int32_t*)(w + l.chunks), (int32_t*)(w + l.first),
                       (int32_t*)(w + l.offsets)},
                      (int32_t*)(w + l.order)};
  hipError_t e = hipSuccess;
  if (d.R > 0) {
    const int tblocks = (int)((transpose_units(d.n_ids, d.rank, d.K, d.N, eb) + 255) / 256);
    const int grid = tblocks + (o.nblk > 1 ? o.nblk : 0);
    if (d.bf16)
      adapter_prepare_kernel<true><<<grid, 256, 0, s>>>((const char*)A, (const char*)B, d.rank, d.K,
                                                        d.N, w + l.at, w + l.bt, tblocks, o);
    else
      adapter_prepare_kernel<false><<<grid, 256, 0, s>>>((const char*)A, (const char*)B, d.rank, d.K,
                                                         d.N, w + l.at, w + l.bt, tblocks, o);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // the data part: the forward from dy's rows to dx's on the transposed weights
    AdapterArgs p{};
    p.x = (const char*)dy;
    p.src_row = src_row;  // not followed: names the rows that have none
    p.row_id = row_id;
    p.a = w + l.bt;
    p.b = w + l.at;
    p.scale = scale;
    p.y = (char*)dx;
    p.v = (float*)(w + l.w);
    p.ldx = d.ldy;
    p.ldy = lddx;
    p.x_rows = d.x_rows;
    p.R = d.R;
    p.K = d.N;
    p.N = d.K;
    p.n_ids = d.n_ids;
    p.rank = d.rank;
    ProfScope ps(MOE_KERNEL_ADAPTER_DGRAD, s);
    e = d.bf16 ? launch_adapter<true>(p, o, s) : launch_adapter<false>(p, o, s);
    if (e != hipSuccess) return e;
  }
  if (dA == nullptr) return e;
  if (d.R == 0) {  // the chunks alone
    adapter_order_kernel<<<1, 256, 0, s>>>(o);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  WgradArgs a{};
  a.p[0] = (const float*)(w + l.w);
  a.p[1] = v;
  a.q[0] = (const char*)x;
  a.q[1] = (const char*)dy;
  a.src_row = src_row;
  a.order = (const int32_t*)(w + l.order);
  a.out[0] = dA;
  a.out[1] = dB;
  a.part = (float*)(w + l.part);
  a.plan = o.plan;
  a.ldq[0] = d.ldx;
  a.ldq[1] = d.ldy;
  a.C[0] = d.K;
  a.C[1] = d.N;
  const bool split = wgrad_split(d.R, d.K, d.N, d.n_ids, d.rank);
  const int cols = split ? 64 : 256;  // of a workgroup
  a.nb0 = (d.K + cols - 1) / cols;
  a.rank = d.rank;
  a.accumulate = accumulate ? 1 : 0;
  const dim3 grid(l.upper, a.nb0 + (d.N + cols - 1) / cols);
  const int rt = (d.rank + 15) / 16;
  {
    ProfScope ps(MOE_KERNEL_ADAPTER_WGRAD, s);
#define MOE_WG(RT, SP)                                                       \
  do {                                                                       \
    if (d.bf16) adapter_wgrad_kernel<true, RT, SP><<<grid, 256, 0, s>>>(a);  \
    else adapter_wgrad_kernel<false, RT, SP><<<grid, 256, 0, s>>>(a);        \
  } while (0)
    if (split) { if (rt <= 1) MOE_WG(1, true); else MOE_WG(2, true); }
    else if (rt <= 1) MOE_WG(1, false);
    else if (rt <= 2) MOE_WG(2, false);
    else if (rt <= 4) MOE_WG(4, false);
    else MOE_WG(8, false);
#undef MOE_WG
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (d.R <= l.chunk) return e;  // no adapter has more than one chunk
  adapter_wgrad_sum_kernel<<<dim3((d.rank * (d.K + d.N) / 4 + 255) / 256, d.n_ids), 256, 0, s>>>(
      l.chunk, o.plan, (const f32x4_t*)(w + l.part), d.rank, d.K, d.N, accumulate ? 1 : 0, (f32x4_t*)dA,
      (f32x4_t*)dB);
  return hipGetLastError();
}

}  // namespace moe
