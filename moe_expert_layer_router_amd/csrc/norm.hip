// RMS norms around the expert layer for gfx950: the residual update with the
// norm before the layer, and the combine with the norm after it, its gate and
// the scaled residual; each with its backward.
//
//   before:  r = x + delta,  n = xh w,  xh = r / sqrt(mean r^2 + eps)
//   after:   c = sum_j w_j y_perm[dest_j],  y = rs residual + gate xh weight,
//            xh = c / sqrt(mean c^2 + eps)
// Backward, for the gradient g of xh (dn w, or dy gate weight) and 1/rms = s:
//   d(r or c) = s (g - xh mean(g xh)),  d weight = sum over rows of (dn or dy gate) xh
// Both sums of a row, of squares and of g times the row, come from one pass, so
// nothing but the inputs is kept from the forward: the backward of "after" reads
// the grouped rows for the gate weights' gradient anyway and forms c again.
//
// A row belongs to a team of W waves, each lane of which holds NC chunks of 16
// bytes of it between its sums and its stores, so each matrix of token rows crosses
// the memory once, which is what bounds all four.  So does y_perm in the backward of
// "after" while a token's local slots are no more than a lane can hold: 8 slots for
// rows of up to 512 chunks (4096 bf16 or 2048 fp32 columns), 4 up to twice and 2 up to
// four (fp32: eight) times that; tokens with more read their grouped rows twice.  The registers of
// four waves a SIMD do not hold all of it everywhere: the compiler spills 4 to 22 of them with
// 8 slots of bf16 (11 for the 2048 columns below), 7 with 4 slots of 8192 columns, 47 and 85
// (bf16, fp32) with 16384 columns, whose norm_bwd_kernel spills 21 and 59.
// 16384 tokens of 2048 bf16 columns, top-8, moved bytes over time: before 47 us, 5.7
// TB/s, its backward 56 us, 4.8 TB/s; after 114 us, 5.9 TB/s, its backward 233 us,
// 4.9 TB/s, with 5 us behind each backward for the sum of the partial rows (a copy of
// 1 GiB reaches 5.0, a fill 6.9).
#include <algorithm>

#include "rows.h"

namespace moe {

namespace {

// Sums of M values (a power of two) over a wave's lanes: lane l gets that of value
// l M / 64.  Halves of the lanes take halves of the values first, so that M values cost
// M - 1 + log2(64 / M) exchanges in place of 6 M.
template <int M>
__device__ __forceinline__ float wave_sums(float (&v)[M]) {
  const int lane = lane_id();
  int o = kWave / 2;
#pragma unroll
  for (int m = M / 2; m > 0; m /= 2, o /= 2) {
    const bool high = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float keep = high ? v[i + m] : v[i], give = high ? v[i] : v[i + m];
      v[i] = keep + __shfl_xor(give, o, kWave);
    }
  }
  float sum = v[0];
#pragma unroll
  for (; o > 0; o /= 2) sum += __shfl_xor(sum, o, kWave);
  return sum;
}

// Sums of M values over the W waves of a team, in a fixed order; every lane gets
// them.  A workgroup with teams of several waves calls it from all its threads.
// The waves' sums meet in lds [W waves of each team][M]; the caller keeps two
// calls on the same lds apart by a barrier (a call on another lds has one).
template <int W, int M>
__device__ __forceinline__ void team_sum(float (&v)[M], float* lds) {
  constexpr int kLanes = kWave / M;  // with the same sum
  const float mine = wave_sums(v);
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  if constexpr (W > 1) {
    if (lane % kLanes == 0) lds[wave * M + lane / kLanes] = mine;
    lds_barrier();
  }
#pragma unroll
  for (int i = 0; i < M; ++i) {
    v[i] = W > 1 ? 0.f : __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), i * kLanes));
    if constexpr (W > 1) {
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += lds[(wave / W * W + w) * M + i];
    }
  }
}

// The same where one thread wants each sum: returns that of value `which` in the lanes
// where `has` is set.
template <int W, int M>
__device__ __forceinline__ float team_sum_apart(float (&v)[M], float* lds, int& which, bool& has) {
  constexpr int kLanes = kWave / M;
  float sum = wave_sums(v);
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  which = lane / kLanes;
  has = lane % kLanes == 0;
  if constexpr (W > 1) {
    if (has) lds[wave * M + which] = sum;
    lds_barrier();
    which = lane % M;
    has = threadIdx.x % (W * kWave) < M;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += lds[(wave / W * W + w) * M + which];
  }
  return sum;
}

// The sum of a row from each lane's sums v of its chunks: over 64 neighbouring chunks
// first, then four of those, then the rest, each in the row's order, so that its bits do
// not depend on how many waves hold the row.  lds [waves][NC].
template <int W, int NC>
__device__ __forceinline__ float row_sum(float (&v)[NC], float* lds) {
  constexpr int kAll = W * NC;
  float all[kAll], sum = 0.f;
#pragma unroll
  for (int u = 0; u < NC; ++u) v[u] = wave_sum(v[u]);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    if (lane_id() == 0) {
#pragma unroll
      for (int u = 0; u < NC; ++u) lds[wave * NC + u] = v[u];
    }
    lds_barrier();
  }
#pragma unroll
  for (int i = 0; i < kAll; ++i) all[i] = W > 1 ? lds[(threadIdx.x >> 6) / W * kAll + i] : v[i % NC];
#pragma unroll
  for (int i = 0; i < kAll; i += 4) {
    float four = all[i];
#pragma unroll
    for (int q = i + 1; q < i + 4 && q < kAll; ++q) four += all[q];
    sum += four;
  }
  return sum;
}

constexpr int threads_of(int W) { return W > 4 ? W * kWave : 256; }

// Where a lane's chunks lie: chunk(u) = first + 64 u of the row's nch.
template <int W, int NC>
struct Place {
  int team, first;  // team in the workgroup
  __device__ Place() {
    const int wave = threadIdx.x >> 6;
    team = wave / W;
    first = (wave % W) * kWave * NC + lane_id();
  }
  static constexpr int kTeams = threads_of(W) / (W * kWave);
};

template <bool BF16, int W, int NC>
__global__ __launch_bounds__(threads_of(W)) void norm_kernel(
    const void* x, const void* delta, const float* __restrict__ weight, float eps, int T, int H,
    void* r, void* __restrict__ n) {
  using R = Row<BF16>;
  __shared__ float lds[threads_of(W) / kWave];
  const Place<W, NC> at;
  const int t = blockIdx.x * at.kTeams + at.team;
  if (W == 1 && t >= T) return;  // (a team of several waves is the whole workgroup or has a row below)
  const bool live = t < T;
  const int nch = H / R::N;
  float v[NC][R::N];
  u32x4_t raw[NC], add[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
    const size_t e = (size_t)t * H + (size_t)c * R::N;
    raw[u] = live && c < nch ? R::ld_s(x, e) : u32x4_t{};
    add[u] = live && c < nch && delta != nullptr ? R::ld_s(delta, e) : u32x4_t{};
  }
  // One wave a row fetches the weights beside the row (16384 x 2048 48.5 -> 47.1 us);
  // with several the registers cost more than the wait (8192 fp32 x 2048 42.8 -> 44.0).
  constexpr bool kAhead = W == 1;
  float wt[kAhead ? NC : 1][R::N];
  if constexpr (kAhead) {
#pragma unroll
    for (int u = 0; u < NC; ++u)
#pragma unroll
      for (int i = 0; i < R::N; ++i) wt[u][i] = weight[min(at.first + u * kWave, nch - 1) * R::N + i];
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    if (delta != nullptr) {
      float a[R::N], b[R::N];
      R::to_f32(raw[u], a);
      R::to_f32(add[u], b);
#pragma unroll
      for (int i = 0; i < R::N; ++i) a[i] += b[i];
      raw[u] = R::from_f32(a);  // the norm reads the sum as it is stored
    }
    R::to_f32(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < R::N; ++i) ss[0] = fmaf(v[u][i], v[u][i], ss[0]);
  }
  team_sum<W>(ss, lds);
  const float s = 1.f / sqrtf(ss[0] / (float)H + eps);
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
    if (!live || c >= nch) continue;
    const size_t e = (size_t)t * H + (size_t)c * R::N;
    if (delta != nullptr) R::st_s(r, e, raw[u]);
    float o[R::N];
#pragma unroll
    for (int i = 0; i < R::N; ++i) o[i] = v[u][i] * s * (kAhead ? wt[kAhead ? u : 0][i] : weight[c * R::N + i]);
    R::st(n, e, R::from_f32(o));  // read next by the router and the products
  }
}

// Adds the column sums that the teams of a workgroup hold (dw, a lane's chunks)
// in team order and writes them as the workgroup's partial row, or, where it is the
// only one, as (or to) the sums themselves.
template <bool BF16, int W, int NC>
__device__ __forceinline__ void write_partial(const Place<W, NC>& at, int nch, int H,
                                              float (&dw)[NC][Row<BF16>::N], float* __restrict__ part,
                                              float* __restrict__ only, int accumulate, float* lds) {
  constexpr int N = Row<BF16>::N;
  constexpr int kTeams = Place<W, NC>::kTeams;
  constexpr int kRow = W * kWave * NC * N;  // elements a team covers
  float* row = gridDim.x == 1 ? only : part + (size_t)blockIdx.x * H;
  const bool add = gridDim.x == 1 && accumulate != 0;
  if constexpr (kTeams > 1) {
    __syncthreads();
    if (at.team > 0) {
#pragma unroll
      for (int u = 0; u < NC; ++u)
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<f32x4_t*>(lds + (at.team - 1) * kRow + (at.first + u * kWave) * N + i) =
              f32x4_t{dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]};
    }
    __syncthreads();
    if (at.team > 0) return;
  }
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
    if (c >= nch) continue;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      f32x4_t v = {dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]};
#pragma unroll
      for (int m = 1; m < kTeams; ++m)
        v += *reinterpret_cast<const f32x4_t*>(lds + (m - 1) * kRow + c * N + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) row[c * N + i + q] = add ? row[c * N + i + q] + v[q] : v[q];
    }
  }
}

template <bool BF16, int W, int NC>
constexpr int partial_lds() {
  return Place<W, NC>::kTeams > 1 ? (Place<W, NC>::kTeams - 1) * W * kWave * NC * Row<BF16>::N : 1;
}

// dx = rs dr + s (g - xh mean(g xh)), g = dn w; the rows' dn xh added up per column.
template <bool BF16, int W, int NC>
__global__ __launch_bounds__(threads_of(W)) void norm_bwd_kernel(
    const void* dn, const void* dr, float rs, const void* __restrict__ r,
    const float* __restrict__ weight, float eps, int T, int H, void* dx, float* __restrict__ part,
    float* __restrict__ dweight, int accumulate) {
  using R = Row<BF16>;
  __shared__ float lds[2][2 * threads_of(W) / kWave];
  __shared__ __align__(16) float sums[partial_lds<BF16, W, NC>()];
  const Place<W, NC> at;
  const int nch = H / R::N;
  float dw[NC][R::N], wt[NC][R::N];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
      dw[u][i] = 0.f;
      wt[u][i] = c < nch ? weight[c * R::N + i] : 0.f;
    }
  }
  int turn = 0;
  for (int t0 = blockIdx.x * at.kTeams; t0 < T; t0 += gridDim.x * at.kTeams, turn ^= 1) {
    const int t = t0 + at.team;
    u32x4_t gr[NC], rr[NC], ar[NC];
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = at.first + u * kWave;
      const bool in = t < T && c < nch;
      const size_t e = (size_t)t * H + (size_t)c * R::N;
      gr[u] = in ? R::ld_s(dn, e) : u32x4_t{};
      rr[u] = in ? R::ld_s(r, e) : u32x4_t{};
      ar[u] = in && dr != nullptr ? R::ld_s(dr, e) : u32x4_t{};
    }
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      float g[R::N], v[R::N];
      R::to_f32(gr[u], g);
      R::to_f32(rr[u], v);
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        s2[0] = fmaf(v[i], v[i], s2[0]);
        s2[1] = fmaf(g[i] * wt[u][i], v[i], s2[1]);
      }
    }
    team_sum<W>(s2, lds[turn]);
    const float s = 1.f / sqrtf(s2[0] / (float)H + eps);
    const float m = s2[1] * s / (float)H;  // mean(g xh)
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = at.first + u * kWave;
      float g[R::N], v[R::N], a[R::N];
      R::to_f32(gr[u], g);
      R::to_f32(rr[u], v);
      R::to_f32(ar[u], a);
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        const float xh = v[i] * s;
        dw[u][i] = fmaf(g[i], xh, dw[u][i]);
        a[i] = fmaf(s, fmaf(-xh, m, g[i] * wt[u][i]), rs * a[i]);
      }
      if (t < T && c < nch) R::st_s(dx, (size_t)t * H + (size_t)c * R::N, R::from_f32(a));
    }
  }
  write_partial<BF16, W, NC>(at, nch, H, dw, part, dweight, accumulate, sums);
}

// out[h] (+)= sum over the G partial rows, in row order within each of 32 shares
// of the rows and then in share order.  32 columns a workgroup.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part, int G, int H,
                                                          int accumulate, float* __restrict__ out) {
  __shared__ float lds[32][33];
  const int col = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + col;
  float sum = 0.f;
  if (h < H) {
#pragma unroll 8
    for (int g = share; g < G; g += 32) sum += part[(size_t)g * H + h];
  }
  lds[share][col] = sum;
  __syncthreads();
  if (share != 0 || h >= H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += lds[i][col];
  out[h] = accumulate ? out[h] + sum : sum;
}

// What a gate is: none (1), one value a token (fp32), one an element (dtype).
enum { kGateNone = MOE_GATE_NONE, kGateToken = MOE_GATE_TOKEN, kGateFull = MOE_GATE_FULL };

// The local slots of a token, packed (rows.h); the same in every wave of a team.
struct Slots {
  int n, dc, jc;
  float wc;
  __device__ Slots(const int32_t* __restrict__ dest_row, const float* __restrict__ topk_w, int t, int T,
                   int k) {
    const int lane = lane_id();
    int d = -1;
    float w = 1.f;
    if (t < T && lane < k) {
      d = dest_row[(size_t)t * k + lane];
      if (topk_w != nullptr) w = topk_w[(size_t)t * k + lane];
    }
    n = pack_slots(d, w, dc, wc, jc);
  }
  __device__ Slots(int d, float w) { n = pack_slots(d, w, dc, wc, jc); }  // of this lane's slot
};

template <bool BF16, int W, int NC>
__global__ __launch_bounds__(threads_of(W)) void combine_norm_kernel(
    const void* __restrict__ y_perm, const float* __restrict__ topk_w,
    const int32_t* __restrict__ dest_row, const void* residual, float rs,
    const void* __restrict__ gate, int gate_kind, const float* __restrict__ weight, float eps, int T,
    int H, int k, void* y) {
  using R = Row<BF16>;
  __shared__ float lds[threads_of(W) / kWave * NC];
  const Place<W, NC> at;
  const int t = blockIdx.x * at.kTeams + at.team;
  if (W == 1 && t >= T) return;
  const Slots slot(dest_row, topk_w, t, T, k);
  const int nch = H / R::N;
  u32x4_t res[NC], gt[NC];
  float acc[NC][R::N];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
    const bool in = t < T && c < nch;
    const size_t e = (size_t)t * H + (size_t)c * R::N;
    res[u] = in && residual != nullptr ? R::ld_s(residual, e) : u32x4_t{};
    gt[u] = in && gate_kind == kGateFull ? R::ld_s(gate, e) : u32x4_t{};
#pragma unroll
    for (int i = 0; i < R::N; ++i) acc[u][i] = 0.f;
  }
  constexpr int kAtOnce = NC == 1 ? 8 : NC == 2 ? 4 : 2;  // slots whose rows are in flight
  gather_rows<BF16, true, NC, kAtOnce>(y_perm, H, nch, at.first - lane_id(), slot.n, slot.dc, slot.wc,
                                       acc);
  float ss[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    ss[u] = 0.f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) ss[u] = fmaf(acc[u][i], acc[u][i], ss[u]);
  }
  const float sum = row_sum<W>(ss, lds);
  if (t >= T) return;
  const float s = 1.f / sqrtf(sum / (float)H + eps);
  const float g1 = gate_kind == kGateToken ? ((const float*)gate)[t] : 1.f;
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    const int c = at.first + u * kWave;
    if (c >= nch) continue;
    float o[R::N], g[R::N];
    R::to_f32(res[u], o);
    R::to_f32(gt[u], g);
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
      const float ge = gate_kind == kGateFull ? g[i] : g1;
      o[i] = fmaf(ge, acc[u][i] * s * weight[c * R::N + i], rs * o[i]);
    }
    R::st_s(y, (size_t)t * H + (size_t)c * R::N, R::from_f32(o));
  }
}

// Four waves a SIMD: with registers as the compiler likes two, and 16384 tokens of
// 2048, top-8, take 271 us for 239.
// HELD slots' rows are in a lane's registers at once; where they are all of a token's,
// they stay there between c and its gradient.
template <bool BF16, int W, int NC, int HELD>
__global__ __launch_bounds__(threads_of(W), 4) void combine_norm_bwd_kernel(
    const void* __restrict__ dy, const void* __restrict__ y_perm, const float* __restrict__ topk_w,
    const int32_t* __restrict__ dest_row, const void* __restrict__ gate, int gate_kind,
    const float* __restrict__ weight, float eps, int T, int H, int k, void* __restrict__ dy_perm,
    float* __restrict__ d_topk_w, void* __restrict__ dgate, float* __restrict__ part,
    float* __restrict__ dweight, int accumulate) {
  using R = Row<BF16>;
  __shared__ float lds[2 * threads_of(W) / kWave], dots[HELD * threads_of(W) / kWave];
  __shared__ __align__(16) float sums[partial_lds<BF16, W, NC>()];
  const Place<W, NC> at;
  const int nch = H / R::N;
  float dw[NC][R::N];
#pragma unroll
  for (int u = 0; u < NC; ++u)
#pragma unroll
    for (int i = 0; i < R::N; ++i) dw[u][i] = 0.f;
  // A token's slots are fetched one token ahead where few rows are held and the wait
  // shows (16384 tokens of 1024, one slot: 38 -> 33 us; with eight held the registers
  // are missing elsewhere, 244 -> 250 for 2048 columns).
  constexpr bool kAhead = HELD <= (BF16 ? 2 : 4);
  int d0 = -1;
  float w0 = 0.f;
  const auto fetch = [&](int t) {
    const size_t i = (size_t)min(t, T - 1) * k + min(lane_id(), k - 1);
    w0 = topk_w[i];
    d0 = t < T && lane_id() < k ? dest_row[i] : -1;
  };
  if (kAhead) fetch(blockIdx.x * at.kTeams + at.team);
  for (int t0 = blockIdx.x * at.kTeams; t0 < T; t0 += gridDim.x * at.kTeams) {
    const int t = t0 + at.team;
    if (!kAhead) fetch(t);
    const Slots slot(d0, w0);
    if (t < T && threadIdx.x % (W * kWave) < k && d0 < 0) d_topk_w[(size_t)t * k + lane_id()] = 0.f;
    if (kAhead) fetch(t + gridDim.x * at.kTeams);
    // the most slots of the workgroup's tokens: the teams take part in each other's barriers
    int most = slot.n;
    if constexpr (W > 1 && Place<W, NC>::kTeams > 1) most = k;
    u32x4_t raw[HELD][NC], dyr[NC], gt[NC];
    float c_[NC][R::N];
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = at.first + u * kWave;
      const bool in = t < T && c < nch;
      const size_t e = (size_t)t * H + (size_t)c * R::N;
      dyr[u] = in ? R::ld_s(dy, e) : u32x4_t{};
      gt[u] = in && gate_kind == kGateFull ? R::ld_s(gate, e) : u32x4_t{};
#pragma unroll
      for (int i = 0; i < R::N; ++i) c_[u][i] = 0.f;
    }
    const float g1 = t < T && gate_kind == kGateToken ? ((const float*)gate)[t] : 1.f;
    const auto load = [&](int j0) {
#pragma unroll
      for (int q = 0; q < HELD; ++q) {
        const int d = __shfl(slot.dc, j0 + q, kWave);
#pragma unroll
        for (int u = 0; u < NC; ++u) {
          const int c = at.first + u * kWave;
          raw[q][u] = j0 + q < slot.n && c < nch
                          ? R::ld_s(y_perm, (size_t)d * H + (size_t)c * R::N) : u32x4_t{};
        }
      }
    };
    for (int j0 = 0; j0 < slot.n; j0 += HELD) {
      load(j0);
#pragma unroll
      for (int q = 0; q < HELD; ++q) {
        const float w = j0 + q < slot.n ? __shfl(slot.wc, j0 + q, kWave) : 0.f;
#pragma unroll
        for (int u = 0; u < NC; ++u) {
          float v[R::N];
          R::to_f32(raw[q][u], v);
#pragma unroll
          for (int i = 0; i < R::N; ++i) c_[u][i] = fmaf(w, v[i], c_[u][i]);
        }
      }
    }
    // sums of c^2 and of dy (gate) weight c: with one gate a token that is also
    // the gate's gradient
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = min(at.first + u * kWave, nch - 1);  // (past the row dy is 0)
      const float* wt = weight + c * R::N;
      float d[R::N], g[R::N];
      R::to_f32(dyr[u], d);
      R::to_f32(gt[u], g);
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        const float ge = gate_kind == kGateFull ? g[i] : 1.f;
        s2[0] = fmaf(c_[u][i], c_[u][i], s2[0]);
        s2[1] = fmaf(d[i] * ge * wt[i], c_[u][i], s2[1]);
      }
    }
    team_sum<W>(s2, lds);
    const float s = 1.f / sqrtf(s2[0] / (float)H + eps);
    const float m = g1 * s2[1] * s / (float)H;  // mean(g xh)
    if (t < T && gate_kind == kGateToken && threadIdx.x % (W * kWave) == 0)
      ((float*)dgate)[t] = s2[1] * s;
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = at.first + u * kWave;
      const float* wt = weight + min(c, nch - 1) * R::N;
      float d[R::N], g[R::N], o[R::N];
      R::to_f32(dyr[u], d);
      R::to_f32(gt[u], g);
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        const float ge = gate_kind == kGateFull ? g[i] : g1;
        const float xh = c_[u][i] * s;
        dw[u][i] = fmaf(d[i] * ge, xh, dw[u][i]);
        o[i] = d[i] * (xh * wt[i]);
        c_[u][i] = s * fmaf(-xh, m, d[i] * ge * wt[i]);  // from here on the gradient of c
      }
      if (gate_kind == kGateFull && t < T && c < nch)
        R::st_s(dgate, (size_t)t * H + (size_t)c * R::N, R::from_f32(o));
    }
    for (int j0 = 0; j0 < most; j0 += HELD) {
      if (slot.n > HELD) load(j0);  // (up to HELD rows are still in registers)
      float dot[HELD];
#pragma unroll
      for (int q = 0; q < HELD; ++q) {
        const int d = __shfl(slot.dc, j0 + q, kWave);
        const float w = __shfl(slot.wc, j0 + q, kWave);
        dot[q] = 0.f;
#pragma unroll
        for (int u = 0; u < NC; ++u) {
          const int c = at.first + u * kWave;
          float v[R::N], o[R::N];
          R::to_f32(raw[q][u], v);
#pragma unroll
          for (int i = 0; i < R::N; ++i) {
            dot[q] = fmaf(c_[u][i], v[i], dot[q]);
            o[i] = w * c_[u][i];
          }
          if (j0 + q < slot.n && c < nch) R::st_s(dy_perm, (size_t)d * H + (size_t)c * R::N, R::from_f32(o));
        }
      }
      if (W > 1 && j0 > 0) lds_barrier();  // the last group's sums have been read
      int q;
      bool has;
      const float sum = team_sum_apart<W>(dot, dots, q, has);
      const int j = __shfl(slot.jc, j0 + q, kWave);
      if (has && j0 + q < slot.n) d_topk_w[(size_t)t * k + j] = sum;
    }
    if (W > 1 && most == 0) lds_barrier();  // lds is read before the next token's sums (no slots: no other barrier)
  }
  write_partial<BF16, W, NC>(at, nch, H, dw, part, dweight, accumulate, sums);
}

// Up to this many tokens a token's slots are loaded at once by a team with one
// chunk a lane: fewer round trips, which is what few tokens wait for (columns of 2048,
// top-8, 512 tokens 8.8 -> 6.7 us, 1024: 10.9 -> 9.2, 2048: no difference; 4096 tokens
// with one local slot lose by it, 11.9 -> 13.0).  A token's bits are the same in both.
constexpr int kFewTokens = 4 * kCUs;

// Partial rows of the weight's gradient, workgroups of the backward at the most: fewer
// for wide rows, which else move more bytes of them than of the rows themselves
// (2048 rows of 8192: 56 us with 1024, 39 with 512, 38 with 256), and one a CU at the
// least (16384 of 4096: 97 us with 1024 or 512, 120 with 256).
int parts_of(int H) { return std::max(kCUs, std::min(1024, (1 << 21) / H)); }

template <int W>
int bwd_blocks(int T, int H) {
  const int teams = threads_of(W) / (W * kWave);
  return std::min((T + teams - 1) / teams, parts_of(H));
}

}  // namespace

// Teams of one wave up to 256 chunks of 16 bytes: no barrier in a row.
#define MOE_NORM_SHAPES(B, M) \
  if (nch <= 64) M(B, 1, 1) else if (nch <= 128) M(B, 1, 2) else if (nch <= 256) M(B, 1, 4) \
  else if (nch <= 512) M(B, 4, 2) else if (nch <= 1024) M(B, 4, 4) else if (nch <= 2048) M(B, 16, 2) \
  else if constexpr (!B) M(B, 16, 4)
// One chunk a lane as long as there are waves for it, so that a lane can hold the rows of
// several slots: with eight (up to 512 chunks), four (1024) or two (above) of a token's, the
// backward reads its grouped rows once, with more of them twice.
#define MOE_NORM_SHAPES1(B, M) \
  if (nch <= 64) M(B, 1, 1) else if (nch <= 128) M(B, 2, 1) else if (nch <= 256) M(B, 4, 1) \
  else if (nch <= 512) M(B, 8, 1) else if (nch <= 1024) M(B, 16, 1) else if (nch <= 2048) M(B, 16, 2) \
  else if constexpr (!B) M(B, 16, 4)

size_t norm_ws_bytes(int H) { return ((size_t)parts_of(H) * H * sizeof(float) + 255) & ~(size_t)255; }

hipError_t launch_norm(const void* x, const void* delta, const float* weight, float eps, int T, int H,
                       bool bf16, void* r, void* n, hipStream_t s) {
  ProfScope ps(MOE_KERNEL_NORM, s);
  const int nch = H / (bf16 ? 8 : 4);
#define MOE_LAUNCH(B, W, NC)                                                                         \
  {                                                                                                  \
    const int teams = threads_of(W) / (W * kWave);                                                   \
    norm_kernel<B, W, NC><<<(T + teams - 1) / teams, threads_of(W), 0, s>>>(x, delta, weight, eps, T, \
                                                                            H, r, n);                \
  }
  if (bf16) { MOE_NORM_SHAPES(true, MOE_LAUNCH) } else { MOE_NORM_SHAPES(false, MOE_LAUNCH) }
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const void* dn, const void* dr, float dr_scale, const void* r,
                           const float* weight, float eps, int T, int H, bool bf16, void* dx,
                           float* dweight, bool accumulate, void* ws, hipStream_t s) {
  ProfScope ps(MOE_KERNEL_NORM_BWD, s);
  const int nch = H / (bf16 ? 8 : 4);
  int blocks = 0;
#define MOE_LAUNCH(B, W, NC)                                                                        \
  {                                                                                                 \
    blocks = bwd_blocks<W>(T, H);                                                                      \
    if (blocks > 0)                                                                                 \
      norm_bwd_kernel<B, W, NC><<<blocks, threads_of(W), 0, s>>>(dn, dr, dr_scale, r, weight, eps,   \
                                                                 T, H, dx, (float*)ws, dweight,     \
                                                                 accumulate);                       \
  }
  if (bf16) { MOE_NORM_SHAPES(true, MOE_LAUNCH) } else { MOE_NORM_SHAPES(false, MOE_LAUNCH) }
#undef MOE_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (blocks != 1)  // (none: zeros)
    column_sum_kernel<<<(H + 31) / 32, 1024, 0, s>>>((const float*)ws, blocks, H, accumulate, dweight);
  return hipGetLastError();
}

hipError_t launch_combine_norm(const void* y_perm, const float* topk_w, const int32_t* dest_row,
                               const void* residual, float residual_scale, const void* gate, int gate_kind,
                               const float* weight, float eps, int T, int H, int k, bool bf16, void* y,
                               hipStream_t s) {
  ProfScope ps(MOE_KERNEL_COMBINE_NORM, s);
  const int nch = H / (bf16 ? 8 : 4);
#define MOE_LAUNCH(B, W, NC)                                                                          \
  {                                                                                                   \
    const int teams = threads_of(W) / (W * kWave);                                                    \
    combine_norm_kernel<B, W, NC><<<(T + teams - 1) / teams, threads_of(W), 0, s>>>(                  \
        y_perm, topk_w, dest_row, residual, residual_scale, gate, gate_kind, weight, eps, T, H, k, y); \
  }
  if (T <= kFewTokens) {
    if (bf16) { MOE_NORM_SHAPES1(true, MOE_LAUNCH) } else { MOE_NORM_SHAPES1(false, MOE_LAUNCH) }
  } else {
    if (bf16) { MOE_NORM_SHAPES(true, MOE_LAUNCH) } else { MOE_NORM_SHAPES(false, MOE_LAUNCH) }
  }
#undef MOE_LAUNCH
  return hipGetLastError();
}

hipError_t launch_combine_norm_bwd(const void* dy, const void* y_perm, const float* topk_w,
                                   const int32_t* dest_row, const void* gate, int gate_kind,
                                   const float* weight, float eps, int T, int H, int k, bool bf16,
                                   void* dy_perm, float* d_topk_w, void* dgate, float* dweight,
                                   bool accumulate, void* ws, hipStream_t s) {
  ProfScope ps(MOE_KERNEL_COMBINE_NORM_BWD, s);
  const int nch = H / (bf16 ? 8 : 4);
  int blocks = 0;
  // As many slots in registers as a token has, up to what fits beside the rest (8 held
  // for 2: 16384 tokens of 2048 132 us, 81 with 2; of 4096 x 4096, top-2, 79 and 45).
#define MOE_LAUNCH_HELD(B, W, NC, HELD)                                                              \
  combine_norm_bwd_kernel<B, W, NC, HELD><<<blocks, threads_of(W), 0, s>>>(                          \
      dy, y_perm, topk_w, dest_row, gate, gate_kind, weight, eps, T, H, k, dy_perm, d_topk_w, dgate, \
      (float*)ws, dweight, accumulate)
#define MOE_LAUNCH(B, W, NC)                                        \
  {                                                                 \
    blocks = bwd_blocks<W>(T, H);                                   \
    if (blocks > 0) {                                               \
      if constexpr (NC > 1) MOE_LAUNCH_HELD(B, W, NC, 2);           \
      else if (k <= 2) MOE_LAUNCH_HELD(B, W, NC, 2);                \
      else if constexpr (W > 8) MOE_LAUNCH_HELD(B, W, NC, 4);       \
      else if (k <= 4) MOE_LAUNCH_HELD(B, W, NC, 4);                \
      else MOE_LAUNCH_HELD(B, W, NC, 8);                            \
    }                                                               \
  }
  if (bf16) { MOE_NORM_SHAPES1(true, MOE_LAUNCH) } else { MOE_NORM_SHAPES1(false, MOE_LAUNCH) }
#undef MOE_LAUNCH
#undef MOE_LAUNCH_HELD
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (blocks != 1)  // (none: zeros)
    column_sum_kernel<<<(H + 31) / 32, 1024, 0, s>>>((const float*)ws, blocks, H, accumulate, dweight);
  return hipGetLastError();
}

}  // namespace moe
