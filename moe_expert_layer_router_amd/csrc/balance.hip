// Router auxiliary losses for gfx950: the load-balance loss with its
// per-expert counts, the z loss, and the gradient of the logits.
//
// With p[t,:] = softmax(z[t,:]), lse_t = log sum_e exp z[t,e], sequences s of
// n_s live tokens (N in all), c[s,e] the slots of s that chose e and
// q[s,e] = sum over s of p[t,e]:
//   balance = E/(k N) sum_s (1/n_s) sum_e c[s,e] q[s,e],   z = (1/N) sum_t lse_t^2
//   d total / d z[t,e] = p[t,e] (cb E/(k N n_s) (c[s,e] - sum_j p[t,j] c[s,j])
//                                + cz 2 lse_t / N)
//
// Forward, two launches.  The token axis is cut into chunks of C tokens, one
// workgroup each; the part of sequence s in chunk b is summed into partial row
// b + s (walking the tokens in order, b or s grows at every new pair, so the
// sum names the pair, and no plan of the ragged lengths is needed).  The
// second launch adds each sequence's partial rows in chunk order and its last
// workgroup the losses, so nothing depends on the order of execution.
#include "common.h"

namespace moe {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / kWave;

// Tokens per chunk: at most 512 chunks, so that the second launch has few
// partial rows to add, and at least 32 tokens, one per 16-lane group and more.
int balance_chunk(int T) {
  const int c = (T + 511) / 512;
  return c <= 32 ? 32 : (c + 31) / 32 * 32;
}

// Offset i of the sequences, inside [0, T] whatever the array holds; without
// offsets the one sequence is all T rows.
__device__ __forceinline__ int seq_off(const int32_t* off, int i, int T) {
  if (off == nullptr) return i == 0 ? 0 : T;
  return min(max(off[i], 0), T);
}

// The first sequence whose end lies behind token t, or S (then t is in none).
__device__ __forceinline__ int seq_find(const int32_t* off, int S, int t, int T) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (seq_off(off, mid + 1, T) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Reductions over the LPT lanes that hold one token.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

// The four values of columns 4 h .. 4 h + 3 of a row of E; VEC: one 16-byte load.
template <bool VEC>
__device__ __forceinline__ f32x4_t load4(const float* row, int e, int E, float fill) {
  if constexpr (VEC) {
    return e < E ? *reinterpret_cast<const f32x4_t*>(row + e) : f32x4_t{fill, fill, fill, fill};
  } else {
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e + i < E ? row[e + i] : fill;
    return v;
  }
}

// Partial rows of the first launch: [slots][E] counts, [slots][E] probability
// sums, [slots] live tokens, [slots] sums of lse^2, then the ticket.
struct BalWs {
  int32_t* counts;
  float* psum;
  int32_t* tokens;
  float* zsum;
  uint32_t* ticket;
  double* terms;   // [workgroups of the second launch] parts of the balance sum
  double* zterms;  // [S] sums of lse^2
};

template <int LPT, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_part_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask, int T, int E, int k,
    int S, int C, float* __restrict__ lse_out, BalWs ws) {
  constexpr int G = kWave / LPT;          // tokens a wave holds at once
  constexpr int NG = kBalWaves * G;       // tokens a workgroup holds at once
  constexpr int U = 4;                    // tokens of one group in flight
  __shared__ int s_cnt[kMaxE];
  __shared__ f32x4_t s_p[NG][LPT];
  __shared__ float s_z[NG];
  __shared__ int s_n[NG];
  const int tid = threadIdx.x, lane = lane_id();
  const int h = lane % LPT, g = (tid >> 6) * G + lane / LPT;
  const int t0 = blockIdx.x * C, t1 = min(T, t0 + C);
  if (blockIdx.x == 0 && tid == 0) *ws.ticket = 0;
  int at = t0;  // rows of the chunk that no sequence takes get lse 0
  for (int s = seq_find(seq_offsets, S, t0, T); s < S; ++s) {
    const int a = max(t0, seq_off(seq_offsets, s, T)), b = min(t1, seq_off(seq_offsets, s + 1, T));
    if (a >= t1) break;
    for (int t = at + tid; t < a; t += kBalThreads) lse_out[t] = 0.f;
    at = max(at, b);
    if (a >= b) continue;
    for (int e = tid; e < E; e += kBalThreads) s_cnt[e] = 0;
    __syncthreads();
    for (int i = a * k + tid; i < b * k; i += kBalThreads) {
      const int e = topk_idx[i];
      const bool live = mask == nullptr || mask[i / k] != 0;
      if (live && e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
    }
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    float z2 = 0.f;
    int n = 0;
    for (int tb = a + g; tb < b; tb += U * NG) {
      f32x4_t z[U];
      bool live[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u * NG;
        live[u] = t < b && (mask == nullptr || mask[t] != 0);
        z[u] = live[u] ? load4<VEC>(logits + (size_t)t * E, 4 * h, E, -INFINITY)
                       : f32x4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float top = group_max<LPT>(fmaxf(fmaxf(z[u][0], z[u][1]), fmaxf(z[u][2], z[u][3])));
        // a row of -inf alone: probabilities 0 and lse 0
        const bool none = top == -INFINITY;
        f32x4_t ex;
#pragma unroll
        for (int i = 0; i < 4; ++i) ex[i] = none ? 0.f : expf(z[u][i] - top);
        const float sum = group_sum<LPT>((ex[0] + ex[1]) + (ex[2] + ex[3]));
        const float inv = none ? 0.f : 1.f / sum;
        const float lse = none ? 0.f : top + logf(sum);
        const int t = tb + u * NG;
        if (live[u]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(ex[i], inv, acc[i]);
          z2 = fmaf(lse, lse, z2);
          ++n;
        }
        if (t < b && h == 0) lse_out[t] = lse;
      }
    }
    s_p[g][h] = acc;
    if (h == 0) {
      s_z[g] = z2;
      s_n[g] = n;
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = tid; e < E; e += kBalThreads) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) q += s_p[i][e / 4][e % 4];
      ws.psum[slot * E + e] = q;
      ws.counts[slot * E + e] = s_cnt[e];
    }
    if (tid == 0) {
      float zs = 0.f;
      int ns = 0;
      for (int i = 0; i < NG; ++i) {
        zs += s_z[i];
        ns += s_n[i];
      }
      ws.zsum[slot] = zs;
      ws.tokens[slot] = ns;
    }
    __syncthreads();
  }
  for (int t = at + tid; t < t1; t += kBalThreads) lse_out[t] = 0.f;
}

// One workgroup per (sequence, 32 experts): 8 threads of a column each add
// every eighth partial row, then the eight in order.  The workgroup that
// finishes last adds the losses over sequences in order.
__global__ __launch_bounds__(kBalThreads) void balance_sum_kernel(
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int C, float cb, float cz,
    BalWs ws, int32_t* __restrict__ counts, float* __restrict__ prob_sum, int32_t* tokens,
    float* __restrict__ loss) {
  __shared__ float s_q[8][32], s_z[8];
  __shared__ int s_c[8][32], s_n[8];
  __shared__ double s_bal[kBalWaves], s_zt[kBalWaves];
  __shared__ int s_tok[kBalWaves];
  __shared__ int s_last;
  const int nb = (E + 31) / 32;
  const int s = blockIdx.x / nb, eb = blockIdx.x % nb;
  const int tid = threadIdx.x, col = tid & 31, part = tid >> 5;
  const int e = 32 * eb + col;
  const int a = seq_off(seq_offsets, s, T), b = seq_off(seq_offsets, s + 1, T);
  const int b0 = a / C, b1 = b > a ? (b - 1) / C + 1 : b0;
  float q = 0.f, zs = 0.f;
  int c = 0, n = 0;
  for (int i = b0 + part; i < b1; i += 8) {
    const size_t slot = (size_t)i + s;
    if (e < E) {
      q += ws.psum[slot * E + e];
      c += ws.counts[slot * E + e];
    }
    n += ws.tokens[slot];
    zs += ws.zsum[slot];
  }
  s_q[part][col] = q;
  s_c[part][col] = c;
  if (col == 0) {
    s_n[part] = n;
    s_z[part] = zs;
  }
  __syncthreads();
  if (tid < 32) {
    q = s_q[0][col];
    c = s_c[0][col];
    n = s_n[0];
    double z2 = s_z[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      q += s_q[i][col];
      c += s_c[i][col];
      n += s_n[i];
      z2 += s_z[i];
    }
    if (e < E) {
      counts[(size_t)s * E + e] = c;
      prob_sum[(size_t)s * E + e] = q;
    }
    double term = e < E && n > 0 ? (double)c * (double)q / n : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor(term, o, 32);
    if (tid == 0) {
      ws.terms[blockIdx.x] = term;
      if (eb == 0) {
        ws.zterms[s] = z2;
        tokens[s] = n;
      }
      // this workgroup's terms before its ticket, the others' behind the last ticket
      __threadfence();
      s_last = atomicAdd(ws.ticket, 1u) == gridDim.x - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  double bal = 0.0, z = 0.0;
  int N = 0;
  for (int i = tid; i < (int)gridDim.x; i += kBalThreads)
    bal += __hip_atomic_load(&ws.terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < S; i += kBalThreads) {
    z += __hip_atomic_load(&ws.zterms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    N += __hip_atomic_load(&tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    bal += __shfl_xor(bal, o, kWave);
    z += __shfl_xor(z, o, kWave);
    N += __shfl_xor(N, o, kWave);
  }
  if (lane_id() == 0) {
    s_bal[tid >> 6] = bal;
    s_zt[tid >> 6] = z;
    s_tok[tid >> 6] = N;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kBalWaves; ++i) {
      bal += s_bal[i];
      z += s_zt[i];
      N += s_tok[i];
    }
    bal = N > 0 ? bal * E / ((double)k * N) : 0.0;
    z = N > 0 ? z / N : 0.0;
    tokens[S] = N;
    loss[0] = (float)bal;
    loss[1] = (float)z;
    loss[2] = (float)(cb * bal + cz * z);
  }
}

template <int LPT, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask,
    const float* __restrict__ d_loss, int T, int E, int k, int S, float cb, float cz, int accumulate,
    float* __restrict__ d_logits) {
  constexpr int G = kWave / LPT;
  const int lane = lane_id(), h = lane % LPT;
  const int t = (blockIdx.x * kBalWaves + (threadIdx.x >> 6)) * G + lane / LPT;
  if (t >= T) return;
  const int s = seq_find(seq_offsets, S, t, T);
  const bool live = s < S && seq_off(seq_offsets, s, T) <= t && (mask == nullptr || mask[t] != 0);
  f32x4_t d = {0.f, 0.f, 0.f, 0.f};
  if (live) {  // the same for the LPT lanes of a token
    const float g = d_loss != nullptr ? *d_loss : 1.f;
    const float n = (float)tokens[s], N = (float)tokens[S];
    const float l = lse[t];
    const f32x4_t z = load4<VEC>(logits + (size_t)t * E, 4 * h, E, -INFINITY);
    const int32_t* cs = counts + (size_t)s * E;
    float c[4], dot = 0.f, p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 4 * h + i < E ? (float)cs[4 * h + i] : 0.f;
      p[i] = expf(z[i] - l);
      dot = fmaf(p[i], c[i], dot);
    }
    dot = group_sum<LPT>(dot);
    const float kb = cb * (float)E / ((float)k * N) / n, kz = cz * 2.f * l / N;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = g * p[i] * fmaf(kb, c[i] - dot, kz);
  }
  float* out = d_logits + (size_t)t * E;
  if (accumulate) d += load4<VEC>(out, 4 * h, E, 0.f);
  if constexpr (VEC) {
    if (4 * h < E) *reinterpret_cast<f32x4_t*>(out + 4 * h) = d;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * h + i < E) out[4 * h + i] = d[i];
  }
}

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

struct BalLayout {
  size_t counts, psum, tokens, zsum, ticket, terms, zterms, total;
};

BalLayout balance_layout(int T, int E, int S) {
  const int C = balance_chunk(T);
  const size_t slots = (size_t)(T + C - 1) / C + S;
  BalLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t was = at; at += up256(bytes); return was; };
  l.counts = take(slots * E * 4);
  l.psum = take(slots * E * 4);
  l.tokens = take(slots * 4);
  l.zsum = take(slots * 4);
  l.ticket = take(4);
  l.terms = take((size_t)S * ((E + 31) / 32) * 8);
  l.zterms = take((size_t)S * 8);
  l.total = at;
  return l;
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

hipError_t launch_balance_loss(const float* logits, const int32_t* topk_idx,
                               const int32_t* seq_offsets, const uint8_t* mask, int T, int E, int k,
                               int S, float cb, float cz, int32_t* counts, float* prob_sum,
                               int32_t* tokens, float* lse, float* loss, void* ws_mem,
                               hipStream_t s) {
  const BalLayout l = balance_layout(T, E, S);
  char* w = (char*)ws_mem;
  const BalWs ws = {(int32_t*)(w + l.counts), (float*)(w + l.psum), (int32_t*)(w + l.tokens),
                    (float*)(w + l.zsum), (uint32_t*)(w + l.ticket), (double*)(w + l.terms),
                    (double*)(w + l.zterms)};
  const int C = balance_chunk(T);
  // one workgroup at least: it also clears the second launch's ticket
  const int grid = T > 0 ? (T + C - 1) / C : 1;
  const bool vec = E % 4 == 0 && ((uintptr_t)logits & 15) == 0;
  ProfScope ps(MOE_KERNEL_BALANCE, s);
#define MOE_BAL(L, V) \
  balance_part_kernel<L, V><<<grid, kBalThreads, 0, s>>>(logits, topk_idx, seq_offsets, mask, T, E, k, S, C, lse, ws)
#define MOE_BAL_LPT(L) do { if (vec) MOE_BAL(L, true); else MOE_BAL(L, false); } while (0)
  if (E <= 32) MOE_BAL_LPT(8);
  else if (E <= 64) MOE_BAL_LPT(16);
  else if (E <= 128) MOE_BAL_LPT(32);
  else MOE_BAL_LPT(64);
#undef MOE_BAL_LPT
#undef MOE_BAL
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  balance_sum_kernel<<<S * ((E + 31) / 32), kBalThreads, 0, s>>>(seq_offsets, T, E, k, S, C, cb, cz,
                                                                ws, counts, prob_sum, tokens, loss);
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(const float* logits, const float* lse, const int32_t* counts,
                                   const int32_t* tokens, const int32_t* seq_offsets,
                                   const uint8_t* mask, const float* d_loss, int T, int E, int k,
                                   int S, float cb, float cz, bool accumulate, float* d_logits,
                                   hipStream_t s) {
  const bool vec = E % 4 == 0 && (((uintptr_t)logits | (uintptr_t)d_logits) & 15) == 0;
  ProfScope ps(MOE_KERNEL_BALANCE_BWD, s);
#define MOE_BAL(L, V)                                                                          \
  balance_bwd_kernel<L, V><<<(T + kBalWaves * (kWave / L) - 1) / (kBalWaves * (kWave / L)),    \
                             kBalThreads, 0, s>>>(logits, lse, counts, tokens, seq_offsets,    \
                                                  mask, d_loss, T, E, k, S, cb, cz,            \
                                                  accumulate ? 1 : 0, d_logits)
#define MOE_BAL_LPT(L) do { if (vec) MOE_BAL(L, true); else MOE_BAL(L, false); } while (0)
  if (E <= 32) MOE_BAL_LPT(8);
  else if (E <= 64) MOE_BAL_LPT(16);
  else if (E <= 128) MOE_BAL_LPT(32);
  else MOE_BAL_LPT(64);
#undef MOE_BAL_LPT
#undef MOE_BAL
  return hipGetLastError();
}

}  // namespace moe
