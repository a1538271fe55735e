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

// Tokens a workgroup takes at once: U for every group of LPT lanes.
constexpr int kBalU = 4;
constexpr int bal_batch(int LPT) { return kBalWaves * (kWave / LPT) * kBalU; }
int lanes_per_token(int E) { return E <= 32 ? 8 : E <= 64 ? 16 : E <= 128 ? 32 : 64; }

// Tokens per chunk: whole batches, at most 1024 chunks, so that the second
// launch has few partial rows to add.
int balance_chunk(int T, int E) {
  const int b = bal_batch(lanes_per_token(E));
  return ((T + 1023) / 1024 + b - 1) / b * b + (T == 0 ? b : 0);
}

// Offset i of the sequences, inside [0, T] whatever the array holds; without
// offsets the one sequence is all T rows.
__device__ __forceinline__ int seq_off(const int32_t* off, int i, int T) {
  if (off == nullptr) return i == 0 ? 0 : T;
  return min(max(off[i], 0), T);
}

// The first sequence whose end lies behind token t (the same in the whole
// wave), or S: t is in none.  64 places are probed at once.
__device__ __forceinline__ int seq_find(const int32_t* off, int S, int t, int T) {
  if (off == nullptr) return 0;
  int lo = 0, n = S;
  for (;;) {
    const int stride = (n + kWave - 1) / kWave;
    const int i = lo + min((lane_id() + 1) * stride, n) - 1;
    const uint64_t m = __ballot(seq_off(off, i + 1, T) > t);
    if (m == 0) return S;
    const int f = __builtin_ctzll(m);
    if (stride == 1) return lo + f;
    lo += f * stride;
    n = min(stride, n - f * stride);
  }
}

// Reductions over the LPT lanes that hold one token: within 16 lanes by data
// moves of the vector unit (neighbour, pair, half-row and row mirrored), the
// last one or two steps by shuffles.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LPT, typename F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  v = f(v, moved<0xB1>(v));   // quad: lanes 1 0 3 2
  v = f(v, moved<0x4E>(v));   // quad: lanes 2 3 0 1
  v = f(v, moved<0x141>(v));  // mirror of 8
  if (LPT > 8) v = f(v, moved<0x140>(v));  // mirror of 16
  if (LPT > 16) v = f(v, __shfl_xor(v, 16, kWave));
  if (LPT > 32) v = f(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return a + b; });
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}

// exp(d) for d <= 0 (NaN stays NaN; below the normal range 0): 2^(d log2 e)
// with the product's rounding error, and that of log2 e, put back to first
// order, so that the error stays near 1 ulp for every d.
__device__ __forceinline__ float exp_neg(float d) {
  d = d < -150.f ? -150.f : d;
  const float hi = d * 1.44269502f;                       // log2 e rounded to fp32
  const float lo = fmaf(d, 1.44269502f, -hi) + d * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.693147181f, e);
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

// A workgroup goes through its chunk in batches, the next batch's logits on
// their way while it computes, with the running sums of the current sequence in
// registers; where a sequence ends inside the chunk, and at the chunk's end,
// the sums go out.
template <int LPT, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_part_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask, int T, int E, int k,
    int S, int C, float* __restrict__ lse_out, BalWs ws) {
  constexpr int G = kWave / LPT;          // tokens a wave holds at once
  constexpr int NG = kBalWaves * G;       // tokens a workgroup holds at once
  constexpr int U = kBalU;                // of them for each group
  constexpr int BT = NG * U;
  __shared__ int s_cnt[kMaxE];
  __shared__ f32x4_t s_p[NG][LPT];
  __shared__ float s_z[NG];
  __shared__ int s_n[NG];
  const int tid = threadIdx.x, lane = lane_id();
  const int h = lane % LPT, g = (tid >> 6) * G + lane / LPT;
  const int t0 = blockIdx.x * C, t1 = min(T, t0 + C);
  if (blockIdx.x == 0 && tid == 0) *ws.ticket = 0;
  if (t0 >= t1) return;
  const f32x4_t none4 = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  constexpr int IQ = 4;  // choices of a thread loaded ahead (a batch has BT k)
  f32x4_t z[U];
  uint8_t mk[U];
  int pick[IQ];
  auto choice = [&](int i, int te) {  // -1: not live
    if (i >= te * k) return -1;
    const int e = topk_idx[i];
    return mask == nullptr || mask[i / k] != 0 ? e : -1;
  };
  auto fetch = [&](int tb) {
#pragma unroll
    for (int q = 0; q < IQ; ++q) pick[q] = choice(tb * k + q * kBalThreads + tid, min(t1, tb + BT));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * NG + g;
      mk[u] = t < t1 ? (mask != nullptr ? mask[t] : (uint8_t)1) : (uint8_t)0;
      z[u] = t < t1 ? load4<VEC>(logits + (size_t)t * E, 4 * h, E, -INFINITY) : none4;
    }
  };
  fetch(t0);
  for (int e = tid; e < E; e += kBalThreads) s_cnt[e] = 0;
  int s = seq_find(seq_offsets, S, t0, T);
  int a = s < S ? seq_off(seq_offsets, s, T) : T, b = s < S ? seq_off(seq_offsets, s + 1, T) : T;
  __syncthreads();
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  float z2 = 0.f;
  int n = 0;
  auto flush = [&]() {
    s_p[g][h] = acc;
    if (h == 0) {
      s_z[g] = z2;
      s_n[g] = n;
    }
    acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    z2 = 0.f;
    n = 0;
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = tid; e < E; e += kBalThreads) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) q += s_p[i][e / 4][e % 4];
      ws.psum[slot * E + e] = q;
      ws.counts[slot * E + e] = s_cnt[e];
      s_cnt[e] = 0;
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
  };
  for (int tb = t0; tb < t1; tb += BT) {
    f32x4_t p[U];
    float lse[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a row that does not count, whatever it holds, as a row of -inf
      live[u] = mk[u] != 0;
      const f32x4_t v = live[u] ? z[u] : none4;
      const float top = group_max<LPT>(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
      // a row of -inf alone: probabilities 0 and lse 0.  (A NaN leaves top
      // unless all are NaN; it comes back with the exponentials' sum.)
      const bool none = top == -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[u][i] = none ? (v[i] == v[i] ? 0.f : v[i]) : exp_neg(v[i] - top);
      const float sum = group_sum<LPT>((p[u][0] + p[u][1]) + (p[u][2] + p[u][3]));
      const float inv = none ? (sum == sum ? 0.f : sum) : 1.f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[u][i] *= inv;
      lse[u] = none ? inv : top + logf(sum);
    }
    const int te = min(t1, tb + BT);
    int now[IQ];
#pragma unroll
    for (int q = 0; q < IQ; ++q) now[q] = pick[q];
    if (tb + BT < t1) fetch(tb + BT);
    uint32_t counted = 0;  // tokens of this batch that a sequence has taken
    while (s < S && a < te) {
      const int pa = max(a, tb), pb = min(b, te);
#pragma unroll
      for (int q = 0; q < IQ; ++q) {
        const int i = tb * k + q * kBalThreads + tid;
        if (i >= pa * k && i < pb * k && now[q] >= 0 && now[q] < E) atomicAdd(&s_cnt[now[q]], 1);
      }
      for (int i = max(pa * k, tb * k + IQ * kBalThreads) + tid; i < pb * k; i += kBalThreads) {
        const int e = choice(i, te);
        if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u * NG + g;
        const bool in = t >= pa && t < pb;
        if (in) counted |= 1u << u;
        if (in && live[u]) {
          acc += p[u];
          z2 = fmaf(lse[u], lse[u], z2);
          ++n;
        }
      }
      if (b > te) break;  // it goes on
      if (max(a, t0) < b) flush();
      ++s;
      a = b;
      b = s < S ? seq_off(seq_offsets, s + 1, T) : T;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * NG + g;
      if (t < t1 && h == 0) lse_out[t] = (counted >> u & 1) && live[u] ? lse[u] : 0.f;
    }
  }
  if (s < S && a < t1) flush();  // the sequence that goes on in the next chunk
}

// One workgroup per (sequence, 16 experts): 64 threads of a column each add
// every 64th partial row, then the 64 in a fixed order.  The workgroup that
// finishes last adds the losses over sequences in order.
constexpr int kSumThreads = 1024;
constexpr int kSumCols = 16;
constexpr int kSumParts = kSumThreads / kSumCols;
constexpr int kSumWaves = kSumThreads / kWave;

template <typename V>
__device__ __forceinline__ void publish(V* to, V v) {
  __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V published(V* from) {
  return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int C, float cb, float cz,
    BalWs ws, int32_t* __restrict__ counts, float* __restrict__ prob_sum, int32_t* tokens,
    float* __restrict__ loss) {
  __shared__ float s_q[kSumWaves][kSumCols], s_z[kSumWaves];
  __shared__ int s_c[kSumWaves][kSumCols], s_n[kSumWaves];
  const int nb = (E + kSumCols - 1) / kSumCols;
  const int s = blockIdx.x / nb, eb = blockIdx.x % nb;
  const int tid = threadIdx.x, col = tid % kSumCols, part = tid / kSumCols;
  const int e = kSumCols * eb + col;
  const int a = seq_off(seq_offsets, s, T), b = seq_off(seq_offsets, s + 1, T);
  const int b0 = a / C, b1 = b > a ? (b - 1) / C + 1 : b0;
  constexpr int U = 8;  // partial rows of a thread in flight
  float q = 0.f, zs = 0.f;
  int c = 0, n = 0;
  for (int i0 = b0 + part; i0 < b1; i0 += U * kSumParts) {
    float qv[U], zv[U];
    int cv[U], nv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSumParts;
      const size_t slot = (size_t)min(i, b1 - 1) + s;
      const int ec = min(e, E - 1);
      qv[u] = ws.psum[slot * E + ec];
      cv[u] = ws.counts[slot * E + ec];
      zv[u] = ws.zsum[slot];
      nv[u] = ws.tokens[slot];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kSumParts >= b1) continue;
      q += qv[u];
      c += cv[u];
      zs += zv[u];
      n += nv[u];
    }
  }
#pragma unroll
  for (int o = kSumCols; o < kWave; o <<= 1) {
    q += __shfl_xor(q, o, kWave);
    c += __shfl_xor(c, o, kWave);
    zs += __shfl_xor(zs, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (lane_id() < kSumCols) {
    s_q[tid / kWave][col] = q;
    s_c[tid / kWave][col] = c;
    if (col == 0) {
      s_n[tid / kWave] = n;
      s_z[tid / kWave] = zs;
    }
  }
  __syncthreads();
  int last = 0;
  if (tid < kSumCols) {
    q = 0.f;
    c = n = 0;
    double z2 = 0.0;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) {
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
    for (int o = kSumCols / 2; o > 0; o >>= 1) term += __shfl_xor(term, o, kSumCols);
    if (tid == 0) {
      // Everything the last workgroup reads of the others goes through
      // agent-scope atomics, performed where all XCDs see them, and this
      // workgroup's have completed before its ticket is drawn.  (Fences would
      // write a whole L2 back: 9.1 us for 6.4 with 96 workgroups.)
      publish(&ws.terms[blockIdx.x], term);
      if (eb == 0) {
        publish(&ws.zterms[s], z2);
        publish(&tokens[s], n);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      last = __hip_atomic_fetch_add(ws.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.x - 1;
      asm volatile("" ::: "memory");
    }
  }
  if (tid >= kWave) return;  // one wave holds tid 0 and adds the losses
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  double bal = 0.0, z = 0.0;
  int N = 0;
  for (int i = tid; i < (int)gridDim.x; i += kWave)
    bal += published(&ws.terms[i]);
  for (int i = tid; i < S; i += kWave) {
    z += published(&ws.zterms[i]);
    N += published(&tokens[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    bal += __shfl_xor(bal, o, kWave);
    z += __shfl_xor(z, o, kWave);
    N += __shfl_xor(N, o, kWave);
  }
  if (tid == 0) {
    bal = N > 0 ? bal * E / ((double)k * N) : 0.0;
    z = N > 0 ? z / N : 0.0;
    tokens[S] = N;
    loss[0] = (float)bal;
    loss[1] = (float)z;
    loss[2] = (float)(cb * bal + cz * z);
  }
}

// U tokens of every group at once, their logits loaded before their sequence
// (the wave's first by search, then by walking) is known.
template <int LPT, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask,
    const float* __restrict__ d_loss, int T, int E, int k, int S, float cb, float cz, int accumulate,
    float* d_logits) {
  constexpr int G = kWave / LPT, U = kBalU;
  const int lane = lane_id(), h = lane % LPT;
  const int tw = (blockIdx.x * kBalWaves + (threadIdx.x >> 6)) * G * U;  // the wave's first token
  if (tw >= T) return;
  f32x4_t z[U];
  float l[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = min(tw + u * G + lane / LPT, T - 1);
    z[u] = load4<VEC>(logits + (size_t)t * E, 4 * h, E, -INFINITY);
    l[u] = lse[t];
    live[u] = mask == nullptr || mask[t] != 0;
  }
  const float gl = d_loss != nullptr ? *d_loss : 1.f;
  const float N = (float)tokens[S];
  // the current sequence of the lane's group: its rows [a, b), counts, factor
  int s = seq_find(seq_offsets, S, tw, T), a = T, b = T;
  float c[4] = {0.f, 0.f, 0.f, 0.f}, kb = 0.f;
  auto enter = [&]() {
    if (s >= S) {
      a = b = T;
      return;
    }
    a = seq_off(seq_offsets, s, T);
    b = seq_off(seq_offsets, s + 1, T);
    const int32_t* cs = counts + (size_t)s * E;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = (float)cs[min(4 * h + i, E - 1)];
    kb = cb * (float)E / ((float)k * N) / (float)tokens[s];
  };
  enter();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = tw + u * G + lane / LPT;
    if (t >= T) continue;
    while (t >= b && s < S) {
      ++s;
      enter();
    }
    f32x4_t d = {0.f, 0.f, 0.f, 0.f};
    if (live[u] && t >= a && t < b) {  // the same in a token's lanes
      float p[4], dot = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = exp_neg(z[u][i] - l[u]);
        dot = fmaf(p[i], c[i], dot);
      }
      dot = group_sum<LPT>(dot);
      const float kz = cz * 2.f * l[u] / N;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = gl * p[i] * fmaf(kb, c[i] - dot, kz);
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
}

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

struct BalLayout {
  size_t counts, psum, tokens, zsum, ticket, terms, zterms, total;
};

BalLayout balance_layout(int T, int E, int S) {
  const int C = balance_chunk(T, E);
  const size_t slots = (size_t)(T + C - 1) / C + S;
  BalLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t was = at; at += up256(bytes); return was; };
  l.counts = take(slots * E * 4);
  l.psum = take(slots * E * 4);
  l.tokens = take(slots * 4);
  l.zsum = take(slots * 4);
  l.ticket = take(4);
  l.terms = take((size_t)S * ((E + kSumCols - 1) / kSumCols) * 8);
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
  const int C = balance_chunk(T, E);
  // one workgroup at least: it also clears the second launch's ticket
  const int grid = T > 0 ? (T + C - 1) / C : 1;
  const bool vec = E % 4 == 0 && ((uintptr_t)logits & 15) == 0;
  ProfScope ps(MOE_KERNEL_BALANCE, s);
#define MOE_BAL(L, V) \
  balance_part_kernel<L, V><<<grid, kBalThreads, 0, s>>>(logits, topk_idx, seq_offsets, mask, T, E, k, S, C, lse, ws)
#define MOE_BAL_LPT(L) do { if (vec) MOE_BAL(L, true); else MOE_BAL(L, false); } while (0)
  switch (lanes_per_token(E)) {
    case 8: MOE_BAL_LPT(8); break;
    case 16: MOE_BAL_LPT(16); break;
    case 32: MOE_BAL_LPT(32); break;
    default: MOE_BAL_LPT(64);
  }
#undef MOE_BAL_LPT
#undef MOE_BAL
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  balance_sum_kernel<<<S * ((E + kSumCols - 1) / kSumCols), kSumThreads, 0, s>>>(seq_offsets, T, E, k, S, C, cb, cz,
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
  balance_bwd_kernel<L, V><<<(T + bal_batch(L) - 1) / bal_batch(L), kBalThreads, 0, s>>>(logits, lse, counts, tokens, seq_offsets,    \
                                                  mask, d_loss, T, E, k, S, cb, cz,            \
                                                  accumulate ? 1 : 0, d_logits)
#define MOE_BAL_LPT(L) do { if (vec) MOE_BAL(L, true); else MOE_BAL(L, false); } while (0)
  switch (lanes_per_token(E)) {
    case 8: MOE_BAL_LPT(8); break;
    case 16: MOE_BAL_LPT(16); break;
    case 32: MOE_BAL_LPT(32); break;
    default: MOE_BAL_LPT(64);
  }
#undef MOE_BAL_LPT
#undef MOE_BAL
  return hipGetLastError();
}

}  // namespace moe
