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
// Forward, two launches (one for few tokens, balance_one).  The token axis is
// cut into chunks of C tokens, one
// workgroup each; the part of sequence s in chunk b is summed into partial row
// b + s (walking the tokens in order, b or s grows at every new pair, so the
// sum names the pair, and no plan of the ragged lengths is needed).  The
// second launch adds each sequence's partial rows in chunk order and its last
// workgroup the losses, so nothing depends on the order of execution.
#include "common.h"

namespace moe {

namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / kWave;

// LPT lanes hold V groups of four logits of a token each, and U tokens at once.
// Two groups share the token's reductions, logarithm and reciprocal among twice
// as many logits (a third fewer instructions than one group on twice the lanes).
constexpr int bal_u(int V) { return V == 1 ? 4 : 2; }
constexpr int bal_batch(int LPT, int V) { return kBalWaves * (kWave / LPT) * bal_u(V); }
int lanes_per_token(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : 32; }
int batch_of(int E) { return bal_batch(lanes_per_token(E), E <= 32 ? 1 : 2); }

// Few tokens in few sequences: one workgroup does all in one launch, 1.4 .. 1.9
// us a batch and 1.2 us a sequence's end against 8.3 .. 10 us for two launches
// (256 tokens of 8 experts in 3 sequences: 8.9 us for 9.9, and 9.5 for 12 where
// the host enqueues every call; 4 batches in 3 sequences: 12.5 for 9.7).
bool balance_one(int T, int E, int S) {
  const int b = batch_of(E);
  return ((long)T + b - 1) / b + S <= 5;
}

// Tokens per chunk: whole batches, at most 1024 chunks, so that the second
// launch has few partial rows to add.
int balance_chunk(int T, int E) {
  const int b = batch_of(E);
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
// last step by a shuffle.
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

// 1 / s for s >= 1 (NaN stays NaN): v_rcp_f32 and a step of Newton's method.
__device__ __forceinline__ float reciprocal(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return fmaf(fmaf(-s, r, 1.f), r, r);
}

// The probabilities of a token's logits p[v][i] (behind the row's end -inf), in
// their place: exp(p - top) over its sum, so that a shift of the whole row, which
// a softmax does not depend on, costs no bits.  (exp(p - lse) in the gradient, with
// lse in fp32, is off by half a step of |lse|; 32768 x 128: 8.4 us, 9.2 so.)
struct Top {
  float top, sum;
  bool none;  // a row of -inf alone: probabilities and sum 0
};
template <int LPT, int V>
__device__ __forceinline__ Top softmax(f32x4_t (&p)[V]) {
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v)
    top = fmaxf(top, fmaxf(fmaxf(p[v][0], p[v][1]), fmaxf(p[v][2], p[v][3])));
  top = group_max<LPT>(top);
  // (A NaN leaves top unless all are NaN; it comes back with the exponentials' sum.)
  const bool none = top == -INFINITY;
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = p[v][i];
      p[v][i] = exp_neg(none ? (x == x ? -INFINITY : x) : x - top);
    }
    sum += (p[v][0] + p[v][1]) + (p[v][2] + p[v][3]);
  }
  sum = group_sum<LPT>(sum);
  const float inv = none ? sum : reciprocal(sum);
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] *= inv;
  return {top, sum, none};
}

// The values of columns e .. e + 3 of a row of E (VEC: one 16-byte load); behind
// the end the last ones again, which the caller replaces (in_row).
template <bool VEC>
__device__ __forceinline__ f32x4_t load4(const float* row, int e, int E) {
  if constexpr (VEC) {
    return *reinterpret_cast<const f32x4_t*>(row + min(e, E - 4));
  } else {
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row[min(e + i, E - 1)];
    return v;
  }
}
// The same with `fill` behind the end.
template <bool VEC, typename T4, typename T>
__device__ __forceinline__ T4 load4_or(const T* row, int e, int E, T fill) {
  if constexpr (VEC) {
    return e < E ? *reinterpret_cast<const T4*>(row + e) : T4{fill, fill, fill, fill};
  } else {
    T4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e + i < E ? row[e + i] : fill;
    return v;
  }
}
template <bool VEC>
__device__ __forceinline__ bool in_row(int e, int i, int E) {
  return VEC ? e < E : e + i < E;
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

// The call's results.
struct BalOut {
  int32_t* counts;   // [S][E]
  float* prob_sum;   // [S][E]
  int32_t* tokens;   // [S + 1]
  float* loss;       // [3]
};

// loss from the sum over sequences of (1/n_s) sum_e c q, that of lse^2, and N.
__device__ __forceinline__ void write_loss(double bal, double z, int N, int E, int k, int S, float cb,
                                           float cz, const BalOut& o) {
  bal = N > 0 ? bal * E / ((double)k * N) : 0.0;
  z = N > 0 ? z / N : 0.0;
  o.tokens[S] = N;
  o.loss[0] = (float)bal;
  o.loss[1] = (float)z;
  o.loss[2] = (float)(cb * bal + cz * z);
}

// A workgroup goes through its chunk in batches, the next batch's logits on
// their way while it computes, with the running sums of the current sequence in
// registers; where a sequence ends inside the chunk, and at the chunk's end,
// the sums go out.  ONE: the only workgroup, whose sums are the results.
template <int LPT, int V, bool VEC, bool ONE>
__global__ __launch_bounds__(kBalThreads) void balance_part_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask, int T, int E, int k,
    int S, int C, float* __restrict__ lse_out, BalWs ws, float cb, float cz, BalOut out) {
  constexpr int G = kWave / LPT;          // tokens a wave holds at once
  constexpr int NG = kBalWaves * G;       // tokens a workgroup holds at once
  constexpr int U = bal_u(V);             // of them for each group
  constexpr int BT = NG * U;
  __shared__ int s_cnt[kMaxE];
  __shared__ f32x4_t s_p[NG][V * LPT];
  __shared__ float s_z[NG];
  __shared__ int s_n[NG];
  const int tid = threadIdx.x, lane = lane_id();
  const int h = lane % LPT, g = (tid >> 6) * G + lane / LPT;
  const int t0 = ONE ? 0 : blockIdx.x * C, t1 = ONE ? T : t0 + min(C, T - t0);
  if constexpr (!ONE) {
    if (blockIdx.x == 0 && tid == 0) *ws.ticket = 0;
    if (t0 >= t1) return;
  }
  constexpr int IQ = 4;  // choices of a thread loaded ahead (a batch has BT k)
  f32x4_t z[U][V];
  uint8_t mk[U];
  int pick[IQ];
  uint8_t mp[IQ];
  int tok[IQ];  // the choices' tokens in a batch
#pragma unroll
  for (int q = 0; q < IQ; ++q) tok[q] = (q * kBalThreads + tid) / k;
  auto fetch = [&](int tb) {  // (t1 > 0: clamped where a batch ends behind it)
#pragma unroll
    for (int q = 0; q < IQ; ++q) {
      pick[q] = topk_idx[min(tb * k + q * kBalThreads + tid, t1 * k - 1)];
      mp[q] = mask != nullptr ? mask[min(tb + tok[q], t1 - 1)] : (uint8_t)1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u * NG + g, t1 - 1);
      mk[u] = mask != nullptr ? mask[t] : (uint8_t)1;
#pragma unroll
      for (int v = 0; v < V; ++v) z[u][v] = load4<VEC>(logits + (size_t)t * E, 4 * (h + v * LPT), E);
    }
  };
  if (t0 < t1) fetch(t0);
  for (int e = tid; e < E; e += kBalThreads) s_cnt[e] = 0;
  int s = ONE ? 0 : seq_find(seq_offsets, S, t0, T);
  int a = s < S ? seq_off(seq_offsets, s, T) : T, b = s < S ? seq_off(seq_offsets, s + 1, T) : T;
  __syncthreads();
  f32x4_t acc[V] = {};
  float z2 = 0.f;
  int n = 0;
  double bal = 0.0, zsum = 0.0;  // ONE, thread 0: the sums over sequences
  int N = 0;
  __shared__ double s_term[kBalWaves];
  auto flush = [&]() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s_p[g][h + v * LPT] = acc[v];
      acc[v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    if (h == 0) {
      s_z[g] = z2;
      s_n[g] = n;
    }
    z2 = 0.f;
    n = 0;
    __syncthreads();
    const size_t slot = ONE ? s : (size_t)blockIdx.x + s;
    double term = 0.0;
    static_assert(kMaxE <= kBalThreads, "a thread per expert");
    if (const int e = tid; e < E) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) q += s_p[i][e / 4][e % 4];
      (ONE ? out.prob_sum : ws.psum)[slot * E + e] = q;
      (ONE ? out.counts : ws.counts)[slot * E + e] = s_cnt[e];
      if (ONE) term = (double)s_cnt[e] * (double)q;
      s_cnt[e] = 0;
    }
    if constexpr (ONE) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) term += __shfl_xor(term, o, kWave);
      if (lane == 0) s_term[tid >> 6] = term;
      __syncthreads();
    }
    if (tid == 0) {
      float zs = 0.f;
      int ns = 0;
      for (int i = 0; i < NG; ++i) {
        zs += s_z[i];
        ns += s_n[i];
      }
      if constexpr (ONE) {
        double t = 0.0;
        for (int i = 0; i < kBalWaves; ++i) t += s_term[i];
        out.tokens[s] = ns;
        bal += ns > 0 ? t / ns : 0.0;
        zsum += zs;
        N += ns;
      } else {
        ws.zsum[slot] = zs;
        ws.tokens[slot] = ns;
      }
    }
    __syncthreads();
  };
  auto empty = [&]() {  // ONE: a sequence without rows
    if (tid < E) {
      out.counts[(size_t)s * E + tid] = 0;
      out.prob_sum[(size_t)s * E + tid] = 0.f;
    }
    if (tid == 0) out.tokens[s] = 0;
  };
  for (int tb = t0; tb < t1; tb += BT) {
    f32x4_t p[U][V];
    float lse[U];
    bool live[U];
    const int te = min(t1, tb + BT);
    int now[IQ];  // -1: not an expert, or not live
#pragma unroll
    for (int q = 0; q < IQ; ++q) now[q] = mp[q] != 0 && (uint32_t)pick[q] < (uint32_t)E ? pick[q] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a row that does not count, whatever it holds, as a row of -inf
      live[u] = mk[u] != 0 && tb + u * NG + g < t1;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[u][v][i] = live[u] && in_row<VEC>(4 * (h + v * LPT), i, E) ? z[u][v][i] : -INFINITY;
    }
    if (tb + BT < t1) fetch(tb + BT);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Top t = softmax<LPT, V>(p[u]);
      lse[u] = t.none ? t.sum : t.top + __builtin_amdgcn_logf(t.sum) * 0.693147181f;
    }
    uint32_t counted = 0;  // tokens of this batch that a sequence has taken
    while (s < S && a < te) {
      const int pa = max(a, tb), pb = min(b, te);
#pragma unroll
      for (int q = 0; q < IQ; ++q) {
        const int t = tb + tok[q];
        if (t >= pa && t < pb && now[q] >= 0) atomicAdd(&s_cnt[now[q]], 1);
      }
      for (int i = max(pa * k, tb * k + IQ * kBalThreads) + tid; i < pb * k; i += kBalThreads) {
        const int e = topk_idx[i];
        if ((mask == nullptr || mask[i / k] != 0) && e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u * NG + g;
        const bool in = t >= pa && t < pb;
        if (in) counted |= 1u << u;
        if (in && live[u]) {
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += p[u][v];
          z2 = fmaf(lse[u], lse[u], z2);
          ++n;
        }
      }
      if (b > te) break;  // it goes on
      if (max(a, t0) < b) flush();
      else if (ONE) empty();
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
  if constexpr (ONE) {
    for (; s < S; ++s) empty();
    if (tid == 0) write_loss(bal, zsum, N, E, k, S, cb, cz, out);
  } else {
    if (s < S && a < t1) flush();  // the sequence that goes on in the next chunk
  }
}

// One workgroup per (sequence, COLS experts): 1024 / COLS threads of a column add
// every such partial row each, then their sums in a fixed order.  The workgroup
// that finishes last adds the losses over sequences in order.
constexpr int kSumThreads = 1024;
constexpr int kSumU = 8;  // partial rows of a thread in flight
constexpr int kSumWaves = kSumThreads / kWave;

template <typename V>
__device__ __forceinline__ void publish(V* to, V v) {
  __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V published(V* from) {
  return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int COLS>
__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int C, float cb, float cz,
    BalWs ws, BalOut out) {
  __shared__ float s_q[kSumWaves][COLS], s_z[kSumWaves];
  __shared__ int s_c[kSumWaves][COLS], s_n[kSumWaves];
  const int nb = (E + COLS - 1) / COLS;
  const int s = blockIdx.x / nb, eb = blockIdx.x % nb;
  const int tid = threadIdx.x, col = tid % COLS, part = tid / COLS;
  const int e = COLS * eb + col;
  const int a = seq_off(seq_offsets, s, T), b = seq_off(seq_offsets, s + 1, T);
  const int b0 = a / C, b1 = b > a ? (b - 1) / C + 1 : b0;
  constexpr int U = kSumU, PARTS = kSumThreads / COLS;
  float q = 0.f, zs = 0.f;
  int c = 0, n = 0;
  for (int i0 = b0 + part; i0 < b1; i0 += U * PARTS) {
    float qv[U], zv[U];
    int cv[U], nv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * PARTS;
      const size_t slot = (size_t)min(i, b1 - 1) + s;
      const int ec = min(e, E - 1);
      qv[u] = ws.psum[slot * E + ec];
      cv[u] = ws.counts[slot * E + ec];
      zv[u] = ws.zsum[slot];
      nv[u] = ws.tokens[slot];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * PARTS >= b1) continue;
      q += qv[u];
      c += cv[u];
      zs += zv[u];
      n += nv[u];
    }
  }
#pragma unroll
  for (int o = COLS; o < kWave; o <<= 1) {
    q += __shfl_xor(q, o, kWave);
    c += __shfl_xor(c, o, kWave);
    zs += __shfl_xor(zs, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (lane_id() < COLS) {
    s_q[tid / kWave][col] = q;
    s_c[tid / kWave][col] = c;
    if (col == 0) {
      s_n[tid / kWave] = n;
      s_z[tid / kWave] = zs;
    }
  }
  __syncthreads();
  int last = 0;
  if (tid < COLS) {
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
      out.counts[(size_t)s * E + e] = c;
      out.prob_sum[(size_t)s * E + e] = q;
    }
    double term = e < E && n > 0 ? (double)c * (double)q / n : 0.0;
#pragma unroll
    for (int o = COLS / 2; o > 0; o >>= 1) term += __shfl_xor(term, o, COLS);
    if (tid == 0) {
      // Everything the last workgroup reads of the others goes through
      // agent-scope atomics, performed where all XCDs see them, and this
      // workgroup's have completed before its ticket is drawn.  (Fences would
      // write a whole L2 back: 9.1 us for 6.4 with 96 workgroups.)
      publish(&ws.terms[blockIdx.x], term);
      if (eb == 0) {
        publish(&ws.zterms[s], z2);
        publish(&out.tokens[s], n);
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
    N += published(&out.tokens[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    bal += __shfl_xor(bal, o, kWave);
    z += __shfl_xor(z, o, kWave);
    N += __shfl_xor(N, o, kWave);
  }
  if (tid == 0) write_loss(bal, z, N, E, k, S, cb, cz, out);
}

// U tokens of every group at once, their logits loaded before their sequence
// (the wave's first by search, then by walking) is known.
template <int LPT, int V, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ seq_offsets, const uint8_t* __restrict__ mask,
    const float* __restrict__ d_loss, int T, int E, int k, int S, float cb, float cz, int accumulate,
    float* d_logits) {
  constexpr int G = kWave / LPT, U = bal_u(V);
  const int lane = lane_id(), h = lane % LPT;
  const int tw = (blockIdx.x * kBalWaves + (threadIdx.x >> 6)) * G * U;  // the wave's first token
  if (tw >= T) return;
  f32x4_t z[U][V];
  float l[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = min(tw + u * G + lane / LPT, T - 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
      z[u][v] = load4_or<VEC, f32x4_t>(logits + (size_t)t * E, 4 * (h + v * LPT), E, -INFINITY);
    l[u] = lse[t];
    live[u] = mask == nullptr || mask[t] != 0;
  }
  const float gl = d_loss != nullptr ? *d_loss : 1.f;
  const float N = (float)tokens[S];
  // the current sequence of the lane's group: its rows [a, b), counts, factor
  int s = seq_find(seq_offsets, S, tw, T), a = T, b = T;
  float c[V][4] = {}, kb = 0.f;
  auto enter = [&]() {
    if (s >= S) {
      a = b = T;
      return;
    }
    a = seq_off(seq_offsets, s, T);
    b = seq_off(seq_offsets, s + 1, T);
    const int32_t* cs = counts + (size_t)s * E;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const i32x4_t n = load4_or<VEC, i32x4_t>(cs, 4 * (h + v * LPT), E, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[v][i] = (float)n[i];
    }
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
    f32x4_t d[V] = {};
    if (live[u] && t >= a && t < b) {  // the same in a token's lanes
      f32x4_t p[V];
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] = z[u][v];
      softmax<LPT, V>(p);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) dot = fmaf(p[v][i], c[v][i], dot);
      dot = group_sum<LPT>(dot);
      const float kz = cz * 2.f * l[u] / N;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = gl * p[v][i] * fmaf(kb, c[v][i] - dot, kz);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 4 * (h + v * LPT);
      float* out = d_logits + (size_t)t * E;
      if (accumulate) d[v] += load4_or<VEC, f32x4_t>(out, e, E, 0.f);
      if constexpr (VEC) {
        if (e < E) *reinterpret_cast<f32x4_t*>(out + e) = d[v];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < E) out[e + i] = d[v][i];
      }
    }
  }
}

// Workgroups of the first launch (no tokens in many sequences: the first clears
// the ticket).
int balance_parts(int T, int E) {
  const int C = balance_chunk(T, E);
  return max(1, (int)(((long)T + C - 1) / C));
}

// Columns of a workgroup of the second launch: 64 where a sequence has at most a
// partial row (parts / S on average) for each of its 16 threads of a column: 236
// tokens of 255 experts in 38 sequences 5.9 us, 12 with 16; 16384 x 128 in 4
// sequences 9.4 us, 6.4 with 16.
int balance_sum_cols(int T, int E, int S) {
  return E > 16 && balance_parts(T, E) / S <= kSumThreads / 64 ? 64 : 16;
}

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

struct BalLayout {
  size_t counts, psum, tokens, zsum, ticket, terms, zterms, total;
};

BalLayout balance_layout(int T, int E, int S) {
  const size_t slots = (size_t)balance_parts(T, E) + S;
  BalLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t was = at; at += up256(bytes); return was; };
  l.counts = take(slots * E * 4);
  l.psum = take(slots * E * 4);
  l.tokens = take(slots * 4);
  l.zsum = take(slots * 4);
  l.ticket = take(4);
  l.terms = take((size_t)S * ((E + 15) / 16) * 8);
  l.zterms = take((size_t)S * 8);
  l.total = at;
  return l;
}

}  // namespace

uint64_t balance_threads(int T, int E, int S) {
  if (balance_one(T, E, S)) return kBalThreads;
  const int cols = balance_sum_cols(T, E, S);
  return (uint64_t)S * ((E + cols - 1) / cols) * kSumThreads;
}
uint64_t balance_bwd_threads(int T, int E) {
  return ((uint64_t)T + batch_of(E) - 1) / batch_of(E) * kBalThreads;
}

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
  const BalOut out = {counts, prob_sum, tokens, loss};
  const int C = balance_chunk(T, E);
  const bool one = balance_one(T, E, S);
  const int grid = one ? 1 : balance_parts(T, E);
  const bool vec = E % 4 == 0 && ((uintptr_t)logits & 15) == 0;
  ProfScope ps(MOE_KERNEL_BALANCE, s);
#define MOE_BAL(L, V, A, O)                                                                          \
  balance_part_kernel<L, V, A, O><<<grid, kBalThreads, 0, s>>>(logits, topk_idx, seq_offsets, mask, T, \
                                                               E, k, S, C, lse, ws, cb, cz, out)
#define MOE_BAL_LPT(L, V)                                                             \
  do {                                                                                \
    if (one) { if (vec) MOE_BAL(L, V, true, true); else MOE_BAL(L, V, false, true); } \
    else { if (vec) MOE_BAL(L, V, true, false); else MOE_BAL(L, V, false, false); }   \
  } while (0)
  if (E <= 32) MOE_BAL_LPT(8, 1);
  else if (E <= 64) MOE_BAL_LPT(8, 2);
  else if (E <= 128) MOE_BAL_LPT(16, 2);
  else MOE_BAL_LPT(32, 2);
#undef MOE_BAL_LPT
#undef MOE_BAL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || one) return e;
#define MOE_BAL_SUM(COLS)                                                                      \
  balance_sum_kernel<COLS><<<S * ((E + COLS - 1) / COLS), kSumThreads, 0, s>>>(seq_offsets, T, \
                                                                               E, k, S, C, cb, cz, ws, out)
  if (balance_sum_cols(T, E, S) == 64) MOE_BAL_SUM(64); else MOE_BAL_SUM(16);
#undef MOE_BAL_SUM
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(const float* logits, const float* lse, const int32_t* counts,
                                   const int32_t* tokens, const int32_t* seq_offsets,
                                   const uint8_t* mask, const float* d_loss, int T, int E, int k,
                                   int S, float cb, float cz, bool accumulate, float* d_logits,
                                   hipStream_t s) {
  const bool vec = E % 4 == 0 && (((uintptr_t)logits | (uintptr_t)counts | (uintptr_t)d_logits) & 15) == 0;
  ProfScope ps(MOE_KERNEL_BALANCE_BWD, s);
  const int batch = batch_of(E), grid = (T + batch - 1) / batch;
#define MOE_BAL(L, V, A)                                                                       \
  balance_bwd_kernel<L, V, A><<<grid, kBalThreads, 0, s>>>(logits, lse, counts, tokens,        \
                                                           seq_offsets, mask, d_loss, T, E, k, \
                                                           S, cb, cz, accumulate ? 1 : 0, d_logits)
#define MOE_BAL_LPT(L, V) do { if (vec) MOE_BAL(L, V, true); else MOE_BAL(L, V, false); } while (0)
  if (E <= 32) MOE_BAL_LPT(8, 1);
  else if (E <= 64) MOE_BAL_LPT(8, 2);
  else if (E <= 128) MOE_BAL_LPT(16, 2);
  else MOE_BAL_LPT(32, 2);
#undef MOE_BAL_LPT
#undef MOE_BAL
  return hipGetLastError();
}

}  // namespace moe
