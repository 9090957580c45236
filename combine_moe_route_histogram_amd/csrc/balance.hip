// The router's losses (load balance and squared log-sum-exp) and their gradient.
//
//   p = softmax(l),  c = picks, P = sum of p over a sequence of n tokens:
//   loss0 = mean_s E / (K n^2) sum_e c_e P_e,   loss1 = mean_t lse_t^2
//   dl_e = p_e (q_e - sum_j p_j q_j + r lse),   q = g0 E / (K n^2 S') c,  r = 2 g1 / N
//
// Both passes read the logits once and are bound by that read where T E is
// large, and by their two launches where it is small.
//
// A row is spread over a group of G lanes with V consecutive experts each (one
// 16-byte load where E is a multiple of 4), so the softmax takes log2(G)
// exchanges and a wave works on 64 / G rows at a time: 8 rows and 3 exchanges
// for 32 experts.  The sums over tokens stay in the lanes' registers until the
// end of a chunk; chunks' sums are joined in a fixed order (no float atomics).
#include "balance.hpp"
#include "common.hpp"

namespace moe {

namespace {

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// The experts of a lane: V consecutive ones (NI = 1), or NI single ones 64 apart (V = 1).
template <int G, int V, int NI>
struct Row {
  static constexpr int N = V * NI;
  static constexpr int kRows = kWave / G;   // rows of a wave at a time
  float v[N];
  __device__ static __forceinline__ int expert(int gl, int i) { return V > 1 ? gl * V + i : gl + i * G; }
  // l[e] of one row; -inf beyond E
  __device__ __forceinline__ void load(const float* __restrict__ row, int E, int gl, bool valid) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = -INFINITY;
    if constexpr (V == 4) {
      if (valid && gl * 4 < E) Elem<float>::unpack(ld16(row + gl * 4), v);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (valid && expert(gl, i) < E) v[i] = row[expert(gl, i)];
    }
  }
  // v <- softmax; returns the log-sum-exp.  (NaN and +inf rows end as NaN: fmaxf passes over a
  // NaN, its own exponential does not.)
  __device__ __forceinline__ float softmax() {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = group_max<G>(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = expf(v[i] - m);
      z += v[i];
    }
    z = group_sum<G>(z);
    const float inv = 1.0f / z;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= inv;
    return m + logf(z);
  }
};

// Tokens [t0, t1) of one sequence by one wave: sums of p (acc, in the lanes of the first group
// after the exchange), of lse^2 and the number of tokens (every lane); picks counted into hist
// (LDS, cleared by the caller).
template <int G, int V, int NI>
__device__ __forceinline__ void wave_sums(const BalanceArgs& a, int64_t t0, int64_t t1, int lane,
                                          float (&acc)[V * NI], float& zsum, int& n, int* hist) {
  using R = Row<G, V, NI>;
  const int gl = lane & (G - 1), sub = lane / G;
#pragma unroll
  for (int i = 0; i < R::N; ++i) acc[i] = 0.f;
  zsum = 0.f;
  n = 0;
  for (int64_t t = t0; t < t1; t += R::kRows) {
    const int64_t tok = t + sub;
    const bool in = tok < t1;
    const bool used = in && (!a.mask || a.mask[tok] != 0);
    R r;
    r.load(a.logits + tok * a.E, a.E, gl, in);
    const float lse = r.softmax();
    if (used) {
#pragma unroll
      for (int i = 0; i < R::N; ++i) acc[i] += r.v[i];
      if (gl == 0) {
        zsum += lse * lse;
        ++n;
      }
    }
  }
#pragma unroll
  for (int o = G; o < kWave; o <<= 1)
#pragma unroll
    for (int i = 0; i < R::N; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
  zsum = wave_sum(zsum);
#pragma unroll
  for (int o = kWave / 2; o >= 1; o >>= 1) n += __shfl_xor(n, o, kWave);
  // picks, K to a token
  const int64_t n_pairs = (t1 - t0) * a.K;
  for (int64_t q = lane; q < n_pairs; q += kWave) {
    const int64_t tok = t0 + q / a.K;
    const int e = a.topk_idx[t0 * a.K + q];
    if ((unsigned)e < (unsigned)a.E && (!a.mask || a.mask[tok] != 0)) atomicAdd(&hist[e], 1);
  }
}

// The sequence's balance loss from its sums, by one wave (or the first wave of a block).
__device__ __forceinline__ float sequence_loss(const BalanceArgs& a, int n, float dot) {
  return n > 0 ? (float)a.E / (float)a.K * (dot / ((float)n * (float)n)) : 0.f;
}

// Short sequences: one wave for each, all of its results.
template <int G, int V, int NI>
__global__ __launch_bounds__(256) void balance_short_kernel(BalanceArgs a) {
  using R = Row<G, V, NI>;
  __shared__ int hists[4][kMaxExperts];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int* const hist = hists[wave];   // of this wave alone: LDS keeps a wave's accesses in order
  for (int64_t s = (int64_t)blockIdx.x * 4 + wave; s < a.S; s += (int64_t)gridDim.x * 4) {
    for (int e = lane; e < a.E; e += kWave) hist[e] = 0;
    __builtin_amdgcn_wave_barrier();
    float acc[R::N], zsum;
    int n;
    const int64_t t0 = s * a.seq_len;
    wave_sums<G, V, NI>(a, t0, min<int64_t>(a.T, t0 + a.seq_len), lane, acc, zsum, n, hist);
    __builtin_amdgcn_wave_barrier();
    float dot = 0.f;
    if (lane < G) {
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        const int e = R::expert(lane, i);
        if (e < a.E) {
          const int c = hist[e];
          a.probs[s * a.E + e] = acc[i];
          a.counts[s * a.E + e] = c;
          dot += (float)c * acc[i];
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) {
      a.tokens[s] = n;
      a.seq_loss[s] = sequence_loss(a, n, dot);
      a.seq_z[s] = zsum;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Long sequences: one block for each chunk of kBalanceChunk tokens, 64 of them for each of its
// waves.  A sequence of one chunk is finished here, others leave their sums to the next launch.
template <int G, int V, int NI>
__global__ __launch_bounds__(kBalanceThreads) void balance_chunk_kernel(BalanceArgs a) {
  using R = Row<G, V, NI>;
  constexpr int NW = kBalanceThreads / kWave;
  __shared__ float part[NW][kMaxExperts];
  __shared__ int hist[kMaxExperts];
  __shared__ float zpart[NW];
  __shared__ int npart[NW];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int s = blockIdx.x / a.cps, c = blockIdx.x - s * a.cps;
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;   // of the next launch
  for (int e = tid; e < a.E; e += kBalanceThreads) hist[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)s * a.seq_len, s1 = min<int64_t>(a.T, s0 + a.seq_len);
  const int64_t t0 = min(s1, s0 + (int64_t)c * kBalanceChunk + wave * (kBalanceChunk / NW));
  const int64_t t1 = min(s1, t0 + kBalanceChunk / NW);
  float acc[R::N], zsum;
  int n;
  wave_sums<G, V, NI>(a, t0, t1, lane, acc, zsum, n, hist);
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < R::N; ++i)
      if (R::expert(lane, i) < a.E) part[wave][R::expert(lane, i)] = acc[i];
  }
  if (lane == 0) {
    zpart[wave] = zsum;
    npart[wave] = n;
  }
  __syncthreads();
  const bool whole = a.cps == 1;
  float dot = 0.f;
  for (int e = tid; e < a.E; e += kBalanceThreads) {   // E <= 256 < kBalanceThreads: one turn
    float p = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) p += part[w][e];
    const int64_t at = (int64_t)blockIdx.x * a.E + e;   // whole: [s, e]
    (whole ? a.probs : a.part_p)[at] = p;
    (whole ? a.counts : a.part_c)[at] = hist[e];
    dot += (float)hist[e] * p;
  }
  float z = 0.f;
  int total = 0;
  for (int w = 0; w < NW; ++w) {
    z += zpart[w];
    total += npart[w];
  }
  if (!whole) {
    if (tid == 0) {
      a.part_z[blockIdx.x] = z;
      a.part_n[blockIdx.x] = total;
    }
    return;
  }
  dot = wave_sum(dot);
  __syncthreads();
  if (lane == 0) zpart[wave] = dot;
  __syncthreads();
  if (tid == 0) {
    dot = 0.f;
    for (int w = 0; w < NW; ++w) dot += zpart[w];
    a.tokens[s] = total;
    a.seq_loss[s] = sequence_loss(a, total, dot);
    a.seq_z[s] = z;
  }
}

// Means over the sequences, by one block: losses, the number of tokens and of sequences with any.
// kShared: the sequences' sums were written by other blocks of this launch.
template <bool kShared>
__device__ __forceinline__ void finish(const BalanceArgs& a, float* lds_f, int* lds_i) {
  constexpr int NW = kBalanceJoin / kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  double l = 0.0, z = 0.0;
  int n = 0, some = 0;
  for (int s = tid; s < a.S; s += kBalanceJoin) {
    float ls, zs;
    int ns;
    if constexpr (kShared) {
      ls = 0.f;
      for (int b = 0; b < a.eb; ++b)
        ls += __hip_atomic_load(a.seq_loss + (int64_t)s * a.eb + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      zs = __hip_atomic_load(a.seq_z + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ns = __hip_atomic_load(a.tokens + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ls = sequence_loss(a, ns, ls);
    } else {
      ls = a.seq_loss[s];
      zs = a.seq_z[s];
      ns = a.tokens[s];
    }
    l += ls;
    z += zs;
    n += ns;
    some += ns > 0;
  }
#pragma unroll
  for (int o = kWave / 2; o >= 1; o >>= 1) {
    l += __shfl_xor(l, o, kWave);
    z += __shfl_xor(z, o, kWave);
    n += __shfl_xor(n, o, kWave);
    some += __shfl_xor(some, o, kWave);
  }
  double* const ld = reinterpret_cast<double*>(lds_f);
  if (lane == 0) {
    ld[wave] = l;
    ld[NW + wave] = z;
    lds_i[wave] = n;
    lds_i[NW + wave] = some;
  }
  __syncthreads();
  if (tid == 0) {
    l = z = 0.0;
    n = some = 0;
    for (int w = 0; w < NW; ++w) {
      l += ld[w];
      z += ld[NW + w];
      n += lds_i[w];
      some += lds_i[NW + w];
    }
    a.tokens[a.S] = n;
    a.tokens[a.S + 1] = some;
    a.loss[0] = some ? (float)(l / some) : 0.f;
    a.loss[1] = n ? (float)(z / n) : 0.f;
  }
}

__global__ __launch_bounds__(kBalanceJoin) void balance_mean_kernel(BalanceArgs a) {
  __shared__ __align__(16) float lf[4 * kBalanceJoin / kWave];
  __shared__ int li[2 * kBalanceJoin / kWave];
  finish<false>(a, lf, li);
}

// Sequences of several chunks: block (s, b) joins the chunks' sums of 32 experts of sequence s,
// 32 chunks side by side; the last block to end takes the means.  Which block that is has no
// effect on the result.
__global__ __launch_bounds__(kBalanceJoin) void balance_join_kernel(BalanceArgs a) {
  constexpr int NR = kBalanceJoin / 32;
  __shared__ __align__(16) float pp[NR][33];
  __shared__ int cc[NR][33];
  __shared__ int last;
  const int tid = threadIdx.x, col = tid & 31, row = tid >> 5;
  const int s = blockIdx.x / a.eb, b = blockIdx.x - s * a.eb;
  const int e = b * 32 + col;
  float p = 0.f;
  int c = 0;
  if (e < a.E) {
    const int64_t base = (int64_t)s * a.cps * a.E + e;
#pragma unroll 4
    for (int i = row; i < a.cps; i += NR) {
      p += a.part_p[base + (int64_t)i * a.E];
      c += a.part_c[base + (int64_t)i * a.E];
    }
  }
  pp[row][col] = p;
  cc[row][col] = c;
  float z = 0.f;
  int n = 0;
  if (b == 0 && tid < kWave) {
    for (int i = tid; i < a.cps; i += kWave) {
      z += a.part_z[(int64_t)s * a.cps + i];
      n += a.part_n[(int64_t)s * a.cps + i];
    }
    z = wave_sum(z);
#pragma unroll
    for (int o = kWave / 2; o >= 1; o >>= 1) n += __shfl_xor(n, o, kWave);
  }
  __syncthreads();
  if (tid < kWave) {
    float dot = 0.f;
    if (tid < 32) {
      p = 0.f;
      c = 0;
      for (int r = 0; r < NR; ++r) {
        p += pp[r][tid];
        c += cc[r][tid];
      }
      if (e < a.E) {
        a.probs[(int64_t)s * a.E + e] = p;
        a.counts[(int64_t)s * a.E + e] = c;
      }
      dot = (float)c * p;
    }
    dot = wave_sum(dot);
    if (tid == 0) {
      // read by the last block, on any XCD: agent-coherent stores, then the count
      __hip_atomic_store(a.seq_loss + (int64_t)s * a.eb + b, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (b == 0) {
        __hip_atomic_store(a.seq_z + s, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(a.tokens + s, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __builtin_amdgcn_s_waitcnt(0);
      const int before = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = before == (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  finish<true>(a, &pp[0][0], &cc[0][0]);
}

// ------------------------------------------------------------------ gradient

template <int G, int V, int NI, bool kRoute>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
  using R = Row<G, V, NI>;
  const int lane = threadIdx.x & (kWave - 1);
  const int gl = lane & (G - 1), sub = lane / G;
  const int64_t step = (int64_t)gridDim.x * 4 * R::kRows;
  const float total = (float)a.tokens[a.S], some = (float)a.tokens[a.S + 1];
  const float g0 = a.dloss[0] * ((float)a.E / (float)a.K) / some;
  const float g1 = 2.f * a.dloss[1] / total;
  // the loop's bound is of the wave's first row: all lanes take part in the exchanges
  for (int64_t tw = ((int64_t)blockIdx.x * 4 + threadIdx.x / kWave) * R::kRows; tw < a.T; tw += step) {
    const int64_t t = tw + sub;
    const bool in = t < a.T;
    const bool used = in && (!a.mask || a.mask[t] != 0);
    const int64_t s = in ? t / a.seq_len : 0;
    R r;
    r.load(a.logits + t * a.E, a.E, gl, in);
    const float lse = r.softmax();
    const float n = (float)a.tokens[s];
    const float f = g0 / (n * n);
    float q[R::N], dot = 0.f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) q[i] = 0.f;
    const int32_t* crow = a.counts + s * a.E;
    if constexpr (V == 4) {
      if (gl * 4 < a.E) {
        const int4 c = *reinterpret_cast<const int4*>(crow + gl * 4);
        q[0] = f * (float)c.x; q[1] = f * (float)c.y; q[2] = f * (float)c.z; q[3] = f * (float)c.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (R::expert(gl, i) < a.E) q[i] = f * (float)crow[R::expert(gl, i)];
    }
#pragma unroll
    for (int i = 0; i < R::N; ++i) dot = fmaf(r.v[i], q[i], dot);
    dot = group_sum<G>(dot);
    const float add = g1 * lse - dot;
    float out[R::N];
#pragma unroll
    for (int i = 0; i < R::N; ++i) out[i] = used ? r.v[i] * (q[i] + add) : 0.f;
    if constexpr (kRoute) {   // w_k (dw_k - sum_j w_j dw_j) for the picked experts
      float inner = 0.f;
      for (int k0 = 0; k0 < a.K; k0 += G) {
        const int k = k0 + gl;
        if (in && k < a.K) inner = fmaf(a.topk_w[t * a.K + k], a.dtopk_w[t * a.K + k], inner);
      }
      inner = group_sum<G>(inner);
      for (int k0 = 0; k0 < a.K; k0 += G) {
        const int k = k0 + gl;
        int e = -1;
        float v = 0.f;
        if (in && k < a.K) {
          e = a.topk_idx[t * a.K + k];
          v = a.topk_w[t * a.K + k] * (a.dtopk_w[t * a.K + k] - inner);
        }
        const int m = min(G, a.K - k0);
        for (int j = 0; j < m; ++j) {
          const int ej = __shfl(e, (lane & ~(G - 1)) + j, kWave);
          const float vj = __shfl(v, (lane & ~(G - 1)) + j, kWave);
#pragma unroll
          for (int i = 0; i < R::N; ++i) out[i] += R::expert(gl, i) == ej ? vj : 0.f;
        }
      }
    }
    if (in) {
      float* dst = a.dlogits + t * a.E;
      if constexpr (V == 4) {
        if (gl * 4 < a.E) st16(dst + gl * 4, Elem<float>::pack(out));
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (R::expert(gl, i) < a.E) dst[R::expert(gl, i)] = out[i];
      }
    }
  }
}

// Lanes of a row: the power of two that holds E / 4 (16-byte loads) or E experts.
template <class F>
hipError_t with_row(int E, F&& f) {
#define MOE_ROW(G, V, NI) return f(std::integral_constant<int, G>{}, std::integral_constant<int, V>{}, std::integral_constant<int, NI>{})
  if (E % 4 == 0) {
    const int q = E / 4;
    if (q <= 1) MOE_ROW(1, 4, 1);
    if (q <= 2) MOE_ROW(2, 4, 1);
    if (q <= 4) MOE_ROW(4, 4, 1);
    if (q <= 8) MOE_ROW(8, 4, 1);
    if (q <= 16) MOE_ROW(16, 4, 1);
    if (q <= 32) MOE_ROW(32, 4, 1);
    MOE_ROW(64, 4, 1);
  }
  if (E <= 4) MOE_ROW(4, 1, 1);
  if (E <= 16) MOE_ROW(16, 1, 1);
  if (E <= 64) MOE_ROW(64, 1, 1);
  if (E <= 128) MOE_ROW(64, 1, 2);
  MOE_ROW(64, 1, 4);
#undef MOE_ROW
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
  return with_row(a.E, [&](auto g, auto v, auto ni) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value, NI = decltype(ni)::value;
    if (a.seq_len <= kBalanceShort) {
      const int blocks = a.S / 4 + (a.S % 4 != 0);
      balance_short_kernel<G, V, NI><<<blocks < 65536 ? blocks : 65536, 256, 0, st>>>(a);
      balance_mean_kernel<<<1, kBalanceJoin, 0, st>>>(a);
    } else {
      balance_chunk_kernel<G, V, NI><<<a.S * a.cps, kBalanceThreads, 0, st>>>(a);
      if (a.cps == 1)
        balance_mean_kernel<<<1, kBalanceJoin, 0, st>>>(a);
      else
        balance_join_kernel<<<a.S * a.eb, kBalanceJoin, 0, st>>>(a);
    }
    return hipGetLastError();
  });
}

hipError_t launch_balance_bwd(const BalanceBwdArgs& a, hipStream_t st) {
  return with_row(a.E, [&](auto g, auto v, auto ni) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value, NI = decltype(ni)::value;
    const int64_t rows = 4 * (kWave / G);
    const int64_t blocks = (a.T + rows - 1) / rows;
    const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192);
    if (a.topk_idx)
      balance_bwd_kernel<G, V, NI, true><<<grid, 256, 0, st>>>(a);
    else
      balance_bwd_kernel<G, V, NI, false><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace moe
