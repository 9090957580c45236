// The router's losses (load balance and squared log-sum-exp) and their gradient.
//
//   p = softmax(l),  c = picks, P = sum of p over a sequence of n tokens:
//   loss0 = mean_s E / (K n^2) sum_e c_e P_e,   loss1 = mean_t lse_t^2
//   dl_e = p_e (q_e - sum_j p_j q_j + r lse),   q = g0 E / (K n^2 S') c,  r = 2 g1 / N
//
// Both passes read the logits once and are bound by that read where T E is
// large, and by their two launches where it is small.
//
// A row is spread over a group of G lanes with 4 consecutive experts each (one
// 16-byte load, of whatever alignment), so the softmax takes log2(G)
// exchanges and a wave works on 64 / G rows at a time: 8 rows and 3 exchanges
// for 32 experts.  The sums over tokens stay in the lanes' registers until the
// end of a chunk; chunks' sums are joined in a fixed order (no float atomics).
#include "balance.hpp"
#include "common.hpp"

namespace moe {

namespace {

// Exchanges inside groups of G lanes without LDS: within 16 lanes by DPP (neighbours, pairs, then the
// mirror images of 8 and of 16 lanes, whose quads and halves hold one value by then), beyond by swapping
// rows of 16 and of 32 lanes.  Every lane is active.  (ds_bpermute, which a shuffle compiles to, takes
// about ten times as long: losses of 131072 tokens 15.6 us with it, see below.)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int G, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  if constexpr (G >= 2) v = op(v, dpp<0xB1>(v));     // quad_perm 1 0 3 2
  if constexpr (G >= 4) v = op(v, dpp<0x4E>(v));     // quad_perm 2 3 0 1
  if constexpr (G >= 8) v = op(v, dpp<0x141>(v));    // row_half_mirror
  if constexpr (G >= 16) v = op(v, dpp<0x140>(v));   // row_mirror
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float x, float y) { return fmaxf(x, y); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<G>(v, [](float x, float y) { return x + y; });
}

// 16 bytes at an address that is a multiple of 4 (rows of E floats need not be 16-byte aligned).
struct __attribute__((packed, aligned(4))) Loose4 { uint32_t v[4]; };
__device__ __forceinline__ u32x4 ld16_loose(const void* p) {
  const Loose4 l = *static_cast<const Loose4*>(p);
  return u32x4{l.v[0], l.v[1], l.v[2], l.v[3]};
}
__device__ __forceinline__ void st16_loose(void* p, const u32x4& v) {
  *static_cast<Loose4*>(p) = Loose4{{v[0], v[1], v[2], v[3]}};
}
// Words [at, at + 4) of a row of n, `none` for those past its end.
__device__ __forceinline__ u32x4 load_row4(const void* row, int at, int n, bool valid, uint32_t none) {
  const uint32_t* const p = static_cast<const uint32_t*>(row) + at;
  u32x4 v = {none, none, none, none};
  if (valid && at + 4 <= n) {
    v = ld16_loose(p);
  } else if (valid && at < n) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (at + i < n) v[i] = p[i];
  }
  return v;
}

// A lane's four experts of a row: G lanes hold it.
template <int G>
struct Row {
  static constexpr int N = 4;
  static constexpr int kRows = kWave / G;   // rows of a wave at a time
  float v[N];
  __device__ static __forceinline__ int expert(int gl, int i) { return gl * 4 + i; }
  // l[e] of one row; -inf beyond E
  __device__ __forceinline__ void load(const float* row, int E, int gl, bool valid) {
    Elem<float>::unpack(load_row4(row, gl * 4, E, valid, 0xFF800000u), v);
  }
  // v <- softmax; returns the log-sum-exp.  The hardware's exponential, logarithm and reciprocal (1 ulp
  // each; the argument (l - max) log2 e carries one rounding of each factor, and z is in [1, E]): the
  // libraries' forms would make these kernels wait for the vector units instead of memory (256 experts:
  // 61 us for 131072 tokens).  NaN and +inf rows end as NaN: fmaxf passes over a NaN, its own
  // exponential does not.
  __device__ __forceinline__ float softmax() {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = group_max<G>(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = __builtin_amdgcn_exp2f((v[i] - m) * 1.44269504f);
      z += v[i];
    }
    z = group_sum<G>(z);
    const float inv = __builtin_amdgcn_rcpf(z);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= inv;
    return fmaf(__builtin_amdgcn_logf(z), 0.693147181f, m);
  }
};

// Tokens [t0, t1) of one sequence by one wave: sums of p (acc, in the lanes of the first
// group after the exchange), of lse^2 and the number of tokens (every lane); picks counted into hist
// (LDS, cleared by the caller).  A wave has few rows and each pass over them would wait for memory, so
// several are loaded ahead.
template <int G>
__device__ __forceinline__ void wave_sums(const BalanceArgs& a, int64_t t0, int64_t t1, int lane,
                                          float (&acc)[4], float& zsum, int& n, int* hist) {
  using R = Row<G>;
  constexpr int U = G < 8 ? G : 8;                 // of the G passes over 64 rows
  const int gl = lane & (G - 1), sub = lane / G;
  const int rows = (int)(t1 - t0);
  const float* const l0 = a.logits + t0 * a.E;
  const uint8_t* const m0 = a.mask ? a.mask + t0 : nullptr;
  // picks: K to a token, the first ones loaded ahead of the rows
  constexpr int kAhead = 4;
  const int n_pairs = rows * a.K;
  const int32_t* const i0 = a.topk_idx + t0 * a.K;
  int pick[kAhead];
  bool pick_on[kAhead];
  auto load_pick = [&](int q, int& e, bool& on) {
    on = q < n_pairs;
    e = on ? i0[q] : -1;
    if (m0 && on) on = m0[(unsigned)q / (unsigned)a.K] != 0;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load_pick(lane + kWave * i, pick[i], pick_on[i]);
#pragma unroll
  for (int i = 0; i < R::N; ++i) acc[i] = 0.f;
  zsum = 0.f;
  n = 0;
  for (int t = 0; t < rows; t += R::kRows * U) {
    R r[U];
    bool used[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = t + u * R::kRows + sub;
      const bool in = row < rows;
      r[u].load(l0 + (int64_t)row * a.E, a.E, gl, in);
      used[u] = in && (!m0 || m0[row] != 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float lse = r[u].softmax();
      if (used[u]) {
#pragma unroll
        for (int i = 0; i < R::N; ++i) acc[i] += r[u].v[i];
        if (gl == 0) {
          zsum += lse * lse;
          ++n;
        }
      }
    }
  }
  auto count = [&](int e, bool on) {
    if (on && (unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) count(pick[i], pick_on[i]);
  for (int q = lane + kWave * kAhead; q < n_pairs; q += kWave) {
    int e;
    bool on;
    load_pick(q, e, on);
    count(e, on);
  }
#pragma unroll
  for (int o = G; o < kWave; o <<= 1)
#pragma unroll
    for (int i = 0; i < R::N; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
  zsum = wave_sum(zsum);
#pragma unroll
  for (int o = kWave / 2; o >= 1; o >>= 1) n += __shfl_xor(n, o, kWave);
}

// The sequence's balance loss from its sums, by one wave (or the first wave of a block).
__device__ __forceinline__ float sequence_loss(const BalanceArgs& a, int n, float dot) {
  return n > 0 ? (float)a.E / (float)a.K * (dot / ((float)n * (float)n)) : 0.f;
}

// A block's sums over its sequences, from those of its four waves.
__device__ __forceinline__ void block_sums(const BalanceArgs& a, float loss, float z, int n, int some, int lane,
                                           int wave) {
  __shared__ float sums[4][2];
  __shared__ int numbers[4][2];
  if (lane == 0) {
    sums[wave][0] = loss;
    sums[wave][1] = z;
    numbers[wave][0] = n;
    numbers[wave][1] = some;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.seq_loss[blockIdx.x] = (sums[0][0] + sums[1][0]) + (sums[2][0] + sums[3][0]);
    a.seq_z[blockIdx.x] = (sums[0][1] + sums[1][1]) + (sums[2][1] + sums[3][1]);
    a.seq_n[blockIdx.x] = (numbers[0][0] + numbers[1][0]) + (numbers[2][0] + numbers[3][0]);
    a.seq_some[blockIdx.x] = (numbers[0][1] + numbers[1][1]) + (numbers[2][1] + numbers[3][1]);
  }
}

// Sequences of a few tokens: one lane group for each (131072 sequences of one token, 32 experts: 174 us
// with a wave for each).
template <int G>
__global__ __launch_bounds__(256) void balance_few_kernel(BalanceArgs a) {
  using R = Row<G>;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int gl = lane & (G - 1), sub = lane / G;
  float loss_sum = 0.f, z_sum = 0.f;
  int n_sum = 0, some = 0;
  // the bounds are of the wave's first sequence and the longest: all lanes take part in the exchanges
  for (int64_t s0 = ((int64_t)blockIdx.x * 4 + wave) * R::kRows; s0 < a.S; s0 += (int64_t)gridDim.x * 4 * R::kRows) {
    const int64_t s = s0 + sub;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int count[4] = {0, 0, 0, 0}, n = 0;
    for (int j = 0; j < a.seq_len; ++j) {
      const int64_t t = s * a.seq_len + j;
      const bool in = s < a.S && t < a.T;
      const bool used = in && (!a.mask || a.mask[t] != 0);
      R r;
      r.load(a.logits + t * a.E, a.E, gl, in);
      const float lse = r.softmax();
      if (used) {
        ++n;
        if (gl == 0) z_sum += lse * lse;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += r.v[i];
        for (int k = 0; k < a.K; k += 4) {
          const u32x4 e = load_row4(a.topk_idx + t * a.K, k, a.K, true, 0xFFFFFFFFu);
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) count[i] += (int)e[h] == R::expert(gl, i);
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = R::expert(gl, i);
      if (s < a.S && e < a.E) {
        a.probs[s * a.E + e] = acc[i];
        a.counts[s * a.E + e] = count[i];
        dot = fmaf((float)count[i], acc[i], dot);
      }
    }
    dot = group_sum<G>(dot);
    if (gl == 0 && s < a.S) {
      a.tokens[s] = n;
      loss_sum += sequence_loss(a, n, dot);
      n_sum += n;
      some += n > 0;
    }
  }
  loss_sum = wave_sum(loss_sum);
  z_sum = wave_sum(z_sum);
#pragma unroll
  for (int o = kWave / 2; o >= 1; o >>= 1) {
    n_sum += __shfl_xor(n_sum, o, kWave);
    some += __shfl_xor(some, o, kWave);
  }
  block_sums(a, loss_sum, z_sum, n_sum, some, lane, wave);
}

// Short sequences: one wave for each, all of its results; the block's sums over its sequences go to the
// next launch (one sequence a block left that with 131072 sequences of one token: 25 us).
template <int G>
__global__ __launch_bounds__(256) void balance_short_kernel(BalanceArgs a) {
  using R = Row<G>;
  __shared__ int hists[4][kMaxExperts];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int* const hist = hists[wave];   // of this wave alone: LDS keeps a wave's accesses in order
  float loss_sum = 0.f, z_sum = 0.f;
  int n_sum = 0, some = 0;
  for (int64_t s = (int64_t)blockIdx.x * 4 + wave; s < a.S; s += (int64_t)gridDim.x * 4) {
    for (int e = lane; e < a.E; e += kWave) hist[e] = 0;
    __builtin_amdgcn_wave_barrier();
    float acc[R::N], zsum;
    int n;
    const int64_t t0 = s * a.seq_len;
    wave_sums<G>(a, t0, min<int64_t>(a.T, t0 + a.seq_len), lane, acc, zsum, n, hist);
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
    if (lane == 0) a.tokens[s] = n;
    loss_sum += sequence_loss(a, n, dot);
    z_sum += zsum;
    n_sum += n;
    some += n > 0;
    __builtin_amdgcn_wave_barrier();
  }
  block_sums(a, loss_sum, z_sum, n_sum, some, lane, wave);
}

// Long sequences: one block for each chunk of tokens, a share of at most 64 of them for each of its
// waves.  A sequence of one chunk is finished here, others leave their sums to the next launch.
template <int G>
__global__ __launch_bounds__(kBalanceThreads) void balance_chunk_kernel(BalanceArgs a) {
  using R = Row<G>;
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
  const int64_t t0 = min(s1, s0 + (int64_t)c * a.chunk + wave * (a.chunk / NW));
  const int64_t t1 = min(s1, t0 + a.chunk / NW);
  float acc[R::N], zsum;
  int n;
  wave_sums<G>(a, t0, t1, lane, acc, zsum, n, hist);
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

// Means over the sequences, by one block: losses, the number of tokens and of sequences with any.  Its
// entries are the sequences, or the short sequences' blocks.  kShared: the sequences' sums were written by
// other blocks of this launch.
template <bool kShared>
__device__ __forceinline__ void finish(const BalanceArgs& a, float* lds_f, int* lds_i) {
  constexpr int NW = kBalanceJoin / kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  double l = 0.0, z = 0.0;
  int n = 0, some = 0;
#pragma unroll 2
  for (int s = tid; s < a.entries; s += kBalanceJoin) {
    float ls, zs;
    int ns, any;
    if constexpr (kShared) {
      ls = 0.f;
      for (int b = 0; b < a.eb; ++b)
        ls += __hip_atomic_load(a.seq_loss + (int64_t)s * a.eb + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      zs = __hip_atomic_load(a.seq_z + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ns = __hip_atomic_load(a.tokens + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ls = sequence_loss(a, ns, ls);
      any = ns > 0;
    } else {
      ls = a.seq_loss[s];
      zs = a.seq_z[s];
      ns = a.seq_n[s];
      any = a.seq_some ? a.seq_some[s] : ns > 0;
    }
    l += ls;
    z += zs;
    n += ns;
    some += any;
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
// 32 chunks side by side.  A single block ends with the losses; of several the last one to end takes
// the means, and which one that is has no effect on the result.
__global__ __launch_bounds__(kBalanceJoin) void balance_join_kernel(BalanceArgs a) {
  constexpr int NW = kBalanceJoin / kWave, NR = kBalanceJoin / 32;
  __shared__ __align__(16) float pp[NW][32];
  __shared__ int cc[NW][32];
  __shared__ float zz;
  __shared__ int nn, last;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, col = tid & 31, row = tid >> 5;
  const int s = blockIdx.x / a.eb, b = blockIdx.x - s * a.eb;
  const int e = b * 32 + col;
  float p = 0.f;
  int c = 0;
  if (e < a.E) {
    const int64_t base = (int64_t)s * a.cps * a.E + e;
#pragma unroll 8
    for (int i = row; i < a.cps; i += NR) {
      p += a.part_p[base + (int64_t)i * a.E];
      c += a.part_c[base + (int64_t)i * a.E];
    }
  }
  if (b == 0 && wave == NW - 1) {
    float z = 0.f;
    int n = 0;
#pragma unroll 4
    for (int i = lane; i < a.cps; i += kWave) {
      z += a.part_z[(int64_t)s * a.cps + i];
      n += a.part_n[(int64_t)s * a.cps + i];
    }
    z = wave_sum(z);
#pragma unroll
    for (int o = kWave / 2; o >= 1; o >>= 1) n += __shfl_xor(n, o, kWave);
    if (lane == 0) {
      zz = z;
      nn = n;
    }
  }
  p += __shfl_xor(p, 32, kWave);
  c += __shfl_xor(c, 32, kWave);
  if (lane < 32) {
    pp[wave][lane] = p;
    cc[wave][lane] = c;
  }
  __syncthreads();
  if (wave == 0) {
    p = 0.f;
    c = 0;
#pragma unroll
    for (int w = 0; w < NW / 2; ++w) {
      p += pp[w + (lane >> 5) * (NW / 2)][col];
      c += cc[w + (lane >> 5) * (NW / 2)][col];
    }
    p += __shfl_xor(p, 32, kWave);
    c += __shfl_xor(c, 32, kWave);
    if (lane < 32 && e < a.E) {
      a.probs[(int64_t)s * a.E + e] = p;
      a.counts[(int64_t)s * a.E + e] = c;
    }
    const float dot = wave_sum(lane < 32 ? (float)c * p : 0.f);
    if (lane == 0) {
      if (gridDim.x == 1) {
        a.tokens[0] = a.tokens[1] = nn;
        a.tokens[2] = nn > 0;
        a.loss[0] = sequence_loss(a, nn, dot);
        a.loss[1] = nn ? zz / (float)nn : 0.f;
        last = 0;
      } else {
        // read by the last block, on any XCD: agent-coherent stores, then the count
        __hip_atomic_store(a.seq_loss + (int64_t)s * a.eb + b, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (b == 0) {
          __hip_atomic_store(a.seq_z + s, zz, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(a.tokens + s, nn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __builtin_amdgcn_s_waitcnt(0);
        const int before = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = before == (int)gridDim.x - 1;
      }
    }
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  finish<true>(a, &pp[0][0], &cc[0][0]);
}

// ------------------------------------------------------------------ gradient

template <int G, bool kRoute>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
  using R = Row<G>;
  constexpr int U = kBwdRows;                      // rows of a lane group in flight
  constexpr int kPicks = 8;                        // of a row, loaded ahead (the same address in its lanes)
  const int lane = threadIdx.x & (kWave - 1);
  const int gl = lane & (G - 1), sub = lane / G;
  const int64_t step = (int64_t)gridDim.x * 4 * R::kRows * U;
  // the loop's bound is of the wave's first row: all lanes take part in the exchanges
  for (int64_t tw = ((int64_t)blockIdx.x * 4 + threadIdx.x / kWave) * R::kRows * U; tw < a.T; tw += step) {
    R r[U], q[U];
    bool in[U], used[U];
    float n[U], pw[U][kPicks], pd[U][kPicks];
    int pe[U][kPicks];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = tw + u * R::kRows + sub;
      in[u] = t < a.T;
      r[u].load(a.logits + t * a.E, a.E, gl, in[u]);
      used[u] = in[u] && (!a.mask || a.mask[t] != 0);
      if constexpr (kRoute) {                       // the first picks; more below
#pragma unroll
        for (int h = 0; h < kPicks; h += 4) {       // the same address in a row's lanes; uniform in K
          const int64_t at = t * a.K;
          const bool on = in[u] && h < a.K;
          Elem<float>::unpack(load_row4(a.topk_w + at, h, a.K, on, 0u), pw[u] + h);
          Elem<float>::unpack(load_row4(a.dtopk_w + at, h, a.K, on, 0u), pd[u] + h);
          const u32x4 e = load_row4(a.topk_idx + at, h, a.K, on, 0xFFFFFFFFu);
#pragma unroll
          for (int i = 0; i < 4; ++i) pe[u][h + i] = (int)e[i];
        }
      }
      const int64_t s = in[u] ? a.seq.of((uint32_t)t) : 0;
      n[u] = (float)a.tokens[s];
      const u32x4 c = load_row4(a.counts + s * a.E, gl * 4, a.E, true, 0u);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[u].v[i] = (float)(int)c[i];
    }
    const float g0 = a.dloss[0] * ((float)a.E / (float)a.K) / (float)a.tokens[a.S + 1];
    const float g1 = 2.f * a.dloss[1] / (float)a.tokens[a.S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = tw + u * R::kRows + sub;
      const float lse = r[u].softmax();
      const float f = g0 / (n[u] * n[u]);
      float dot = 0.f, out[R::N];
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        q[u].v[i] *= f;
        dot = fmaf(r[u].v[i], q[u].v[i], dot);
      }
      dot = group_sum<G>(dot);
      const float add = g1 * lse - dot;
#pragma unroll
      for (int i = 0; i < R::N; ++i) out[i] = used[u] ? r[u].v[i] * (q[u].v[i] + add) : 0.f;
      if constexpr (kRoute) {   // w_k (dw_k - sum_j w_j dw_j) for the picked experts
        float inner = 0.f;
#pragma unroll
        for (int k = 0; k < kPicks; ++k) inner = fmaf(pw[u][k], pd[u][k], inner);
        const int64_t at = t * a.K;
        if (in[u])
          for (int k = kPicks; k < a.K; ++k) inner = fmaf(a.topk_w[at + k], a.dtopk_w[at + k], inner);
        auto add_pick = [&](int e, float v) {
#pragma unroll
          for (int i = 0; i < R::N; ++i) out[i] += R::expert(gl, i) == e ? v : 0.f;
        };
#pragma unroll
        for (int k = 0; k < kPicks; ++k) add_pick(pe[u][k], pw[u][k] * (pd[u][k] - inner));
        if (in[u])
          for (int k = kPicks; k < a.K; ++k) add_pick(a.topk_idx[at + k], a.topk_w[at + k] * (a.dtopk_w[at + k] - inner));
      }
      if (in[u]) {
        float* dst = a.dlogits + t * a.E + gl * 4;
        if (gl * 4 + 4 <= a.E) {
          st16_loose(dst, Elem<float>::pack(out));
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (gl * 4 + i < a.E) dst[i] = out[i];
        }
      }
    }
  }
}

template <class F>
hipError_t with_row(int E, F&& f) {
  switch (balance_lanes(E)) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    default: return f(std::integral_constant<int, 64>{});
  }
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
  return with_row(a.E, [&](auto g) {
    constexpr int G = decltype(g)::value;
    if (a.by == kByGroup) {
      balance_few_kernel<G><<<a.entries, 256, 0, st>>>(a);
      balance_mean_kernel<<<1, kBalanceJoin, 0, st>>>(a);
    } else if (a.by == kByWave) {
      balance_short_kernel<G><<<a.entries, 256, 0, st>>>(a);
      balance_mean_kernel<<<1, kBalanceJoin, 0, st>>>(a);
    } else {
      balance_chunk_kernel<G><<<a.S * a.cps, kBalanceThreads, 0, st>>>(a);
      if (a.cps == 1)
        balance_mean_kernel<<<1, kBalanceJoin, 0, st>>>(a);
      else
        balance_join_kernel<<<a.S * a.eb, kBalanceJoin, 0, st>>>(a);
    }
    return hipGetLastError();
  });
}

hipError_t launch_balance_bwd(const BalanceBwdArgs& a, hipStream_t st) {
  return with_row(a.E, [&](auto g) {
    constexpr int G = decltype(g)::value;
    const int64_t rows = 4 * (kWave / G) * kBwdRows;
    const int64_t blocks = (a.T + rows - 1) / rows;
    const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192);
    if (a.topk_idx)
      balance_bwd_kernel<G, true><<<grid, 256, 0, st>>>(a);
    else
      balance_bwd_kernel<G, false><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  });
}

}  // namespace moe
