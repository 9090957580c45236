// The whole MoE layer for a few tokens (1..256): logits to output rows.
//
//   idx[t], g[t] = top-k of logits[t], softmax over the k picked
//   a = x_t W1_e, b = x_t W3_e, h = silu(a) b, y = h W2_e      for e in idx[t] and the shared experts
//   out[t] = sum_k g[t,k] y_k + sum_s y_s
//
// Bound: the bytes of the picked experts' weights, each read once.  An expert
// has a handful of rows, so the products are matrix times a few vectors; they
// run on MFMA all the same, with the weights as the 16-row operand and the
// (zero-padded) rows as the 16-column one: the matrix cores are idle
// otherwise, and one instruction takes the place of 16 x rows
// multiply-adds.  The weights go from memory to registers without LDS.
#include "common.hpp"
#include "decode.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kWaves = 8;               // waves of a product block, splitting its k steps
constexpr int kThreads = kWaves * kWave;
constexpr int kRouteThreads = 1024;

enum Fmt : int { kFmtBf16 = 0, kFmtF32 = 1, kFmtMxBf16 = 2, kFmtMxF32 = 3 };
constexpr bool fmt_mx(int f) { return f >= kFmtMxBf16; }
constexpr bool fmt_f32(int f) { return f == kFmtF32 || f == kFmtMxF32; }
// MFMA column groups (of 16 columns) a wave computes, and rows of a k step.
constexpr int fmt_groups(int f) { return f == kFmtBf16 ? 8 : 4; }
constexpr int fmt_step(int f) { return fmt_mx(f) ? 128 : 32; }

// ------------------------------------------------------------------ routing

// Order-preserving image of a logit as in the routing kernels (-0.0 on +0.0),
// but at least 1: 0 marks an expert that is picked already or not there, so
// the picks are distinct experts whatever the logits hold.
__device__ __forceinline__ uint32_t logit_key(float l) {
  uint32_t u = __float_as_uint(l);
  if ((u << 1) == 0u) u = 0u;
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return u ? u : 1u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Wave maximum by DPP row shifts and row broadcasts (lane 63 ends with it).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_DPP_MAX(ctrl)                                                                    \
  {                                                                                          \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true); \
    v = o > v ? o : v;                                                                       \
  }
  MOE_DPP_MAX(0x111) MOE_DPP_MAX(0x112) MOE_DPP_MAX(0x114) MOE_DPP_MAX(0x118)   // row_shr 1, 2, 4, 8
  MOE_DPP_MAX(0x142) MOE_DPP_MAX(0x143)                                         // row_bcast 15, 31
#undef MOE_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One wave's top-k of a token: lane l holds the logits of experts l, l + 64,
// ... (EC chunks).  Writes the K picks and their weights; the same keys, order
// and weight arithmetic as moe_route, hence the same bits.
template <int EC>
__device__ __forceinline__ void route_token(const float* __restrict__ row, int E, int K, int lane,
                                            int32_t* __restrict__ idx, float* __restrict__ w) {
  uint32_t key[EC];
#pragma unroll
  for (int c = 0; c < EC; ++c) key[c] = lane + kWave * c < E ? logit_key(row[lane + kWave * c]) : 0u;
  float l0 = 0.f, zsum = 0.f, pl[EC];
  int pe[EC];
#pragma unroll
  for (int c = 0; c < EC; ++c) {
    pl[c] = 0.f;
    pe[c] = 0;
  }
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int c = 1; c < EC; ++c) best = key[c] > best ? key[c] : best;
    best = wave_max_u32(best);
    int e = -1;
#pragma unroll
    for (int c = 0; c < EC; ++c) {   // the lowest expert that holds the maximum
      const uint64_t m = __ballot(key[c] == best);
      if (e < 0 && m) e = kWave * c + __builtin_ctzll(m);
    }
    const float l = key_logit(best);
    if (k == 0) l0 = l;
    zsum += expf(l - l0);
#pragma unroll
    for (int c = 0; c < EC; ++c) {
      if (lane + kWave * c == e) key[c] = 0u;
      if (lane + kWave * c == k) {
        pl[c] = l;
        pe[c] = e;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < EC; ++c)
    if (lane + kWave * c < K) {
      idx[lane + kWave * c] = pe[c];
      w[lane + kWave * c] = expf(pl[c] - l0) / zsum;
    }
}

// One block routes all tokens and lists the work: the rows of every expert
// that has some (expert-contiguous), cut into entries of at most row_tile
// rows.  A row's place among its expert's rows is taken from an LDS counter;
// no result depends on it (a row's sums do not mix with its neighbours').
template <int EC>
__global__ __launch_bounds__(kRouteThreads) void decode_route_kernel(DecodeArgs a, int row_tile) {
  __shared__ int count[kMaxExperts], start[kMaxExperts], first[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int E = a.E, K = a.K;
  int n = a.T;
  if (a.n_tokens) n = min(max(*a.n_tokens, 0), a.T);
  if (tid < kMaxExperts) count[tid] = 0;
  for (int t = wave; t < n; t += kRouteThreads / kWave)
    route_token<EC>(a.logits + (int64_t)t * E, E, K, lane, a.topk_idx + (int64_t)t * K,
                    a.topk_w + (int64_t)t * K);
  __syncthreads();
  const int pairs = n * K;
  for (int p = tid; p < pairs; p += kRouteThreads) a.slot[p] = atomicAdd(&count[a.topk_idx[p]], 1);
  __syncthreads();
  // prefix sums over the experts: rows, and entries
  if (tid < kMaxExperts) {
    start[tid] = count[tid];
    first[tid] = (count[tid] + row_tile - 1) / row_tile;
  }
  __syncthreads();
  for (int o = 1; o < kMaxExperts; o <<= 1) {
    int s = 0, f = 0;
    if (tid < kMaxExperts && tid >= o) {
      s = start[tid - o];
      f = first[tid - o];
    }
    __syncthreads();
    if (tid < kMaxExperts) {
      start[tid] += s;
      first[tid] += f;
    }
    __syncthreads();
  }
  if (tid < kMaxExperts) {   // exclusive from here on: start[e] - count[e]
    const int c = count[tid], s0 = start[tid] - c, m = (c + row_tile - 1) / row_tile, f0 = first[tid] - m;
    for (int i = 0; i < m; ++i)
      a.entries[f0 + i] = make_int4(tid, s0 + i * row_tile, min(row_tile, c - i * row_tile), 0);
    start[tid] = s0;
  }
  const int routed = first[kMaxExperts - 1];
  const int per = (n + row_tile - 1) / row_tile;   // entries of one shared expert
  for (int i = tid; i < a.Ns * per; i += kRouteThreads) {
    const int s = i / per, r = (i - s * per) * row_tile;
    a.entries[routed + i] = make_int4(a.E + s, a.R + s * a.T + r, min(row_tile, n - r), 0);
  }
  if (tid == 0) *a.n_entries = routed + a.Ns * per;
  __syncthreads();
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int row = start[a.topk_idx[p]] + a.slot[p];
    a.slot[p] = row;
    a.row_token[row] = p / K;
  }
}

// ----------------------------------------------------------------- products

__device__ __forceinline__ bf16x8 as_bf16x8(const u32x4& v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ u32x4 ld16_stream(const void* p) {
  return __builtin_nontemporal_load(static_cast<const u32x4*>(p));
}

// x = hi + lo (+ lo2), each part a bf16: what a rounding leaves is exact in
// float32, so two parts keep 16 bits of it and three all 24.
template <int P>
__device__ __forceinline__ void split_bf16(const float* f, u32x4* part) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = f[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t v = pack_bf16x2(r[2 * d], r[2 * d + 1]);
      part[p][d] = v;
      r[2 * d] -= __uint_as_float(v << 16);
      r[2 * d + 1] -= __uint_as_float(v & 0xFFFF0000u);
    }
  }
}

// bf16 parts of the row operand: x is bf16 already; h keeps two parts, so the
// second product sees it to 16 bits instead of 8; float32 rows on 4-bit
// weights keep all three.
constexpr int act_parts(int f, bool up) { return f == kFmtMxF32 ? 3 : fmt_f32(f) ? 1 : up ? 1 : 2; }
// 16-byte vectors of a lane's row operand per k step.
constexpr int act_vecs(int f, bool up) {
  return f == kFmtF32 ? 2 : f == kFmtMxF32 ? 8 : (fmt_mx(f) ? 4 : 1) * act_parts(f, up);
}

// One k step of a wave in registers: the weights and the rows' values.
template <int F, bool UP, int NT>
struct Stage {
  static constexpr int kLoads = fmt_mx(F) ? fmt_groups(F) : 8;
  u32x4 w[kLoads];
  uint32_t s[fmt_mx(F) ? fmt_groups(F) : 1];
  u32x4 act[NT][act_vecs(F, UP)];
};

// A lane's place: the matrix and column(s) it reads, and its rows.
template <int F, bool UP, int NT>
struct Lane {
  const char* w[fmt_mx(F) ? 2 : 1];        // mx: W1 and W3 (up) or W2 twice; else the lane's matrix
  const char* sc[fmt_mx(F) ? 2 : 1];       // scales
  bool col_ok[fmt_mx(F) ? fmt_groups(F) : 1];
  int32_t col[fmt_mx(F) ? fmt_groups(F) : 1];
  const char* act[NT];                     // null: no such row
};

template <int F, bool UP, int NT>
__device__ __forceinline__ void load_stage(Stage<F, UP, NT>& s, const Lane<F, UP, NT>& L, int step, int q,
                                           int Kd, int N, int64_t plane) {
  const u32x4 zero = {0, 0, 0, 0};
  if constexpr (fmt_mx(F)) {
    const int kb = 4 * step + q, KB = Kd / kMxGroup;
#pragma unroll
    for (int j = 0; j < fmt_groups(F); ++j) {
      s.w[j] = zero;
      s.s[j] = 127;
      if (kb < KB && L.col_ok[j]) {
        const int64_t at = (int64_t)kb * N + L.col[j];
        s.w[j] = ld16_stream(L.w[UP ? j & 1 : 0] + at * kMxCodeBytes);
        s.s[j] = static_cast<const uint8_t*>(static_cast<const void*>(L.sc[UP ? j & 1 : 0]))[at];
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      constexpr int V = act_vecs(F, UP);
#pragma unroll
      for (int v = 0; v < V; ++v) s.act[nt][v] = zero;
      if (L.act[nt] && kb < KB) {
        if constexpr (F == kFmtMxF32) {
          const char* p = L.act[nt] + (int64_t)kb * kMxGroup * 4;
#pragma unroll
          for (int v = 0; v < V; ++v) s.act[nt][v] = ld16(p + v * 16);
        } else {
          const char* p = L.act[nt] + (int64_t)kb * kMxGroup * 2;
#pragma unroll
          for (int v = 0; v < V; ++v) s.act[nt][v] = ld16(p + (v & 3) * 16 + (v >> 2) * plane);
        }
      }
    }
  } else {
    constexpr int B = fmt_f32(F) ? 4 : 2;
    const int k = fmt_step(F) * step + 8 * q;
    const bool ok = k < Kd;
    const char* p = L.w[0] + (int64_t)k * N * B;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.w[i] = zero;
      if (ok && L.col_ok[0]) s.w[i] = ld16_stream(p + (int64_t)i * N * B);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      constexpr int V = act_vecs(F, UP);
#pragma unroll
      for (int v = 0; v < V; ++v) s.act[nt][v] = zero;
      if (L.act[nt] && ok) {
        const char* r = L.act[nt] + (int64_t)k * B;
#pragma unroll
        for (int v = 0; v < V; ++v) s.act[nt][v] = ld16(r + (F == kFmtF32 ? (int64_t)v * 16 : v * plane));
      }
    }
  }
}

// acc[nt][j] += the step's weights (16 columns of group j) x rows (16 of tile nt).
template <int F, bool UP, int NT>
__device__ __forceinline__ void mma_stage(const Stage<F, UP, NT>& s, f32x4 (&acc)[NT][fmt_groups(F)]) {
  if constexpr (F == kFmtBf16) {
    // A lane holds 8 columns of 8 rows; an operand wants 8 rows of one column:
    // halves of two rows' words are put together, one v_perm per two weights.
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        u32x4 A;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          A[d] = __builtin_amdgcn_perm(s.w[2 * d + 1][r], s.w[2 * d][r], odd ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int p = 0; p < act_parts(F, UP); ++p)
            acc[nt][2 * r + odd] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                as_bf16x8(A), as_bf16x8(s.act[nt][p]), acc[nt][2 * r + odd], 0, 0, 0);
      }
    }
  } else if constexpr (F == kFmtF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[nt][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              __uint_as_float(s.w[i][j]), __uint_as_float(s.act[nt][i >> 2][i & 3]), acc[nt][j], 0, 0, 0);
  } else {
    constexpr int P = act_parts(F, UP);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 b[NT][P];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (F == kFmtMxF32) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(s.act[nt][2 * i + (e >> 2)][e & 3]);
          split_bf16<3>(f, b[nt]);
        } else {
#pragma unroll
          for (int p = 0; p < P; ++p) b[nt][p] = s.act[nt][4 * p + i];
        }
      }
#pragma unroll
      for (int j = 0; j < fmt_groups(F); ++j) {
        const float sc = __uint_as_float(s.s[j] << 23);
        u32x4 A;   // fp4 x 2^s is exact in bf16
        A[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.w[j][i], sc, 0));
        A[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.w[j][i], sc, 1));
        A[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.w[j][i], sc, 2));
        A[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.w[j][i], sc, 3));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int p = 0; p < P; ++p)
            acc[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(A), as_bf16x8(b[nt][p]), acc[nt][j], 0, 0, 0);
      }
    }
  }
}

// Column of (group j, MFMA row m) inside a wave's tile of 16 * groups columns
// of one matrix (down), or of W1 | W3 side by side (up; `second` = W3).
template <int F, bool UP>
__device__ __forceinline__ int tile_col(int j, int m, bool& second) {
  constexpr int G = fmt_groups(F);
  if constexpr (fmt_mx(F)) {
    second = UP && (j & 1);
    return UP ? 16 * (j >> 1) + m : 16 * j + m;
  } else {
    second = UP && m >= 8;
    return G * (UP ? m & 7 : m) + j;
  }
}

// The LDS index of (wave, row n of 16, group j, MFMA row m): one padded row of
// 16 * groups sums per (wave, n).
template <int F>
constexpr int red_stride() { return 16 * fmt_groups(F) + 4; }

// One block: one entry (up to 16 NT rows of one expert) x one column tile x
// one k slice, its k steps spread over the 8 waves and the waves' sums added
// in wave order through LDS.
template <int F, bool UP, int NT>
__global__ __launch_bounds__(kThreads) void decode_ffn_kernel(DecodeArgs a, int tiles, int slice_steps) {
  constexpr int G = fmt_groups(F), B = fmt_f32(F) ? 4 : 2, COLS = UP ? 8 * G : 16 * G;
  __shared__ float red[kWaves * 16 * red_stride<F>()];
  const int entry = blockIdx.y;
  if (entry >= *a.n_entries) return;
  const int4 en = a.entries[entry];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int m = lane & 15, q = lane >> 4;
  const int tile = blockIdx.x % tiles, slice = blockIdx.x / tiles;
  const int Kd = UP ? a.H : a.I, N = UP ? a.I : a.H;
  const bool shared = en.x >= a.E;
  const int64_t RA = (int64_t)a.R + (int64_t)a.Ns * a.T;
  const int64_t plane = RA * a.I * 2;   // bytes between h's two bf16 planes

  Lane<F, UP, NT> L;
  if constexpr (fmt_mx(F)) {
    const int g = shared ? en.x - a.E : en.x, groups = shared ? a.Ns : a.E;
    const int64_t one = (int64_t)(Kd / kMxGroup) * N;   // groups of 32 of one matrix
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const void* base = UP ? (i ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
      L.w[i] = static_cast<const char*>(base) + g * one * kMxCodeBytes;
      L.sc[i] = static_cast<const char*>(base) + groups * one * kMxCodeBytes + g * one;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      bool second;
      L.col[j] = tile * COLS + tile_col<F, UP>(j, m, second);
      L.col_ok[j] = L.col[j] < N;
    }
  } else {
    bool second;
    const int col = tile * COLS + tile_col<F, UP>(0, m, second);
    const int g = shared ? en.x - a.E : en.x;
    const void* base = UP ? (second ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
    L.w[0] = static_cast<const char*>(base) + ((int64_t)g * Kd * N + col) * B;
    L.col[0] = col;
    L.col_ok[0] = col < N;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = 16 * nt + m;
    L.act[nt] = nullptr;
    if (n < en.z) {
      if constexpr (UP) {
        const int t = shared ? en.y + n - a.R - (en.x - a.E) * a.T : a.row_token[en.y + n];
        L.act[nt] = static_cast<const char*>(a.x) + (int64_t)t * a.H * B;
      } else {
        L.act[nt] = static_cast<const char*>(a.h) + (int64_t)(en.y + n) * a.I * B;
      }
      // dense: a lane's k offset is added per step (8 q rows inside it)
    }
  }

  f32x4 acc[NT][G];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[nt][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (Kd + fmt_step(F) - 1) / fmt_step(F);
  const int begin = slice * slice_steps, end = min(steps, begin + slice_steps);
  Stage<F, UP, NT> s0, s1;
  int k = begin + wave;
  if (k < end) {
    load_stage<F, UP, NT>(s0, L, k, q, Kd, N, plane);
    for (;;) {
      const bool more1 = k + kWaves < end;
      if (more1) load_stage<F, UP, NT>(s1, L, k + kWaves, q, Kd, N, plane);
      mma_stage<F, UP, NT>(s0, acc);
      if (!more1) break;
      const bool more0 = k + 2 * kWaves < end;
      if (more0) load_stage<F, UP, NT>(s0, L, k + 2 * kWaves, q, Kd, N, plane);
      mma_stage<F, UP, NT>(s1, acc);
      if (!more0) break;
      k += 2 * kWaves;
    }
  }

  constexpr int RS = red_stride<F>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rows = min(16, en.z - 16 * nt);
    if (rows <= 0) break;
    if (nt) __syncthreads();
    if (m < rows) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        *reinterpret_cast<f32x4*>(&red[(wave * 16 + m) * RS + 16 * j + 4 * q]) = acc[nt][j];
    }
    __syncthreads();
    for (int o = tid; o < rows * COLS; o += kThreads) {
      const int n = o / COLS, c = o - n * COLS;
      if (tile * COLS + c >= N) continue;
      const int64_t row = en.y + 16 * nt + n;
      int at, at3 = 0;
      if constexpr (fmt_mx(F)) {
        at = UP ? 32 * (c >> 4) + (c & 15) : c;
        at3 = at + 16;
      } else {
        at = 16 * (c % G) + c / G;
        at3 = at + 8;
      }
      float s = 0.f, s3 = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        s += red[(w * 16 + n) * RS + at];
        if constexpr (UP) s3 += red[(w * 16 + n) * RS + at3];
      }
      const int64_t dst = row * N + tile * COLS + c;
      if constexpr (UP) {
        const float hv = silu_f(s) * s3;
        if constexpr (fmt_f32(F)) {
          static_cast<float*>(a.h)[dst] = hv;
        } else {
          const uint32_t hi = f32_to_bf16(hv);
          uint16_t* hp = static_cast<uint16_t*>(a.h);
          hp[dst] = (uint16_t)hi;
          hp[RA * a.I + dst] = (uint16_t)f32_to_bf16(hv - bf16_to_f32(hi));
        }
      } else {
        a.y[(int64_t)slice * RA * N + dst] = s;
      }
    }
  }
}

// out[t] = sum_k g[t,k] (sum over slices of y[slot[t,k]]) + the shared rows',
// in that order; one rounding.  4 columns a thread.
template <typename S>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecodeArgs a, int slices) {
  const int t = blockIdx.y;
  if (a.n_tokens && t >= *a.n_tokens) return;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.H) return;
  const int64_t RA = (int64_t)a.R + (int64_t)a.Ns * a.T;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.K + a.Ns; ++k) {
    const int64_t row = k < a.K ? (int64_t)a.slot[(int64_t)t * a.K + k] : a.R + (int64_t)(k - a.K) * a.T + t;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < slices; ++s) v += *reinterpret_cast<const f32x4*>(a.y + ((int64_t)s * RA + row) * a.H + c);
    const float w = k < a.K ? a.topk_w[(int64_t)t * a.K + k] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = fmaf(w, v[i], sum[i]);
  }
  S* out = static_cast<S*>(a.out) + (int64_t)t * a.H + c;
  if constexpr (sizeof(S) == 4) {
    *reinterpret_cast<f32x4*>(out) = sum;
  } else {
    u32x2 v;
    v[0] = pack_bf16x2(sum[0], sum[1]);
    v[1] = pack_bf16x2(sum[2], sum[3]);
    *reinterpret_cast<u32x2*>(out) = v;
  }
}

template <int F, int NT>
hipError_t launch_ffn(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  decode_ffn_kernel<F, true, NT><<<dim3(p.up_tiles, p.entries), kThreads, 0, st>>>(
      a, p.up_tiles, (a.H + fmt_step(F) - 1) / fmt_step(F));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  decode_ffn_kernel<F, false, NT><<<dim3(p.down_tiles * p.slices, p.entries), kThreads, 0, st>>>(
      a, p.down_tiles, p.slice_steps);
  return hipGetLastError();
}

template <int F>
hipError_t launch_ffn_nt(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  return p.row_tile == 16 ? launch_ffn<F, 1>(a, p, st) : launch_ffn<F, 2>(a, p, st);
}

}  // namespace

DecodePlan decode_plan(bool is_bf16, bool mx, int T, int H, int E, int K, int I, int Ns) {
  const int f = mx ? (is_bf16 ? kFmtMxBf16 : kFmtMxF32) : (is_bf16 ? kFmtBf16 : kFmtF32);
  const int cols = 16 * fmt_groups(f), step = fmt_step(f);
  DecodePlan p;
  p.row_tile = T <= 16 ? 16 : 32;
  const int64_t R = (int64_t)T * K;
  const int busy = (int)(R < E ? R : E);   // experts with rows, at most
  // an expert with c rows has at most 1 + (c - 1) / row_tile entries
  p.entries = busy + (int)((R - busy) / p.row_tile) + Ns * ((T + p.row_tile - 1) / p.row_tile);
  p.up_tiles = (I + cols / 2 - 1) / (cols / 2);
  p.down_tiles = (H + cols - 1) / cols;
  const int steps = (I + step - 1) / step;
  // enough blocks for the 256 CUs twice over, each with work for its 8 waves
  const int want = (int)((512 + (int64_t)p.down_tiles * (busy + Ns) - 1) / ((int64_t)p.down_tiles * (busy + Ns)));
  int s = want < 1 ? 1 : want > 8 ? 8 : want;
  const int most = (steps + kWaves - 1) / kWaves;
  if (s > most) s = most;
  p.slice_steps = (steps + s - 1) / s;
  p.slices = (steps + p.slice_steps - 1) / p.slice_steps;
  return p;
}

hipError_t launch_decode(bool is_bf16, bool mx, const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if (a.E <= kWave)
    decode_route_kernel<1><<<1, kRouteThreads, 0, st>>>(a, p.row_tile);
  else
    decode_route_kernel<4><<<1, kRouteThreads, 0, st>>>(a, p.row_tile);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (mx) e = is_bf16 ? launch_ffn_nt<kFmtMxBf16>(a, p, st) : launch_ffn_nt<kFmtMxF32>(a, p, st);
  else e = is_bf16 ? launch_ffn_nt<kFmtBf16>(a, p, st) : launch_ffn_nt<kFmtF32>(a, p, st);
  if (e != hipSuccess) return e;
  const dim3 grid((a.H / 4 + 255) / 256, a.T);
  if (is_bf16) decode_combine_kernel<uint16_t><<<grid, 256, 0, st>>>(a, p.slices);
  else decode_combine_kernel<float><<<grid, 256, 0, st>>>(a, p.slices);
  return hipGetLastError();
}

}  // namespace moe
