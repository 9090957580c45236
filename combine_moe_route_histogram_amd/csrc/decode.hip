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

constexpr int kMaxWaves = 8;            // waves of a product block: 8, or 4 side by side
constexpr int kRedRows = 8;             // rows whose sums go through LDS at once
constexpr int kRouteThreads = 1024;
constexpr int kHeadTokens = 32;   // routing inside the first product's blocks up to here
constexpr int kTailTokens = 4;    // the output's sum inside the second product up to here
constexpr double kWideBlocks = 224;

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

// Wave maxima by DPP row shifts and row broadcasts (lane 63 ends with them).
template <int N>
__device__ __forceinline__ void wave_max_u32(uint32_t (&v)[N]) {
#define MOE_DPP_MAX(ctrl)                                                                           \
  _Pragma("unroll") for (int i = 0; i < N; ++i) {                                                   \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[i], ctrl, 0xF, 0xF, true);   \
    v[i] = o > v[i] ? o : v[i];                                                                     \
  }
  MOE_DPP_MAX(0x111) MOE_DPP_MAX(0x112) MOE_DPP_MAX(0x114) MOE_DPP_MAX(0x118)   // row_shr 1, 2, 4, 8
  MOE_DPP_MAX(0x142) MOE_DPP_MAX(0x143)                                         // row_bcast 15, 31
#undef MOE_DPP_MAX
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (uint32_t)__builtin_amdgcn_readlane((int)v[i], 63);
}

// One wave's top-k of TOK tokens t, t + dt, ... below T: lane l holds the
// logits of experts l, l + 64, ... (EC chunks).  Writes the K picks and their
// weights of the tokens below n; the same keys, order and weight arithmetic as
// moe_route, hence the same bits.  A pick is a chain of dependent lane
// operations, so several tokens at once hide each other's latency; the logits
// are asked for before n is known.
template <int EC, int TOK>
__device__ __forceinline__ void route_tokens(const float* __restrict__ logits, int t, int dt, int T, int n, int E,
                                             int K, int lane, int32_t* __restrict__ idx, float* __restrict__ w) {
  uint32_t key[TOK][EC], first[TOK];
  float pl[TOK][EC];
  int pe[TOK][EC];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    first[i] = 0u;
#pragma unroll
    for (int c = 0; c < EC; ++c) {
      pl[i][c] = 0.f;
      pe[i][c] = 0;
      key[i][c] = t + i * dt < T && lane + kWave * c < E
                      ? logit_key(logits[(int64_t)(t + i * dt) * E + lane + kWave * c]) : 0u;
    }
  }
  for (int k = 0; k < K; ++k) {
    uint32_t best[TOK];
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      best[i] = key[i][0];
#pragma unroll
      for (int c = 1; c < EC; ++c) best[i] = key[i][c] > best[i] ? key[i][c] : best[i];
    }
    wave_max_u32<TOK>(best);
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      int e = -1;
#pragma unroll
      for (int c = 0; c < EC; ++c) {   // the lowest expert that holds the maximum
        const uint64_t m = __ballot(key[i][c] == best[i]);
        if (e < 0 && m) e = kWave * c + __builtin_ctzll(m);
      }
      if (k == 0) first[i] = best[i];
#pragma unroll
      for (int c = 0; c < EC; ++c) {
        if (lane + kWave * c == e) key[i][c] = 0u;
        if (lane + kWave * c == k) {
          pl[i][c] = key_logit(best[i]);
          pe[i][c] = e;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    float ex[EC], sum = 0.f;
#pragma unroll
    for (int c = 0; c < EC; ++c) ex[c] = expf(pl[i][c] - key_logit(first[i]));
    for (int k = 0; k < K; ++k) {   // in the order of the picks
      float v = lane_float(ex[0], k & (kWave - 1));
#pragma unroll
      for (int c = 1; c < EC; ++c)
        if (k >= kWave * c) v = lane_float(ex[c], k & (kWave - 1));
      sum += v;
    }
#pragma unroll
    for (int c = 0; c < EC; ++c)
      if (t + i * dt < n && lane + kWave * c < K) {
        const int64_t at = (int64_t)(t + i * dt) * K + lane + kWave * c;
        idx[at] = pe[i][c];
        w[at] = ex[c] / sum;
      }
  }
}

// All tokens, by the block's `waves` waves.
__device__ __forceinline__ void route_all(const DecodeArgs& a, int n, int wave, int waves, int lane, int32_t* idx,
                                          float* w) {
  if (a.E > kWave) {
    for (int t = wave; t < a.T; t += waves)
      route_tokens<kMaxExperts / kWave, 1>(a.logits, t, waves, a.T, n, a.E, a.K, lane, idx, w);
  } else if (a.T <= waves) {
    if (wave < a.T) route_tokens<1, 1>(a.logits, wave, waves, a.T, n, a.E, a.K, lane, idx, w);
  } else {
    for (int t = wave; t < a.T; t += 4 * waves)
      route_tokens<1, 4>(a.logits, t, waves, a.T, n, a.E, a.K, lane, idx, w);
  }
}

__device__ __forceinline__ int tokens_in_use(const DecodeArgs& a) {
  return a.n_tokens ? min(max(*a.n_tokens, 0), a.T) : a.T;
}

// The work is a list of entries, each some rows (at most row_tile) of one
// expert: entries[i] = {group, rows}, their row ids at lists[i * row_tile].  A
// row id is the pair t K + k, or R + s T + t for shared expert s.  The order
// of an entry's rows comes from a counter; no result depends on it (a row's
// sums do not mix with its neighbours').
//
// One block routes all tokens and writes the list (batches beyond what each
// product block routes for itself, see decode_plan).
__global__ __launch_bounds__(kRouteThreads) void decode_route_kernel(DecodeArgs a, int row_tile) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], fill[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int E = a.E, K = a.K, n = tokens_in_use(a);
  if (tid < kMaxExperts) count[tid] = fill[tid] = 0;
  route_all(a, n, wave, kRouteThreads / kWave, lane, a.topk_idx, a.topk_w);
  __syncthreads();
  const int pairs = n * K;
  for (int p = tid; p < pairs; p += kRouteThreads) atomicAdd(&count[a.topk_idx[p]], 1);
  __syncthreads();
  if (tid < kMaxExperts) first[tid] = (count[tid] + row_tile - 1) / row_tile;
  __syncthreads();
  for (int o = 1; o < kMaxExperts; o <<= 1) {   // entries up to each expert
    int f = 0;
    if (tid < kMaxExperts && tid >= o) f = first[tid - o];
    __syncthreads();
    if (tid < kMaxExperts) first[tid] += f;
    __syncthreads();
  }
  const int routed = first[kMaxExperts - 1];
  __syncthreads();
  if (tid < kMaxExperts) {
    const int c = count[tid], m = (c + row_tile - 1) / row_tile, f0 = first[tid] - m;
    for (int i = 0; i < m; ++i) a.entries[f0 + i] = make_int2(tid, min(row_tile, c - i * row_tile));
    first[tid] = f0;
  }
  const int per = (n + row_tile - 1) / row_tile;   // entries of one shared expert
  for (int i = tid; i < a.Ns * per; i += kRouteThreads) {
    const int s = i / per, r = (i - s * per) * row_tile;
    a.entries[routed + i] = make_int2(E + s, min(row_tile, n - r));
  }
  for (int i = tid; i < a.Ns * n; i += kRouteThreads) {
    const int s = i / n, t = i - s * n;
    a.lists[(int64_t)(routed + s * per + t / row_tile) * row_tile + t % row_tile] = a.R + s * a.T + t;
  }
  if (tid == 0) *a.n_entries = routed + a.Ns * per;
  __syncthreads();
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int e = a.topk_idx[p], at = atomicAdd(&fill[e], 1);
    a.lists[(int64_t)(first[e] + at / row_tile) * row_tile + at % row_tile] = p;
  }
}

// The same list, entry by entry, by every block of the first product for
// itself (at most one pair a thread).  It costs a block the latency of one
// load and of its picks; a launch of its own costs more, on the host too.
// Writes what the second product and the caller need: the entry and its rows
// by the blocks of column tile 0, the picks by the very first block.
template <int NW>
struct BlockRoute {
  int32_t idx[NW * kWave];
  float w[NW * kWave];
  int32_t list[32];
  int32_t count[kMaxExperts];
  int32_t below[NW];
};
template <int NW>
__device__ __forceinline__ bool block_route(const DecodeArgs& a, BlockRoute<NW>& r, int entry, bool write_entry,
                                            bool write_picks, int row_tile, int tid, int& group, int& rows) {
  const int lane = tid & (kWave - 1), wave = tid / kWave;
  const int E = a.E, K = a.K, n = tokens_in_use(a), pairs = n * K;
  for (int e = tid; e < kMaxExperts; e += NW * kWave) r.count[e] = 0;
  route_all(a, n, wave, NW, lane, r.idx, r.w);
  __syncthreads();
  if (a.T == 1) {   // each pick is an entry of its own, and so is each shared expert
    if (write_picks) {
      if (tid < pairs) {
        a.topk_idx[tid] = r.idx[tid];
        a.topk_w[tid] = r.w[tid];
      }
      if (tid == 0) *a.n_entries = n * (K + a.Ns);
    }
    if (entry >= n * (K + a.Ns)) return false;
    const bool pick = entry < K;
    group = pick ? r.idx[entry] : E + entry - K;
    rows = 1;
    __syncthreads();
    if (tid == 0) r.list[0] = pick ? entry : a.R + entry - K;
    __syncthreads();
    if (write_entry && tid == 0) {
      a.entries[entry] = make_int2(group, 1);
      a.lists[entry * row_tile] = r.list[0];
    }
    return true;
  }
  const int mine = tid < pairs ? r.idx[tid] : -1;
  if (tid < pairs) atomicAdd(&r.count[mine], 1);
  __syncthreads();
  // the expert that holds this entry, and which of its entries it is
  int seen = 0, e = -1, part = 0;
  for (int c = 0; c < E; c += kWave) {
    const int cnt = lane + c < E ? r.count[lane + c] : 0;
    const int m = (cnt + row_tile - 1) / row_tile;
    int before, in;   // entries of the chunk's lower experts, and of all of them
    if (a.T <= row_tile) {
      const uint64_t mask = __ballot(m != 0);
      before = __popcll(mask & ((1ull << lane) - 1));
      in = __popcll(mask);
    } else {
      before = m;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(before, o, kWave);
        if (lane >= o) before += v;
      }
      in = __builtin_amdgcn_readlane(before, kWave - 1);
      before -= m;
    }
    const int want = entry - seen;
    if (e < 0 && want < in) {
      const int l = __builtin_ctzll(__ballot(want >= before && want < before + m));
      e = c + l;
      part = want - __builtin_amdgcn_readlane(before, l);
      rows = min(row_tile, __builtin_amdgcn_readlane(cnt, l) - part * row_tile);
    }
    seen += in;
  }
  const int per = (n + row_tile - 1) / row_tile, total = seen + a.Ns * per;
  if (write_picks) {
    if (tid < pairs) {
      a.topk_idx[tid] = mine;
      a.topk_w[tid] = r.w[tid];
    }
    if (tid == 0) *a.n_entries = total;
  }
  if (entry >= total) return false;
  if (e >= 0) {   // the entry's rows: the expert's pairs in order, from part * row_tile on
    group = e;
    const uint64_t mask = __ballot(mine == e);
    if (lane == 0) r.below[wave] = __popcll(mask);
    __syncthreads();
    int rank = __popcll(mask & ((1ull << lane) - 1)) - part * row_tile;
    for (int v = 0; v < wave; ++v) rank += r.below[v];
    if (mine == e && rank >= 0 && rank < row_tile) r.list[rank] = tid;
  } else {
    const int s = (entry - seen) / per, t0 = (entry - seen - s * per) * row_tile;
    group = E + s;
    rows = min(row_tile, n - t0);
    if (tid < rows) r.list[tid] = a.R + s * a.T + t0 + tid;
  }
  __syncthreads();
  if (write_entry) {
    if (tid == 0) a.entries[entry] = make_int2(group, rows);
    if (tid < rows) a.lists[entry * row_tile + tid] = r.list[tid];
  }
  return true;
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

// A lane's place: its column(s) in row 0 of the matrix it reads, and its rows.
template <int F, bool UP, int NT>
struct Lane {
  const char* w[fmt_mx(F) && UP ? 2 : 1];   // 4 bit: in W1 and W3 (up) or in W2
  const char* sc[fmt_mx(F) && UP ? 2 : 1];  // scales
  int groups;                               // 4 bit: column groups inside the matrix (whole ones: N % 32 == 0)
  bool col_ok;                              // else: the lane's columns are inside
  const char* act[NT];                      // null: no such row
};

template <int F, bool UP, int NT>
__device__ __forceinline__ void load_stage(Stage<F, UP, NT>& s, const Lane<F, UP, NT>& L, int step, int q,
                                           int Kd, int N, int64_t plane) {
  const u32x4 zero = {0, 0, 0, 0};
  if constexpr (fmt_mx(F)) {
    const int kb = 4 * step + q;
    const bool ok = kb < Kd / kMxGroup;
    const int64_t at = (int64_t)kb * N;
#pragma unroll
    for (int j = 0; j < fmt_groups(F); ++j) {
      s.w[j] = zero;
      s.s[j] = 127;
      const int jj = UP ? j >> 1 : j;
      if (ok && jj < L.groups) {
        s.w[j] = ld16_stream(L.w[UP ? j & 1 : 0] + at * kMxCodeBytes + jj * 16 * kMxCodeBytes);
        s.s[j] = static_cast<const uint8_t*>(static_cast<const void*>(L.sc[UP ? j & 1 : 0]))[at + jj * 16];
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      constexpr int V = act_vecs(F, UP);
#pragma unroll
      for (int v = 0; v < V; ++v) s.act[nt][v] = zero;
      if (L.act[nt] && ok) {
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
      if (ok && L.col_ok) s.w[i] = ld16_stream(p + (int64_t)i * N * B);
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

// out[t] of one 4-column vector: sum over the pairs k in order, then the
// shared rows, each over its k slices; item i = (pair, slice).
__device__ __forceinline__ int64_t item_row(const DecodeArgs& a, int t, int k) {
  return k < a.K ? (int64_t)t * a.K + k : (int64_t)a.R + (int64_t)(k - a.K) * a.T + t;
}
constexpr int kItemBatch = 8;   // loads in flight per thread
__device__ __forceinline__ f32x4 combine_items(const DecodeArgs& a, int slices, int t, int c, int first, int stride) {
  const int64_t RA = (int64_t)a.R + (int64_t)a.Ns * a.T;
  const int items = (a.K + a.Ns) * slices;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = first; i0 < items; i0 += stride * kItemBatch) {
    f32x4 v[kItemBatch];
    float w[kItemBatch];
#pragma unroll
    for (int u = 0; u < kItemBatch; ++u) {
      const int i = i0 + u * stride;
      v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      w[u] = 0.f;
      if (i < items) {
        const int k = i / slices, s = i - k * slices;
        v[u] = *reinterpret_cast<const f32x4*>(a.y + ((int64_t)s * RA + item_row(a, t, k)) * a.H + c);
        w[u] = k < a.K ? a.topk_w[(int64_t)t * a.K + k] : 1.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kItemBatch; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = fmaf(w[u], v[u][j], sum[j]);
  }
  return sum;
}
template <bool BF16>
__device__ __forceinline__ void store_out(const DecodeArgs& a, int t, int c, const f32x4& sum) {
  if constexpr (!BF16) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + (int64_t)t * a.H + c) = sum;
  } else {
    u32x2 v;
    v[0] = pack_bf16x2(sum[0], sum[1]);
    v[1] = pack_bf16x2(sum[2], sum[3]);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + (int64_t)t * a.H + c) = v;
  }
}

// One block: one entry (up to 16 NT rows of one expert) x one tile of columns x
// one k slice.  Its NW waves are CW column tiles next to each other x NW / CW
// shares of the k steps, whose sums are added in wave order through LDS.
//
// HEAD: the first product's blocks route for themselves (block_route).
// TAIL: the second's add up the output of a column tile when they are its
// last: a block stores its sums coherently, waits until they are written, and
// counts itself; whoever counts last reads them all.  Nobody waits for
// anybody.  The first product's first block clears the counters.
template <int F, bool UP, int NT, int NW, int CW, bool FUSED>
__global__ __launch_bounds__(NW * kWave, NT == 1 && (!fmt_mx(F) || (UP && F == kFmtMxBf16)) ? 4 : 2) void decode_ffn_kernel(DecodeArgs a, int tiles, int slices, int slice_steps) {
  constexpr bool HEAD = UP && FUSED, TAIL = !UP && FUSED;
  constexpr int G = fmt_groups(F), B = fmt_f32(F) ? 4 : 2, KW = NW / CW, kThreads = NW * kWave;
  constexpr int WCOLS = UP ? 8 * G : 16 * G, COLS = WCOLS * CW;   // columns of a wave, of the block
  __shared__ __align__(16) float red[NW * kRedRows * red_stride<F>()];
  __shared__ int last;
  static_assert(sizeof(BlockRoute<NW>) <= sizeof(red) && kThreads * 16 <= sizeof(red), "other uses of the sums' LDS");
  const int entry = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int m = lane & 15, q = lane >> 4;
  const int tile = blockIdx.x % tiles, slice = blockIdx.x / tiles;
  const int Kd = UP ? a.H : a.I, N = UP ? a.I : a.H;
  const int64_t RA = (int64_t)a.R + (int64_t)a.Ns * a.T;
  const int64_t plane = RA * a.I * 2;   // bytes between h's two bf16 planes
  int group, rows, ids[NT], n_entries = 0;   // ids: this lane's rows
  if (UP && blockIdx.x == 0 && entry == 0)
    for (int i = tid; i < a.n_done; i += kThreads) a.done[i * kDoneStride] = 0;
  if constexpr (HEAD) {
    BlockRoute<NW>& r = *reinterpret_cast<BlockRoute<NW>*>(red);
    if (!block_route(a, r, entry, blockIdx.x == 0, blockIdx.x == 0 && entry == 0, 16 * NT, tid, group, rows)) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ids[nt] = 16 * nt + m < rows ? r.list[16 * nt + m] : 0;
    __syncthreads();   // the list is read; its LDS becomes the sums'
  } else {
    n_entries = *a.n_entries;
    const int2 en = a.entries[entry];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ids[nt] = a.lists[(int64_t)entry * (16 * NT) + 16 * nt + m];
    if (entry >= n_entries) return;
    group = en.x;
    rows = en.y;
  }
  const bool shared = group >= a.E;
  const int g = shared ? group - a.E : group;
  const int col0 = tile * COLS + wave % CW * WCOLS;   // the wave's first column

  Lane<F, UP, NT> L;
  if constexpr (fmt_mx(F)) {
    const int64_t one = (int64_t)(Kd / kMxGroup) * N;   // groups of 32 of one matrix
#pragma unroll
    for (int i = 0; i < (UP ? 2 : 1); ++i) {
      const void* base = UP ? (i ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
      L.w[i] = static_cast<const char*>(base) + (g * one + col0 + m) * kMxCodeBytes;
      L.sc[i] = static_cast<const char*>(base) + (shared ? a.Ns : a.E) * one * kMxCodeBytes + g * one + col0 + m;
    }
    L.groups = (N - col0) / 16;
  } else {
    bool second;
    const int col = col0 + tile_col<F, UP>(0, m, second);
    const void* base = UP ? (second ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
    L.w[0] = static_cast<const char*>(base) + ((int64_t)g * Kd * N + col) * B;
    L.col_ok = col < N;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    L.act[nt] = nullptr;
    if (16 * nt + m < rows) {
      if constexpr (UP) {
        const int t = shared ? ids[nt] - a.R - g * a.T : ids[nt] / a.K;
        L.act[nt] = static_cast<const char*>(a.x) + (int64_t)t * a.H * B;
      } else {
        L.act[nt] = static_cast<const char*>(a.h) + (int64_t)ids[nt] * a.I * B;
      }
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
  int k = begin + wave / CW;
  if (k < end && col0 < N) {
    load_stage<F, UP, NT>(s0, L, k, q, Kd, N, plane);
    for (;;) {
      const bool more1 = k + KW < end;
      if (more1) load_stage<F, UP, NT>(s1, L, k + KW, q, Kd, N, plane);
      mma_stage<F, UP, NT>(s0, acc);
      if (!more1) break;
      const bool more0 = k + 2 * KW < end;
      if (more0) load_stage<F, UP, NT>(s0, L, k + 2 * KW, q, Kd, N, plane);
      mma_stage<F, UP, NT>(s1, acc);
      if (!more0) break;
      k += 2 * KW;
    }
  }

  constexpr int RS = red_stride<F>();
#pragma unroll
  for (int r0 = 0; r0 < 16 * NT; r0 += kRedRows) {   // kRedRows rows at a time
    const int nt = r0 / 16, n0 = r0 % 16, here = min(kRedRows, rows - r0);
    if (here <= 0) break;
    if (r0) __syncthreads();
    if (m >= n0 && m < n0 + here) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        *reinterpret_cast<f32x4*>(&red[(wave * kRedRows + m - n0) * RS + 16 * j + 4 * q]) = acc[nt][j];
    }
    __syncthreads();
    for (int o = tid; o < here * COLS; o += kThreads) {
      const int n = o / COLS, bc = o - n * COLS, cw = bc / WCOLS, c = bc - cw * WCOLS;
      int at, at3 = 0;
      if constexpr (fmt_mx(F)) {
        at = UP ? 32 * (c >> 4) + (c & 15) : c;
        at3 = at + 16;
      } else {
        at = 16 * (c % G) + c / G;
        at3 = at + 8;
      }
      const int64_t row = __shfl(ids[nt], n0 + n, 16);   // every group of 16 lanes holds the 16 ids
      float s = 0.f, s3 = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        s += red[((w * CW + cw) * kRedRows + n) * RS + at];
        if constexpr (UP) s3 += red[((w * CW + cw) * kRedRows + n) * RS + at3];
      }
      if (tile * COLS + bc >= N) continue;
      const int64_t dst = row * N + tile * COLS + bc;
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
      } else if constexpr (TAIL) {
        __hip_atomic_store(&a.y[(int64_t)slice * RA * N + dst], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      } else {
        a.y[(int64_t)slice * RA * N + dst] = s;
      }
    }
  }

  if constexpr (TAIL) {
    __builtin_amdgcn_s_waitcnt(0);   // this wave's sums are written
    __syncthreads();
    if (tid == 0)
      last = __hip_atomic_fetch_add(&a.done[tile * kDoneStride], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             n_entries * slices - 1;
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    // the threads = vectors of the tile x (tokens x parts of a token's items);
    // the parts' sums are added in order
    constexpr int VECS = COLS / 4, SLOTS = kThreads / VECS;
    const int n = tokens_in_use(a), items = (a.K + a.Ns) * slices;
    const int parts = max(1, min(SLOTS / a.T, items)), par = min(a.T, SLOTS);
    const int vec = tid % VECS, slot = tid / VECS, c = tile * COLS + 4 * vec;
    f32x4* part_sum = reinterpret_cast<f32x4*>(red);
    for (int t0 = 0; t0 < n; t0 += par) {
      const int t = t0 + slot / parts, part = slot % parts;
      const bool ok = slot < par * parts && t < n && c < a.H;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      if (ok) sum = combine_items(a, slices, t, c, part, parts);
      if (parts > 1) {
        __syncthreads();
        part_sum[tid] = sum;
        __syncthreads();
        if (ok && part == 0) {
          for (int i = 1; i < parts; ++i) sum += part_sum[tid + i * VECS];
        }
      }
      if (ok && part == 0) store_out<!fmt_f32(F)>(a, t, c, sum);
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecodeArgs a, int slices) {
  const int t = blockIdx.y;
  if (t >= tokens_in_use(a)) return;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (c < a.H) store_out<BF16>(a, t, c, combine_items(a, slices, t, c, 0, 1));
}

template <int F, bool UP, int NT, int NW, int CW>
hipError_t launch_product(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  const int tiles = UP ? p.up_tiles : p.down_tiles, slices = UP ? 1 : p.slices;
  const int steps = UP ? (a.H + fmt_step(F) - 1) / fmt_step(F) : p.slice_steps;
  const dim3 grid(tiles * slices, p.entries);
  if (UP ? p.head : p.tail)
    decode_ffn_kernel<F, UP, NT, NW, CW, true><<<grid, NW * kWave, 0, st>>>(a, tiles, slices, steps);
  else
    decode_ffn_kernel<F, UP, NT, NW, CW, false><<<grid, NW * kWave, 0, st>>>(a, tiles, slices, steps);
  return hipGetLastError();
}
template <int F, bool UP>
hipError_t launch_product(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  const bool wide = (UP ? p.up_waves : p.down_waves) == 4;
  if (p.row_tile == 16)
    return wide ? launch_product<F, UP, 1, 4, 4>(a, p, st) : launch_product<F, UP, 1, 8, 1>(a, p, st);
  return wide ? launch_product<F, UP, 2, 4, 4>(a, p, st) : launch_product<F, UP, 2, 8, 1>(a, p, st);
}

template <int F>
hipError_t launch_fmt(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if (!p.head) {
    decode_route_kernel<<<1, kRouteThreads, 0, st>>>(a, p.row_tile);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipError_t e = launch_product<F, true>(a, p, st);
  if (e == hipSuccess) e = launch_product<F, false>(a, p, st);
  if (p.tail || e != hipSuccess) return e;
  decode_combine_kernel<!fmt_f32(F)><<<dim3((a.H / 4 + 255) / 256, a.T), 256, 0, st>>>(a, p.slices);
  return hipGetLastError();
}

}  // namespace

DecodePlan decode_plan(bool is_bf16, bool mx, int T, int H, int E, int K, int I, int Ns) {
  const int f = mx ? (is_bf16 ? kFmtMxBf16 : kFmtMxF32) : (is_bf16 ? kFmtBf16 : kFmtF32);
  const int cols = 16 * fmt_groups(f), step = fmt_step(f);
  DecodePlan p;
  p.row_tile = T <= 16 ? 16 : 32;
  const int64_t R = (int64_t)T * K;
  p.head = R <= 4 * kWave && T <= kHeadTokens;   // a pair for every thread of the smaller blocks
  p.tail = T <= kTailTokens;
  const int busy = (int)(R < E ? R : E);   // experts with rows, at most
  // an expert with c rows has at most 1 + (c - 1) / row_tile entries
  p.entries = busy + (int)((R - busy) / p.row_tile) + Ns * ((T + p.row_tile - 1) / p.row_tile);
  // experts with rows as expected of even routing, and the shared ones
  double miss = 1.0;
  for (int t = 0; t < T; ++t) miss *= 1.0 - (double)K / E;
  const double groups = E * (1.0 - miss) + Ns;
  // Four column tiles side by side read 0.5 to 1 KiB of a row at once, where
  // that leaves enough blocks for the 256 CUs.
  const int up1 = (I + cols / 2 - 1) / (cols / 2), up4 = (I + 2 * cols - 1) / (2 * cols);
  p.up_waves = up4 * groups >= kWideBlocks ? 4 : 1;
  p.up_tiles = p.up_waves == 4 ? up4 : up1;
  const int down1 = (H + cols - 1) / cols, down4 = (H + 4 * cols - 1) / (4 * cols);
  const int steps = (I + step - 1) / step;
  p.down_waves = down4 * groups * steps >= 8 * kWideBlocks ? 4 : 1;
  p.down_tiles = p.down_waves == 4 ? down4 : down1;
  // k slices: enough blocks for the CUs twice over, each with a step for every wave
  const int shares = p.down_waves == 4 ? 1 : 8;
  int s = (int)(512.0 / (p.down_tiles * groups) + 0.999);
  const int most = (steps + shares - 1) / shares;
  s = s < 1 ? 1 : s > 8 ? 8 : s;
  if (s > most) s = most;
  p.slice_steps = (steps + s - 1) / s;
  p.slices = (steps + p.slice_steps - 1) / p.slice_steps;
  return p;
}

hipError_t launch_decode(bool is_bf16, bool mx, const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if (mx) return is_bf16 ? launch_fmt<kFmtMxBf16>(a, p, st) : launch_fmt<kFmtMxF32>(a, p, st);
  return is_bf16 ? launch_fmt<kFmtBf16>(a, p, st) : launch_fmt<kFmtF32>(a, p, st);
}

}  // namespace moe
