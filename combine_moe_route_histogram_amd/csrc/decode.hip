// The whole MoE layer for a few tokens (1..256): logits to output rows.
//
//   idx[t], g[t] = top-k of logits[t], softmax over the k picked
//   a = x_t W1_e, b = x_t W3_e, h = silu(a) b, y = h W2_e      for e in idx[t] and the shared experts
//   out[t] = sum_k g[t,k] y_k + sum_s y_s
//
// Bound: the bytes of the picked experts' weights, read once for every entry of
// 8 to 64 rows that an expert has (see row_tile_of), so once where its rows fit
// into one.  An expert has a handful of rows, so the products are matrix times a
// few vectors; they run on MFMA all the same, with the weights as the 16-row
// operand and the (zero-padded) rows as the 16-column one: the matrix cores are
// idle otherwise, and one instruction takes the place of 16 x rows
// multiply-adds.  The weights go from memory to registers without LDS.
//
// Measured (times of a call, launches and gaps included; streaming reads reach
// 6.9 TB/s on this card): bf16 [4096, 14336] x 2 in 8 experts, 32 tokens 440 us,
// 6.4 TB/s; [2048, 1408] x 6 in 64 experts and 2 shared ones, one token 30.5 us,
// 4.5 TB/s, of which the routing, the two launches and the sum are about 7;
// 4-bit weights, the same 17.0 and, 200 tokens of 4 in 32 experts, 58 us.
#include "common.hpp"
#include "decode.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;               // waves of a product block
constexpr int kThreads = kWaves * kWave;
constexpr int kRedRows = 8;             // rows whose sums go through LDS at once
constexpr int kRouteThreads = 1024;

// The thresholds below, against other values: time of a call relative to the
// value that stands, mean (least to most) over the calls that it changes, of ten
// layers ([128, 256] x 2 in 8 experts; [224, 960] x 6 in 42 and 2 shared; [512,
// 2048] x 2 in 16 and 1; [1024, 4096] x 4 in 16; [2048, 1408] x 4 in 32; x 6 in
// 64 and 2; [2880, 2880] x 4 in 32; [3712, 928] x 3 in 8 and 1; [4096, 2048] x 8
// in 64 and 1; [4096, 14336] x 2 in 8), all four formats, 1 to 256 tokens.
//
// Up to kHeadTokens the first product's blocks pick the experts for themselves,
// up to kTailTokens the second product's last blocks add up the output; beyond,
// each has a launch.  1 in the place of 4 tokens: picks 1.07 (0.97 to 1.24), sum
// 1.09 (0.97 to 1.59).  8: picks 0.98 (0.85 to 1.07: small layers gain, [224, 960]
// f32 loses), sum 0.97 (0.85 to 1.06).
constexpr int kHeadTokens = 4;
constexpr int kTailTokens = 4;
//
// A block's width (see tile_width).  Rows of kLongRow bytes or more are long:
// 2048 1.07 (0.94 to 1.43), 8192 0.97 (0.82 to 1.11; f32 0.96, bf16 0.98).  Blocks
// that a width has to leave, long rows: 110 1.00 (0.75 to 1.30), 440 0.98 (0.82 to
// 1.12; the largest layer up to 1.12).  Short rows: 256 1.04 (0.95 to 1.09), 1024
// 0.98 (0.87 to 1.02; 12 calls).
constexpr int64_t kLongRow = 4096;      // bytes
constexpr int kLineBytes = 128;         // what the memory moves at once
constexpr double kFillBlocks = 220, kManyBlocks = 512;
//
// The down projection is cut along k for so many blocks, into so many slices at
// most.  150 blocks 0.98 (0.74 to 1.28): calls whose blocks are many already gain
// ([2048, 1408] x 4 in 32, f32, 8 tokens 146 -> 124 us), those of few, large
// experts lose (bf16 [4096, 14336] x 2 in 8, 32 and 64 tokens 437 -> 496, 464 ->
// 536; f32 [1024, 4096] x 4 in 16, 128 tokens 346 -> 445); no format gains or
// loses as a whole (0.98 to 0.99 each).
constexpr double kSliceBlocks = 400;
constexpr int kMaxSlices = 8;

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
// expert: entries[i] = {group, rows}, their row ids at lists[i * row_tile]; the
// entries that are not in use, up to the plan's bound, have no rows.  A
// row id is the pair t K + k, or R + s T + t for shared expert s.  The order
// of an entry's rows comes from a counter; no result depends on it (a row's
// sums do not mix with its neighbours').
//
// One block routes all tokens and writes the list (more pairs than a product's
// block lists for itself, see decode_plan).
__global__ __launch_bounds__(kRouteThreads) void decode_route_kernel(DecodeArgs a, int row_tile, int entries) {
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
  for (int i = routed + a.Ns * per + tid; i < entries; i += kRouteThreads) a.entries[i] = make_int2(0, 0);
  __syncthreads();
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int e = a.topk_idx[p], at = atomicAdd(&fill[e], 1);
    a.lists[(int64_t)(first[e] + at / row_tile) * row_tile + at % row_tile] = p;
  }
}

// The top-k alone, a wave a token: the list is then made by each block of the
// first product.
__global__ __launch_bounds__(kThreads) void decode_topk_kernel(DecodeArgs a) {
  const int lane = threadIdx.x & (kWave - 1), t = blockIdx.x * kWaves + threadIdx.x / kWave;
  if (t >= a.T) return;
  const int n = tokens_in_use(a);
  if (a.E <= kWave) route_tokens<1, 1>(a.logits, t, 1, a.T, n, a.E, a.K, lane, a.topk_idx, a.topk_w);
  else route_tokens<kMaxExperts / kWave, 1>(a.logits, t, 1, a.T, n, a.E, a.K, lane, a.topk_idx, a.topk_w);
}

// The same list, entry by entry, by every block of the first product for
// itself: from the picks, or (few tokens) from the logits.  It costs a block
// the latency of a load or two; a launch of its own costs more, on the host
// too, and one block that does it for all takes longer (200 tokens of 4 picks:
// 17 us).  Writes what the second product and the caller need: the entry and
// its rows by the blocks of column tile 0, the picks by the very first block.
constexpr int kListRounds = 8, kListPairs = kListRounds * kThreads;   // pairs a block can list
constexpr int kMaxRowTile = 64;
constexpr int kXcds = 8;   // blocks that follow each other go to the chiplets in turn
struct BlockRoute {
  int32_t idx[kThreads];   // picks and weights made here: at most a pair a thread
  float w[kThreads];
  int32_t list[kMaxRowTile];
  int32_t count[kMaxExperts];
  int32_t below[kListRounds * kWaves];
};
__device__ __forceinline__ bool block_route(const DecodeArgs& a, BlockRoute& r, int entry, bool write_entry,
                                            bool write_picks, int row_tile, int tid, int& group, int& rows) {
  const int lane = tid & (kWave - 1), wave = tid / kWave;
  const int E = a.E, K = a.K;
  int mine[kListRounds];   // the expert of pair tid + 256 i
  const int rounds = a.picked ? (a.R + kThreads - 1) / kThreads : 1;
  if (a.picked) {
#pragma unroll
    for (int i = 0; i < kListRounds; ++i) {
      const int p = tid + i * kThreads;
      mine[i] = p < a.R ? a.topk_idx[p] : -1;
    }
  }
  const int n = tokens_in_use(a), pairs = n * K;
  for (int e = tid; e < kMaxExperts; e += kThreads) r.count[e] = 0;
  if (!a.picked) route_all(a, n, wave, kWaves, lane, r.idx, r.w);
  __syncthreads();
  if (a.T == 1 && !a.picked) {   // each pick is an entry of its own, and so is each shared expert
    if (write_picks) {
      if (tid < pairs) {
        a.topk_idx[tid] = r.idx[tid];
        a.topk_w[tid] = r.w[tid];
      }
      if (tid == 0) *a.n_entries = n * (K + a.Ns);
    }
    if (entry >= n * (K + a.Ns)) {
      if (write_entry && tid == 0) a.entries[entry] = make_int2(0, 0);
      return false;
    }
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
  if (!a.picked) {
    mine[0] = r.idx[tid];
#pragma unroll
    for (int i = 1; i < kListRounds; ++i) mine[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kListRounds; ++i) {
    if (i >= rounds) break;
    if (tid + i * kThreads >= pairs) mine[i] = -1;
    if (mine[i] >= 0) atomicAdd(&r.count[mine[i]], 1);
  }
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
    if (!a.picked && tid < pairs) {
      a.topk_idx[tid] = mine[0];
      a.topk_w[tid] = r.w[tid];
    }
    if (tid == 0) *a.n_entries = total;
  }
  if (entry >= total) {
    if (write_entry && tid == 0) a.entries[entry] = make_int2(0, 0);
    return false;
  }
  if (e >= 0) {   // the entry's rows: the expert's pairs in order, from part * row_tile on
    group = e;
    uint64_t mask[kListRounds];
#pragma unroll
    for (int i = 0; i < kListRounds; ++i) {
      if (i >= rounds) break;
      mask[i] = __ballot(mine[i] == e);
      if (lane == 0) r.below[i * kWaves + wave] = __popcll(mask[i]);
    }
    __syncthreads();
    int sum = lane < rounds * kWaves ? r.below[lane] : 0;   // up to and with a wave's share
#pragma unroll
    for (int o = 1; o < kListRounds * kWaves; o <<= 1) {
      const int v = __shfl_up(sum, o, kWave);
      if (lane >= o) sum += v;
    }
#pragma unroll
    for (int i = 0; i < kListRounds; ++i) {
      if (i >= rounds) break;
      const int at = i * kWaves + __builtin_amdgcn_readfirstlane(wave);
      const int base = __builtin_amdgcn_readlane(sum, at) - __popcll(mask[i]) - part * row_tile;
      const int rank = base + __popcll(mask[i] & ((1ull << lane) - 1));
      if (mine[i] == e && rank >= 0 && rank < row_tile) r.list[rank] = tid + i * kThreads;
    }
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
__device__ __forceinline__ u32x4 ld16_stream(uint64_t address) {
  return __builtin_nontemporal_load(reinterpret_cast<const __attribute__((address_space(1))) u32x4*>(address));
}

// x = hi + lo (+ lo2), each part a bf16: what a rounding leaves is exact in
// float32, so two parts keep 16 bits of it and three all 24.  The first part of
// a number that would round to infinity is the largest bf16, and the rest, less
// than 2^120 there, is the other parts' (an infinite first part would leave
// -inf, and the row NaN).
constexpr float kMaxBf16 = 0x1.FEp127f;
__device__ __forceinline__ float first_part(float v) { return __builtin_amdgcn_fmed3f(v, -kMaxBf16, kMaxBf16); }
template <int P>
__device__ __forceinline__ void split_bf16(const float* f, u32x4* part) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = f[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t v = p == 0 ? pack_bf16x2(first_part(r[2 * d]), first_part(r[2 * d + 1]))
                                : pack_bf16x2(r[2 * d], r[2 * d + 1]);
      part[p][d] = v;
      r[2 * d] -= __uint_as_float(v << 16);
      r[2 * d + 1] -= __uint_as_float(v & 0xFFFF0000u);
    }
  }
}

// Rows of an entry at most.  4-bit weights with bf16 rows: up to 8 tokens the
// two parts of a row are columns of one operand, and beyond that the rows go
// through LDS; a kernel that holds the parts of 16 rows side by side would need
// 146 registers, three waves on a SIMD in the place of four.  (The way a row is
// summed must not depend on how many rows its expert has, so the choice is by
// the number of tokens.)
//
// Where the experts have kManyRows rows each or more, on average, an entry
// holds 64: the weights are read half as often, and through the caches, since
// other entries of the expert read them too.  (us a call with entries of 32,
// read past the caches, and of 64.  bf16 [4096, 14336] x 2 in 8 experts, 24, 32
// and 64 rows each: 519 and 655, 773 and 677, 1256 and 898; [2048, 1408] x 4 in
// 32, 8 and 32 rows: 104 and 129, 179 and 153.  f32 [4096, 14336] x 2 in 4, 24,
// 32, 48, 64 and 128 rows: 814 and 825, 1314 and 996, 1706 and 1370, 2016 and
// 2064, 3854 and 3293.  4 bit bf16 [4096, 14336] x 2 in 8, 24, 32 and 64 rows:
// 181 and 178, 225 and 201, 358 and 313; [2048, 1408] x 4 in 32, 8 and 32 rows:
// 44.0 and 46.7, 72.7 and 67.1; but with one expert of 64 rows, which leaves 112
// blocks, 58 and 76: there the 32.)  Shared experts do not count: they have all T
// rows and so several entries of 32 beyond 32 tokens, but entries of 64 for their
// sake take 1.19 times as long in the mean (0.92 to 1.83, 43 calls of the five
// layers above that have some), and weights through the caches 0.99 (plain
// formats; [2048, 1408] x 6 in 64 and 2, bf16, 64 tokens 212 -> 226 us, 256 tokens
// 278 -> 260).  Two bf16 parts of 64 rows do not fit into
// the registers of the plain products: there two blocks next to each other on
// one chiplet take 32 of an entry's rows each.  Three parts of them (f32 on 4
// bit) would take two thirds of a CU's LDS.
constexpr int kManyRows = 32;
constexpr int row_tile_of(int f, int nt) { return f == kFmtMxBf16 && nt == 1 ? 8 : 16 * nt; }

// bf16 parts of the row operand: x is bf16 already; h keeps two parts, so the
// second product sees it to 16 bits instead of 8; float32 rows on 4-bit
// weights keep all three.
constexpr int act_parts(int f, bool up) { return f == kFmtMxF32 ? 3 : fmt_f32(f) ? 1 : up ? 1 : 2; }
// 16-byte vectors of a lane's row operand per k step, with `parts` of them.
constexpr int act_vecs(int f, int parts) { return f == kFmtF32 ? 2 : f == kFmtMxF32 ? 8 : (fmt_mx(f) ? 4 : 1) * parts; }

// Steps in flight a wave.  (Four, with two waves on a SIMD in the place of
// four: 4-bit fine layer T=1 19.3 us against 17.8, wide bf16 T=32 441 against
// 436.)
constexpr int kStages = 2;

// One k step of a wave in registers: the weights and the rows' values.
template <int F, int P, int NT>
struct Stage {
  static constexpr int kLoads = fmt_mx(F) ? fmt_groups(F) : 8;
  u32x4 w[kLoads];
  uint32_t s;   // 4 bit: the scales of 4 columns next to each other (see lane_scales)
  u32x4 act[NT][act_vecs(F, P)];
};

// A lane's place: its column(s) in row 0 of the matrix it reads, and its rows.
// Lanes without a column or a row of their own repeat a valid one.
template <int F, bool UP, int NT>
struct Lane {
  const char* w[fmt_mx(F) && UP ? 2 : 1];   // 4 bit: in W1 and W3 (up) or in W2
  const char* sc;                           // 4 bit: this lane's 4 scales in row 0
  int groups;                               // 4 bit: column groups inside the matrix (whole ones: N % 32 == 0)
  const char* act[NT];
};

// What lanes behind the matrix's end, or behind the wave's last step, take for
// their rows' values.
__device__ const u32x4 kZeros[64] = {};
// A load of one of two places (a choice of pointers would make it a flat load,
// which waits for everything).
__device__ __forceinline__ u32x4 ld16_global(uint64_t address) {
  return *reinterpret_cast<const __attribute__((address_space(1))) u32x4*>(address);
}

// Nothing here is conditional: behind a branch the compiler no longer knows
// how many loads are in flight and waits for all of them before the next step
// is computed.  Weights outside the matrix repeat the last ones inside: what
// comes of such columns is not stored, and of the rows' values, places at or
// behind Kd are zeros, so weights repeated along k add nothing.  A step behind
// the wave's last one (real = false) loads zeros for both.
constexpr int step_len(int f) { return fmt_mx(f) ? kMxGroup : 8; }   // a lane's rows in one k step
template <int F, bool UP, int NT, bool CACHED, class S>
__device__ __forceinline__ void load_weights(S& s, const Lane<F, UP, NT>& L, int step, int q, int Kd, int N,
                                             bool real = true) {
  const int k = min(fmt_step(F) * step + step_len(F) * q, Kd - step_len(F));
  const uint64_t zeros = reinterpret_cast<uint64_t>(kZeros);
  if constexpr (fmt_mx(F)) {
    const int64_t at = (int64_t)(k / kMxGroup) * N;
    uint64_t p[UP ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (UP ? 2 : 1); ++i) p[i] = real ? reinterpret_cast<uint64_t>(L.w[i]) + at * kMxCodeBytes : zeros;
#pragma unroll
    for (int j = 0; j < fmt_groups(F); ++j) {
      const int jj = min(UP ? j >> 1 : j, L.groups - 1);
      s.w[j] = CACHED ? ld16_global(p[UP ? j & 1 : 0] + jj * 16 * kMxCodeBytes) : ld16_stream(p[UP ? j & 1 : 0] + jj * 16 * kMxCodeBytes);
    }
    const uint64_t sc = real ? reinterpret_cast<uint64_t>(L.sc) + at : zeros;
    s.s = *reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(sc);
  } else {
    constexpr int B = fmt_f32(F) ? 4 : 2;
    const uint64_t p = real ? reinterpret_cast<uint64_t>(L.w[0]) + (int64_t)k * N * B : zeros;
    const int64_t row = real ? (int64_t)N * B : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s.w[i] = CACHED ? ld16_global(p + i * row) : ld16_stream(p + i * row);
  }
}

// 4-bit weights: where column c of h is kept in its row.  Inside 128 columns the
// four lanes' groups of 32 take turns, 8 columns at a time, so what the lanes
// read of a row with one load lies together (64 bytes).  Rows are padded to
// whole 128s.
__device__ __forceinline__ int mx_h_place(int c) {
  return (c & ~127) | ((c >> 3) & 3) << 5 | ((c >> 5) & 3) << 3 | (c & 7);
}

template <int F, bool UP, int NT, bool CACHED, int NTL, int P>
__device__ __forceinline__ void load_stage(Stage<F, P, NTL>& s, const Lane<F, UP, NT>& L, int step, int q,
                                           int Kd, int N, bool real, int64_t plane) {
  constexpr int V = act_vecs(F, P), B = fmt_f32(F) ? 4 : 2, LEN = step_len(F);
  constexpr int PER = LEN * B / 16;   // vectors of a lane's values from one plane
  constexpr int V8 = 8 * B / 16;      // and of 8 values
  constexpr bool TURNS = fmt_mx(F) && !UP;   // h in the order of mx_h_place
  load_weights<F, UP, NT, CACHED>(s, L, step, q, Kd, N, real);
  const int at = fmt_step(F) * step + LEN * q, k = TURNS ? fmt_step(F) * step + 8 * q : at;
#pragma unroll
  for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
    for (int v0 = 0; v0 < V; v0 += PER) {
      const uint64_t p = reinterpret_cast<uint64_t>(L.act[nt]) + (int64_t)k * B + v0 / PER * plane;
      const uint64_t from = real && at < Kd ? p : reinterpret_cast<uint64_t>(kZeros);
#pragma unroll
      for (int v = 0; v < PER; ++v)
        s.act[nt][v0 + v] = ld16_global(from + (TURNS ? v / V8 * 32 * B + v % V8 * 16 : v * 16));
    }
}

// The scales 2^s of a lane's columns 16 j + m.  They are loaded 4 columns to a
// lane (lane m of the 16 that share a group of 32 rows has columns 4 m .. 4 m +
// 3; up: lanes 0..7 of W1, 8..15 of W3), one load in the place of one for each
// column group's bytes (which cost the wide layer's first product 13 % of its
// time), and handed to the lanes that want them.
template <int F, bool UP>
__device__ __forceinline__ void lane_scales(uint32_t loaded, int lane, float (&sc)[fmt_groups(F)]) {
  const int from = 4 * ((lane & 48) + ((lane & 15) >> 2)), shift = 8 * (lane & 3);
#pragma unroll
  for (int j = 0; j < fmt_groups(F); ++j) {
    const int at = UP ? 32 * (j & 1) + 16 * (j >> 1) : 16 * j;   // bytes from `from` to the source lane
    const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute(from + at, (int)loaded);
    sc[j] = __uint_as_float(((v >> shift) & 0xFFu) << 23);
  }
}

// acc[nt][j] += word i of the lanes' codes (8 rows of column group j) x the
// rows' values b of those 8; fp4 x 2^s is exact in bf16.
template <int F, int NT, int NTL, int P>
__device__ __forceinline__ void mma_mx(const u32x4 (&w)[fmt_groups(F)], const float (&sc)[fmt_groups(F)], int i,
                                       const u32x4 (&b)[NTL][P], f32x4 (&acc)[NT][fmt_groups(F)]) {
#pragma unroll
  for (int j = 0; j < fmt_groups(F); ++j) {
    u32x4 A;
    A[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][i], sc[j], 0));
    A[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][i], sc[j], 1));
    A[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][i], sc[j], 2));
    A[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][i], sc[j], 3));
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
      for (int p = 0; p < P; ++p)
        acc[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(A), as_bf16x8(b[nt][p]), acc[nt][j], 0, 0, 0);
  }
}

// acc[nt][j] += the step's weights (16 columns of group j) x rows (16 of tile nt).
template <int F, bool UP, int NT, int NTL, int P>
__device__ __forceinline__ void mma_stage(const Stage<F, P, NTL>& s, int lane, f32x4 (&acc)[NT][fmt_groups(F)]) {
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
        for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
          for (int p = 0; p < P; ++p)
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
        for (int nt = 0; nt < NTL; ++nt)
          acc[nt][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              __uint_as_float(s.w[i][j]), __uint_as_float(s.act[nt][i >> 2][i & 3]), acc[nt][j], 0, 0, 0);
  } else {
    float sc[fmt_groups(F)];
    lane_scales<F, UP>(s.s, lane, sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 b[NTL][P];
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt) {
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
      mma_mx<F, NT, NTL, P>(s.w, sc, i, b, acc);
    }
  }
}

// A wave's k steps first, first + stride, ... below end.  kStages steps are in
// flight; a step's loads follow the products of the one whose registers it
// takes, so every wait is for the oldest.  The count is filled up with steps
// that load zeros from one place.  (The barriers keep the scheduler from
// moving loads up, into registers of their own.)
template <int F, bool UP, int NT, bool CACHED, int NTL, int P = act_parts(F, UP)>
__device__ __forceinline__ void product_loop(const Lane<F, UP, NT>& L, f32x4 (&acc)[NT][fmt_groups(F)], int first,
                                             int stride, int end, int lane, int Kd, int N, int64_t plane) {
  constexpr int S = kStages;
  const int q = lane >> 4;
  Stage<F, P, NTL> s[S];
  auto load = [&](Stage<F, P, NTL>& st, int k) {
    load_stage<F, UP, NT, CACHED, NTL, P>(st, L, k, q, Kd, N, k < end, plane);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mma = [&](Stage<F, P, NTL>& st) {
    mma_stage<F, UP, NT, NTL, P>(st, lane, acc);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (first >= end) return;
#pragma unroll
  for (int i = 0; i < S; ++i) load(s[i], first + i * stride);
  mma(s[0]);
#pragma unroll 1
  for (int k = first + S * stride; k < end; k += S * stride) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      load(s[i], k + i * stride);
      mma(s[(i + 1) % S]);
    }
  }
#pragma unroll
  for (int i = 1; i < S; ++i) mma(s[i]);
}

// 4-bit weights, more than 8 tokens (f32: 16): the rows' values are the larger half of
// what a step loads, and each lane's 16 bytes of them lie 64 bytes from its
// neighbour's.  The block's waves, side by side on the same steps, load each
// value once, whole lines at a time, split it into its bf16 parts, and hand it
// on through LDS, one step ahead.
constexpr int kActPitch = 128 * 2 + 16;   // bytes of a row in LDS: 16 rows' vectors on different banks
template <int F, bool UP, int NT>
constexpr int act_bytes() { return act_parts(F, UP) * 16 * NT * kActPitch; }

template <int F>
struct WeightStage {
  u32x4 w[fmt_groups(F)];
  uint32_t s;
};

template <int F, bool UP, int NT, bool CACHED, int NTL>
__device__ __forceinline__ void shared_loop(const Lane<F, UP, NT>& L, f32x4 (&acc)[NT][fmt_groups(F)], int begin,
                                            int end, int tid, int Kd, int N, int64_t plane,
                                            const char* const (&src)[NT], char* lds) {
  constexpr int P = act_parts(F, UP), B = fmt_f32(F) ? 4 : 2, VECS = F == kFmtMxF32 ? 2 : P;
  const int lane = tid & (kWave - 1), m = lane & 15, q = lane >> 4, piece = tid & 15, row = tid >> 4;
  WeightStage<F> s0, s1;
  u32x4 v[NTL][VECS];   // this thread's 8 values of rows tid / 16, 16 + tid / 16
  auto load_w = [&](WeightStage<F>& s, int k) {
    load_weights<F, UP, NT, CACHED>(s, L, k, q, Kd, N);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_act = [&](int k) {
    const int at = fmt_step(F) * k + 8 * piece;
    const int col = UP ? at : fmt_step(F) * k + 32 * (piece & 3) + 8 * (piece >> 2);   // see mx_h_place
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const uint64_t p = reinterpret_cast<uint64_t>(src[nt]) + (int64_t)at * B + (F == kFmtMxF32 ? (int64_t)i * 16 : i * plane);
        v[nt][i] = ld16_global(col < Kd ? p : reinterpret_cast<uint64_t>(kZeros));
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto store_act = [&](int buf) {
    char* base = lds + buf * act_bytes<F, UP, NT>() + row * kActPitch + piece * 16;
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt) {
      u32x4 part[P];
      if constexpr (F == kFmtMxF32) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[nt][e >> 2][e & 3]);
        split_bf16<P>(f, part);
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) part[p] = v[nt][p];
      }
#pragma unroll
      for (int p = 0; p < P; ++p) st16(base + (p * NT + nt) * 16 * kActPitch, part[p]);
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mma = [&](const WeightStage<F>& s, int buf) {
    const char* base = lds + buf * act_bytes<F, UP, NT>() + m * kActPitch + q * (UP ? 64 : 16);
    float sc[fmt_groups(F)];
    lane_scales<F, UP>(s.s, lane, sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 b[NTL][P];
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
        for (int p = 0; p < P; ++p) b[nt][p] = ld16(base + (p * NT + nt) * 16 * kActPitch + i * (UP ? 16 : 64));
      mma_mx<F, NT, NTL, P>(s.w, sc, i, b, acc);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // steps behind the end: their weights are not used, and their values not read
  load_act(begin);
  load_w(s0, begin);
  load_w(s1, min(begin + 1, end - 1));
  store_act(0);
  int k = begin;
#pragma unroll 1
  for (; k + 2 < end; k += 2) {
    load_act(k + 1);
    mma(s0, 0);
    load_w(s0, k + 2);
    store_act(1);
    load_act(k + 2);
    mma(s1, 1);
    load_w(s1, min(k + 3, end - 1));
    store_act(0);
  }
  load_act(min(k + 1, end - 1));
  mma(s0, 0);
  store_act(1);
  if (k + 1 < end) mma(s1, 1);
  __syncthreads();   // the values are read; their LDS becomes the sums'
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

// All arguments in scalar registers at once: read where they are first used,
// each cache line of them is a trip of its own to host memory.
__device__ __forceinline__ void pin_args(const DecodeArgs& a) {
  asm volatile("" ::"s"(a.T), "s"(a.H), "s"(a.E), "s"(a.K), "s"(a.I), "s"(a.Ns), "s"(a.R), "s"(a.logits), "s"(a.x),
               "s"(a.w1), "s"(a.w3), "s"(a.w2), "s"(a.ws1), "s"(a.ws3), "s"(a.ws2), "s"(a.n_tokens), "s"(a.topk_idx),
               "s"(a.topk_w), "s"(a.out), "s"(a.entries), "s"(a.n_entries), "s"(a.lists), "s"(a.done), "s"(a.n_done),
               "s"(a.h), "s"(a.y), "s"(a.picked));
}

// One block: one entry (up to 16 NT rows of one expert; MANY: or 16 NT of an
// entry's 64) x one tile of columns x one k slice.  Its 4 waves are CW column tiles next to each other x 4 / CW
// shares of the k steps, whose sums are added in wave order through LDS.
//
// HEAD: the first product's blocks make the list for themselves (block_route).
// TAIL: the second's add up the output of a column tile when they are its
// last: a block stores its sums coherently, waits until they are written, and
// counts itself; whoever counts last reads them all.  Nobody waits for
// anybody.  The first product's first block clears the counters.
template <int F, bool UP, int NT, int CW, bool FUSED, bool MANY, bool CACHED>
__global__ __launch_bounds__(kThreads, NT == 1 && F != kFmtMxF32 ? 4 : 2) void decode_ffn_kernel(DecodeArgs a, int slices, int slice_steps) {
  constexpr bool HEAD = UP && FUSED, TAIL = !UP && FUSED;
  constexpr int G = fmt_groups(F), B = fmt_f32(F) ? 4 : 2, KW = kWaves / CW;
  constexpr int WCOLS = UP ? 8 * G : 16 * G, COLS = WCOLS * CW;   // columns of a wave, of the block
  constexpr bool SHARED = fmt_mx(F) && NT >= 2;   // rows' values by way of LDS
  // No sums to join, W1's and W3's in one lane: the sums are stored from the
  // registers (through LDS, 8 rows at a time: 4 bit, 200 tokens of 4 in 32
  // experts 64.4 us in the place of 59.2).  A plain kernel of 16 rows would
  // need a register too many.
  constexpr bool DIRECT = KW == 1 && !TAIL && (fmt_mx(F) || (!UP && NT > 1));
  constexpr int RT = row_tile_of(F, NT);           // rows of an entry at most
  constexpr int kRedFloats = kWaves * kRedRows * red_stride<F>();
  constexpr int kActFloats = SHARED ? act_bytes<F, UP, NT>() / 2 : 0;
  constexpr int kRouteFloats = HEAD ? (sizeof(BlockRoute) + 15) / 16 * 4 : 0;
  constexpr int kMainFloats = kRedFloats > kActFloats ? kRedFloats : kActFloats;
  __shared__ __align__(16) float red[kMainFloats > kRouteFloats ? kMainFloats : kRouteFloats];
  __shared__ int last;
  static_assert(kThreads * 16 <= sizeof(red), "the parts' sums of a token");
  pin_args(a);
  asm volatile("" ::"s"(slices), "s"(slice_steps));
  constexpr int HALVES = MANY ? kMaxRowTile / RT : 1;   // blocks that share an entry's rows
  const int entry = blockIdx.y, half = HALVES > 1 ? blockIdx.x / kXcds % HALVES : 0;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int m = lane & 15, q = lane >> 4;
  const int tile = HALVES > 1 ? blockIdx.x / (HALVES * kXcds) * kXcds + blockIdx.x % kXcds : blockIdx.x;
  const int slice = blockIdx.z;
  const int Kd = UP ? a.H : a.I, N = UP ? a.I : a.H;
  const int64_t RA = (int64_t)a.R + (int64_t)a.Ns * a.T;
  const int64_t Ih = fmt_mx(F) ? (a.I + 127) / 128 * 128 : a.I;   // a row of h
  const int64_t plane = RA * Ih * 2;   // bytes between h's two bf16 planes
  int group, rows, ids[NT];   // ids: this lane's rows
  if (UP && blockIdx.x == 0 && entry == 0)
    for (int i = tid; i < a.n_done; i += kThreads) a.done[i * kDoneStride] = 0;
  if constexpr (HEAD) {
    BlockRoute& r = *reinterpret_cast<BlockRoute*>(red);
    if (!block_route(a, r, entry, blockIdx.x == 0, blockIdx.x == 0 && entry == 0, RT, tid, group, rows)) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ids[nt] = r.list[min((16 * nt + m) % RT, rows - 1)];
    __syncthreads();   // the list is read; its LDS becomes the sums'
  } else {
    const int2 en = a.entries[entry];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ids[nt] = a.lists[(int64_t)(entry * HALVES + half) * RT + (16 * nt + m) % RT];
    group = en.x;
    rows = HALVES > 1 ? min(en.y - half * RT, RT) : en.y;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) asm volatile("" : "+v"(ids[nt]));   // asked for before rows is known
    if (rows <= 0 || (HALVES > 1 && tile * COLS >= N)) return;   // not in use
    // Lanes without a row repeat the first one's.  (Read outside the choice:
    // inside it, lane 0 would be switched off.)
    const int id0 = __builtin_amdgcn_readfirstlane(ids[0]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ids[nt] = (16 * nt + m) % RT < rows ? ids[nt] : id0;
  }
  group = __builtin_amdgcn_readfirstlane(group);
  rows = __builtin_amdgcn_readfirstlane(rows);
  const bool shared = group >= a.E;
  const int g = shared ? group - a.E : group;
  int col0 = tile * COLS + wave % CW * WCOLS;   // the wave's first column
  if constexpr (SHARED) col0 = min(col0, N - 32);   // all waves work: nothing is stored for one behind the end

  Lane<F, UP, NT> L;
  if constexpr (fmt_mx(F)) {
    const int64_t one = (int64_t)(Kd / kMxGroup) * N;   // groups of 32 of one matrix
#pragma unroll
    for (int i = 0; i < (UP ? 2 : 1); ++i) {
      const void* base = UP ? (i ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
      L.w[i] = static_cast<const char*>(base) + (g * one + col0 + m) * kMxCodeBytes;
      if (i == 0 || m >= 8)
        L.sc = static_cast<const char*>(base) + (shared ? a.Ns : a.E) * one * kMxCodeBytes + g * one + col0 +
               min(4 * (UP ? m & 7 : m), N - col0 - 4);
    }
    L.groups = (N - col0) / 16;
  } else {
    bool second;
    const int col = min(col0 + tile_col<F, UP>(0, m, second), N - G);
    const void* base = UP ? (second ? (shared ? a.ws3 : a.w3) : (shared ? a.ws1 : a.w1)) : (shared ? a.ws2 : a.w2);
    L.w[0] = static_cast<const char*>(base) + ((int64_t)g * Kd * N + col) * B;
  }
  auto row_values = [&](int id) {   // where a row's values begin
    if constexpr (UP) {
      const int t = shared ? id - a.R - g * a.T : id / a.K;
      return static_cast<const char*>(a.x) + (int64_t)t * a.H * B;
    } else {
      return static_cast<const char*>(a.h) + id * Ih * B;
    }
  };

  f32x4 acc[NT][G];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[nt][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (Kd + fmt_step(F) - 1) / fmt_step(F);
  const int begin = slice * slice_steps, end = min(steps, begin + slice_steps);
  if constexpr (SHARED) {
    const char* src[NT];   // lane l of every wave holds ids l % 16; this thread's rows are tid / 16 and 16 more
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) src[nt] = row_values(__shfl(ids[nt], tid >> 4, kWave));
    char* lds = reinterpret_cast<char*>(red);
    if (rows <= 16) shared_loop<F, UP, NT, CACHED, 1>(L, acc, begin, end, tid, Kd, N, plane, src, lds);
    else if (NT > 2 && rows <= 32) shared_loop<F, UP, NT, CACHED, 2>(L, acc, begin, end, tid, Kd, N, plane, src, lds);
    else if (NT > 3 && rows <= 48) shared_loop<F, UP, NT, CACHED, 3>(L, acc, begin, end, tid, Kd, N, plane, src, lds);
    else shared_loop<F, UP, NT, CACHED, NT>(L, acc, begin, end, tid, Kd, N, plane, src, lds);
  } else if (col0 < N) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) L.act[nt] = row_values(ids[nt]);
    if constexpr (RT == 8) {
      // The second part of row n is column n + 8 of the operand, in the place
      // of a second product.  (Lanes n and n + 8 have the same row.)
      if (!UP && m >= 8) L.act[0] += plane;
      product_loop<F, UP, NT, CACHED, 1, 1>(L, acc, begin + wave / CW, KW, end, lane, Kd, N, plane);
      if constexpr (!UP) {
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[0][j][i] += __shfl_xor(acc[0][j][i], 8, 16);
      }
    } else if (NT > 1 && rows <= 16) {
      product_loop<F, UP, NT, CACHED, 1>(L, acc, begin + wave / CW, KW, end, lane, Kd, N, plane);
    } else if (NT > 2 && rows <= 32) {
      product_loop<F, UP, NT, CACHED, 2>(L, acc, begin + wave / CW, KW, end, lane, Kd, N, plane);
    } else if (NT > 3 && rows <= 48) {
      product_loop<F, UP, NT, CACHED, 3>(L, acc, begin + wave / CW, KW, end, lane, Kd, N, plane);
    } else {
      product_loop<F, UP, NT, CACHED, NT>(L, acc, begin + wave / CW, KW, end, lane, Kd, N, plane);
    }
  }

  if constexpr (DIRECT) {   // a wave's sums are whole: from its registers to memory, 4 columns a lane
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (16 * nt + m >= rows) continue;
      const int64_t row = ids[nt];
      const int c0 = tile * COLS + wave % CW * WCOLS;
#pragma unroll
      for (int j = 0; j < (UP ? G / 2 : G); ++j) {
        if constexpr (UP) {
          const int c = c0 + 16 * j + 4 * q;
          if (c >= N) continue;
          float hv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) hv[i] = silu_f(acc[nt][2 * j][i]) * acc[nt][2 * j + 1][i];
          const int64_t place = row * Ih + mx_h_place(c);
          if constexpr (fmt_f32(F)) {
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.h) + place) = f32x4{hv[0], hv[1], hv[2], hv[3]};
          } else {
            u32x2 hi, lo;
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              hi[d] = pack_bf16x2(first_part(hv[2 * d]), first_part(hv[2 * d + 1]));
              lo[d] = pack_bf16x2(hv[2 * d] - __uint_as_float(hi[d] << 16), hv[2 * d + 1] - __uint_as_float(hi[d] & 0xFFFF0000u));
            }
            uint16_t* hp = static_cast<uint16_t*>(a.h) + place;
            *reinterpret_cast<u32x2*>(hp) = hi;
            *reinterpret_cast<u32x2*>(hp + RA * Ih) = lo;
          }
        } else if constexpr (fmt_mx(F)) {
          const int c = c0 + 16 * j + 4 * q;
          if (c < N) *reinterpret_cast<f32x4*>(a.y + ((int64_t)slice * RA + row) * N + c) = acc[nt][j];
        } else if (j % 4 == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + G * (4 * q + i) + j;
            if (c < N)
              *reinterpret_cast<f32x4*>(a.y + ((int64_t)slice * RA + row) * N + c) =
                  f32x4{acc[nt][j][i], acc[nt][j + 1][i], acc[nt][j + 2][i], acc[nt][j + 3][i]};
          }
        }
      }
    }
    return;
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
        const int64_t place = row * Ih + (fmt_mx(F) ? mx_h_place(tile * COLS + bc) : tile * COLS + bc);
        if constexpr (fmt_f32(F)) {
          static_cast<float*>(a.h)[place] = hv;
        } else {
          const uint32_t hi = f32_to_bf16(first_part(hv));
          uint16_t* hp = static_cast<uint16_t*>(a.h);
          hp[place] = (uint16_t)hi;
          hp[RA * Ih + place] = (uint16_t)f32_to_bf16(hv - bf16_to_f32(hi));
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
             *a.n_entries * slices - 1;
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

// The kernels that are built: what decode_plan can ask for.
constexpr bool kernel_built(int f, bool up, int nt, int cw, bool fused, bool many, bool cached) {
  if (many ? f == kFmtMxF32 || nt != (f == kFmtBf16 && !up ? 2 : 4) || !cached : nt > 2 || (cached && fmt_mx(f))) return false;
  if (fmt_mx(f) && (nt == 1) == (cw == 4)) return false;   // 1 and 2 column tiles; with rows by way of LDS, 4
  static_assert(8 * kMaxExperts <= kListPairs && kTailTokens <= 8);
  if (up) return fused || row_tile_of(f, nt) != 8;         // up to 8 tokens every block makes the list
  return !fused || (nt == 1 && !many);                     // the output's sum inside: up to kTailTokens
}

template <int F, bool UP, int NT, int CW, bool FUSED, bool MANY, bool CACHED>
hipError_t launch_kernel(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if constexpr (!kernel_built(F, UP, NT, CW, FUSED, MANY, CACHED)) {
    return hipErrorInvalidValue;
  } else {
    const int tiles = UP ? p.up_tiles : p.down_tiles, slices = UP ? 1 : p.slices;
    const int steps = UP ? (a.H + fmt_step(F) - 1) / fmt_step(F) : p.slice_steps;
    constexpr int halves = MANY ? kMaxRowTile / (16 * NT) : 1;
    const dim3 grid(halves > 1 ? (tiles + kXcds - 1) / kXcds * kXcds * halves : tiles, p.entries, slices);
    decode_ffn_kernel<F, UP, NT, CW, FUSED, MANY, CACHED><<<grid, kThreads, 0, st>>>(a, slices, steps);
    return hipGetLastError();
  }
}
template <int F, bool UP, int NT, int CW, bool FUSED>
hipError_t launch_kernel(const DecodeArgs& a, const DecodePlan& p, const DecodeKernel& k, hipStream_t st) {
  if (k.many) return launch_kernel<F, UP, NT, CW, FUSED, true, true>(a, p, st);
  return k.cached ? launch_kernel<F, UP, NT, CW, FUSED, false, true>(a, p, st)
                  : launch_kernel<F, UP, NT, CW, FUSED, false, false>(a, p, st);
}
template <int F, bool UP, int NT>
hipError_t launch_kernel(const DecodeArgs& a, const DecodePlan& p, const DecodeKernel& k, hipStream_t st) {
  switch (k.width) {
    case 1: return k.fused ? launch_kernel<F, UP, NT, 1, true>(a, p, k, st) : launch_kernel<F, UP, NT, 1, false>(a, p, k, st);
    case 2: return k.fused ? launch_kernel<F, UP, NT, 2, true>(a, p, k, st) : launch_kernel<F, UP, NT, 2, false>(a, p, k, st);
    case 4: return k.fused ? launch_kernel<F, UP, NT, 4, true>(a, p, k, st) : launch_kernel<F, UP, NT, 4, false>(a, p, k, st);
    default: return hipErrorInvalidValue;
  }
}
template <int F, bool UP>
hipError_t launch_product(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  const DecodeKernel& k = UP ? p.up : p.down;
  switch (k.row_tiles) {
    case 1: return launch_kernel<F, UP, 1>(a, p, k, st);
    case 2: return launch_kernel<F, UP, 2>(a, p, k, st);
    case 4: return launch_kernel<F, UP, 4>(a, p, k, st);
    default: return hipErrorInvalidValue;
  }
}

template <int F>
hipError_t launch_fmt(const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if (!p.up.fused || a.picked) {
    if (p.up.fused) decode_topk_kernel<<<(a.T + kWaves - 1) / kWaves, kThreads, 0, st>>>(a);
    else decode_route_kernel<<<1, kRouteThreads, 0, st>>>(a, p.row_tile, p.entries);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipError_t e = launch_product<F, true>(a, p, st);
  if (e == hipSuccess) e = launch_product<F, false>(a, p, st);
  if (p.down.fused || e != hipSuccess) return e;
  decode_combine_kernel<!fmt_f32(F)><<<dim3((a.H / 4 + 255) / 256, a.T), 256, 0, st>>>(a, p.slices);
  return hipGetLastError();
}

}  // namespace

// Column tiles a block's waves take side by side (1, 2 or 4).  Where a row of
// the matrix is long, pieces of it that are read at the same time and are far
// apart use few of the memory's channels, so the block reads as wide a piece as
// leaves kFillBlocks blocks (bf16 [4096, 14336] x 2, 32 tokens: 1, 2, 4 tiles
// 507, 465, 437 us a call; one token: 136, 123, 146).  Short rows want more
// blocks ([2048, 1408] x 2, 1 and 2 tiles: 16 tokens of 4 in 32 experts 95 and
// 102 us, of 6 in 64 experts 167 and 165, 32 tokens 203 and 194).  4-bit rows
// are long ones, and their waves work side by side on the same rows' values
// where those go through LDS.
static int tile_width(bool mx, int row_tile, int64_t row_bytes, int columns, int tile, double groups_and_slices) {
  if (mx && row_tile >= 32) return 4;
  const bool short_row = !mx && row_bytes < kLongRow;
  for (int w = !mx && row_bytes >= 2 * kLongRow ? 4 : 2; w > 1; w /= 2)
    if ((columns + w * tile - 1) / (w * tile) * groups_and_slices >= (short_row ? kManyBlocks : kFillBlocks)) return w;
  return 1;
}

// Weights are read past the caches (through them the calls take 5 to 12 % longer)
// unless others read the same lines: other entries of the expert (kManyRows), or
// the tiles to the left and right where rows do not begin on a line ([2816,
// 2840] x 8 in 26 experts, one token 110.6 us past, 105.8 through the caches;
// [584, 2632] x 8 in 100, 14 tokens 172 and 154; [2048, 1400] x 4 in 32, 2
// tokens 44.6 and 39.2).
static DecodeKernel decode_kernel(int f, bool up, int row_tile, int64_t row_bytes, int width, bool fused) {
  DecodeKernel k;
  k.many = row_tile == kMaxRowTile;
  k.row_tiles = k.many ? (f == kFmtBf16 && !up ? 2 : 4) : row_tile < 32 ? 1 : 2;
  k.width = width;
  k.fused = fused;
  k.cached = k.many || (!fmt_mx(f) && row_bytes % kLineBytes);
  return k;
}

DecodePlan decode_plan(bool is_bf16, bool mx, int T, int H, int E, int K, int I, int Ns) {
  const int f = mx ? (is_bf16 ? kFmtMxBf16 : kFmtMxF32) : (is_bf16 ? kFmtBf16 : kFmtF32);
  const int tile = 16 * fmt_groups(f), step = fmt_step(f), size = is_bf16 ? 2 : 4;
  DecodePlan p;
  p.row_tile = T <= row_tile_of(f, 1) ? row_tile_of(f, 1) : row_tile_of(f, 2);
  const int64_t R = (int64_t)T * K;
  const bool head = R <= kListPairs, tail = T <= kTailTokens;
  p.picked = T > kHeadTokens || R > kThreads;
  // experts with rows as expected of even routing, and the shared ones
  double miss = 1.0;
  for (int t = 0; t < T; ++t) miss *= 1.0 - (double)K / E;
  const double groups = E * (1.0 - miss) + Ns;
  if (f != kFmtMxF32 && T > p.row_tile && R >= (int64_t)kManyRows * E) {
    const double entries = R / (double)kMaxRowTile > groups ? R / (double)kMaxRowTile : groups;
    if (!mx || I / (kWaves * tile / 2) * entries >= kFillBlocks) p.row_tile = kMaxRowTile;
  }
  const int busy = (int)(R < E ? R : E);   // experts with rows, at most
  // an expert with c rows has at most 1 + (c - 1) / row_tile entries
  p.entries = busy + (int)((R - busy) / p.row_tile) + Ns * ((T + p.row_tile - 1) / p.row_tile);
  const int64_t up_bytes = (int64_t)I * size, down_bytes = (int64_t)H * size;
  const int up_width = tile_width(mx, p.row_tile, up_bytes, I, tile / 2, groups);
  p.up_tiles = (I + up_width * tile / 2 - 1) / (up_width * tile / 2);
  p.up = decode_kernel(f, true, p.row_tile, up_bytes, up_width, head);
  const int steps = (I + step - 1) / step, most = steps < kMaxSlices ? steps : kMaxSlices;
  const int down_width = tile_width(mx, p.row_tile, down_bytes, H, tile, groups * (most < 2 ? most : 2));
  p.down_tiles = (H + down_width * tile - 1) / (down_width * tile);
  p.down = decode_kernel(f, false, p.row_tile, down_bytes, down_width, tail);
  int s = (int)(kSliceBlocks / (p.down_tiles * groups) + 0.999);
  s = s < 1 ? 1 : s > most ? most : s;
  p.slice_steps = (steps + s - 1) / s;
  p.slices = (steps + p.slice_steps - 1) / p.slice_steps;
  return p;
}

hipError_t launch_decode(bool is_bf16, bool mx, const DecodeArgs& a, const DecodePlan& p, hipStream_t st) {
  if (mx) return is_bf16 ? launch_fmt<kFmtMxBf16>(a, p, st) : launch_fmt<kFmtMxF32>(a, p, st);
  return is_bf16 ? launch_fmt<kFmtBf16>(a, p, st) : launch_fmt<kFmtF32>(a, p, st);
}

}  // namespace moe
