// The router's losses: what the C entry points hand to the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernels.hpp"

namespace moe {

constexpr int kBalanceFew = 8;         // sequences up to this long take a lane group each
constexpr int kBalanceShort = 64;      // sequences up to this long take one wave each
// A wave each, too, up to this long where there are so many of them (131072 tokens, 32 experts, in sequences
// of 70: 12.8 us by waves, 25.9 by blocks; of 100: 14.4 and 20.5; of 128: 16.5 and 15.7).
constexpr int kBalanceShortMany = 112, kBalanceMany = 1024;
enum BalanceBy { kByGroup, kByWave, kByChunk };
constexpr int kBalanceShortBlocks = 2048;   // at most, of four waves
constexpr int kBalanceThreads = 512;   // of a chunk's block
constexpr int kBalanceChunk = 512;     // most tokens of a chunk: 64 for each wave
constexpr int kBwdRows = 2;            // rows of a lane group in flight in the gradient's pass
constexpr int kBalanceJoin = 1024;     // threads of the joining blocks

// Lanes of a row: the power of two that holds E / 4 (E <= kMaxExperts).
inline int balance_lanes(int E) {
  int g = 1;
  while (4 * g < E) g *= 2;
  return g;
}

struct BalanceArgs {
  int T, E, K, seq_len, S;
  int by;     // BalanceBy
  int chunk;  // tokens of a chunk
  int cps;    // chunks of a sequence
  int eb;     // joining blocks of a sequence
  int entries;   // that the last step takes the mean of: sequences, or the short ones' blocks
  const float* logits;
  const int32_t* topk_idx;
  const uint8_t* mask;
  int32_t *counts, *tokens;
  float *probs, *loss;
  // workspace
  float *part_p, *part_z, *seq_loss, *seq_z;
  int32_t *part_c, *part_n, *ticket, *seq_n, *seq_some;
};

// n / d for n below 2^31 by a multiplication: with 2^(l-1) < d <= 2^l and m = ceil(2^(31+l) / d) < 2^32,
// n m / 2^(31+l) exceeds n / d by less than 1 / d.
struct DivBy {
  uint32_t m = 0;
  int shift = -1;   // -1: d = 1
  DivBy() = default;
  explicit DivBy(uint32_t d) {
    int l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    shift = l - 1;
    if (l) m = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
  }
  __host__ __device__ uint32_t of(uint32_t n) const {
    return shift < 0 ? n : (uint32_t)(((uint64_t)n * m) >> 32) >> shift;
  }
};

struct BalanceBwdArgs {
  int T, E, K, S;
  DivBy seq;        // by seq_len
  const float* logits;
  const uint8_t* mask;
  const int32_t *counts, *tokens;
  const float *dloss, *dtopk_w, *topk_w;
  const int32_t* topk_idx;
  float* dlogits;
};

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st);
hipError_t launch_balance_bwd(const BalanceBwdArgs& a, hipStream_t st);

}  // namespace moe
