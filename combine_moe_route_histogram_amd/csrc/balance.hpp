// The router's losses: what the C entry points hand to the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernels.hpp"

namespace moe {

constexpr int kBalanceShort = 64;      // sequences up to this long take one wave each
constexpr int kBalanceThreads = 512;   // of a chunk's block
constexpr int kBalanceChunk = 512;     // most tokens of a chunk: 64 for each wave
constexpr int kBwdRows = 2;            // rows of a lane group in flight in the gradient's pass
constexpr int kBalanceJoin = 1024;     // threads of the joining blocks

struct BalanceArgs {
  int T, E, K, seq_len, S;
  int chunk;  // tokens of a chunk
  int cps;    // chunks of a sequence
  int eb;     // joining blocks of a sequence
  const float* logits;
  const int32_t* topk_idx;
  const uint8_t* mask;
  int32_t *counts, *tokens;
  float *probs, *loss;
  // workspace
  float *part_p, *part_z, *seq_loss, *seq_z;
  int32_t *part_c, *part_n, *ticket;
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
