// The router's losses: what the C entry points hand to the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernels.hpp"

namespace moe {

constexpr int kBalanceShort = 64;      // sequences up to this long take one wave each
constexpr int kBalanceThreads = 512;   // of a chunk's block
constexpr int kBalanceChunk = 512;     // tokens of a chunk: 64 for each wave
constexpr int kBalanceJoin = 1024;     // threads of the joining blocks

struct BalanceArgs {
  int T, E, K, seq_len, S;
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

struct BalanceBwdArgs {
  int T, E, K, seq_len, S;
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
