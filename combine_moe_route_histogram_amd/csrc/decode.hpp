// Host-side launchers of the layer for a few tokens (decode.hip) and of the
// 4-bit weight format (mx.hip); internal, the public ABI is moe.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Tokens a decode call takes at most (one routing block holds them all).
constexpr int kDecodeMaxTokens = 256;
// Words from one column tile's counter to the next: increments of one 64-byte
// line follow each other every 13 ns, whichever counter they mean (512 of
// them: 6.6 us).
constexpr int kDoneStride = 64;
// Largest H and I of the decode calls (lane offsets into a matrix's rows are
// formed in 32 bits inside a k step).
constexpr int kDecodeMaxDim = 1 << 20;

// Weights along the reduction dim that share one scale, and the bytes of
// their codes.
constexpr int kMxGroup = 32;
constexpr int kMxCodeBytes = 16;

// Which of the built kernels one of the two products runs.
struct DecodeKernel {
  int row_tiles;  // 16-row operands of a block (1, 2 or 4)
  int width;      // column tiles its waves span (1, 2 or 4)
  bool fused;     // gate/up: its blocks list the work for themselves; down: its last ones add up the output
  bool many;      // entries of 64 rows
  bool cached;    // weights through the caches
};

// How a call is cut.
struct DecodePlan {
  DecodeKernel up, down;   // gate/up and down projection
  bool picked;      // with up.fused: the top-k has a launch of its own
  int row_tile;     // rows of one entry at most (8, 16, 32 or 64)
  int entries;      // bound on the number of entries (expert x row tile)
  int up_tiles;     // blocks' column tiles of the gate/up projection
  int down_tiles;   // column tiles of the down projection
  int slices;       // k slices of the down projection
  int slice_steps;  // k steps in each
};
DecodePlan decode_plan(bool is_bf16, bool mx, int T, int H, int E, int K, int I, int Ns);

struct DecodeArgs {
  int T, H, E, K, I, Ns, R;
  const float* logits;
  const void* x;
  const void* w1;
  const void* w3;
  const void* w2;
  const void* ws1;
  const void* ws3;
  const void* ws2;
  const int32_t* n_tokens;  // null: T
  int32_t* topk_idx;
  float* topk_w;
  void* out;
  // workspace
  int2* entries;       // {group, rows}
  int32_t* n_entries;
  int32_t* lists;      // [entries, row_tile] row ids
  int32_t* done;       // [n_done], kDoneStride apart: blocks of a column tile that have stored their sums
  int n_done;          // 0: the sum has a launch of its own
  void* h;             // [RA, I] (4 bit: rows of whole 128s): f32, or two bf16 planes (value, what it left)
  float* y;            // [slices, RA, H]
  int picked;          // topk_idx and topk_w are written before the first product
};
hipError_t launch_decode(bool is_bf16, bool mx, const DecodeArgs& a, const DecodePlan& p, hipStream_t st);

hipError_t launch_mx_quantize(bool is_bf16, int64_t G, int K, int N, const void* w, void* mx, hipStream_t st);
hipError_t launch_mx_dequantize(bool is_bf16, int64_t G, int K, int N, const void* mx, void* w, hipStream_t st);

}  // namespace moe
