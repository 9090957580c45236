// Newton-Schulz products of stacked matrices and the update of weights built
// on them: sizes, workspace and arguments (shared by the C entry points and the
// kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kNewtonMaxDim = 1 << 20;
constexpr int kNewtonMaxStack = 1 << 30;   // a matrix's number plus those worked on at a time stay in 31 bits
constexpr int64_t kNewtonMaxMatrix = (int64_t)1 << 32;   // elements: keeps tile and block counts in 31 bits
constexpr int kNewtonPad = 64;       // of both sides of a stored matrix: whole k slices, zero-filled
// Fewer rows (or columns) than this take factors of two parts whatever the type: their roundings do
// not average out (up to 4e-3 of the norm), and the call's time is that of its launches.
constexpr int kNewtonFewRows = 32;
// Matrices of few rows worked on at a time: 63 MB of sums and polynomials for 48 rows, 109 MB for 64.  The workspace also
// holds what the chain of products would take for them (2.2 GB for 2048 [64, 2048]), as its size is asked for without
// the coefficients, which decide between the two.
constexpr int kNewtonFewBatch = 2048;
constexpr int kNormParts = 256;      // partial sums of a matrix's squares

// Sizes of one call.  A matrix is worked on as X [s, l] with s <= l (the
// transpose of a tall one), padded with zeros to [sp, lp].
struct NewtonPlan {
  int G, R, C;
  bool tall;           // R > C
  int s, l, sp, lp;
  bool exact;          // factors of two fp16 parts (22 bits)
  bool small;          // small tiles for X, which is kept with its transpose
  bool few;            // few rows: the iteration on [s, s] where its coefficients allow that
  int few_batch;       // matrices at a time, then
  int chunk, chunks;   // and in the first pass: columns of a block, blocks of a matrix
  int batch;           // matrices worked on at a time
  // workspace sections (byte offsets)
  size_t parts, xh[2], xl[2], th[2], tl[2], ah, al, bh, bl, total;
};
NewtonPlan newton_plan(int G, int R, int C, bool exact);

struct NewtonCall {
  NewtonPlan p;
  void* ws;
  int steps;
  const float (*coef)[3];
  bool bf16;
  const float* g;        // gradient, or the matrices themselves
  void* out;             // moe_orthogonalize (NULL: the update)
  // the update
  float *mom, *master;
  uint16_t* w;
  const float* lr_dev;
  float lr, momentum, weight_decay, scale;
  bool nesterov;
};
hipError_t launch_newton(const NewtonCall& c, hipStream_t st);

}  // namespace moe
