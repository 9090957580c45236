// MXFP4 weight matrices: [G, K, N] bf16 or f32 <-> packed 4-bit codes.
//
// A group is 32 weights of one column, consecutive along the reduction dim K.
// Its scale is 2^s with s = floor(log2 max|w|) - 2, which puts the largest
// magnitude into [4, 8) of the code grid {0, .5, 1, 1.5, 2, 3, 4, 6}; a code is
// the nearest grid value of w / 2^s, ties to the even code, magnitudes above 6
// to 6 (OCP Microscaling, MXFP4).  Division by 2^s is exact, so the only
// rounding is the code's own; gfx950 has it as one instruction per two
// weights, in both directions.  The instruction takes the exponent field of
// its scale operand, so byte << 23 is every scale byte of the format: field 0
// is 2^-127 and not the float 0, field 255 makes NaN.
//
// Bound: bytes.  A thread owns 4 columns of one group: it reads 32 rows of 8
// or 16 bytes (a wave reads 512 or 1024 contiguous bytes of each row) and
// writes 4 x 16 bytes of codes, contiguous with its neighbours'.  Measured:
// bf16 [64, 2048, 1408] (467 MB in all) 87 us either way, 5.4 TB/s; bf16
// [8, 4096, 14336] back 230 us, 5.2 TB/s (a large copy: 4.9).
#include "common.hpp"
#include "decode.hpp"

namespace moe {

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

constexpr int kMxCols = 4;   // columns a thread owns (N is a multiple of 8)

template <typename S> __device__ __forceinline__ void load4(const S* p, float* f);
template <> __device__ __forceinline__ void load4<uint16_t>(const uint16_t* p, float* f) {
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
  f[0] = __uint_as_float(v[0] << 16); f[1] = __uint_as_float(v[0] & 0xFFFF0000u);
  f[2] = __uint_as_float(v[1] << 16); f[3] = __uint_as_float(v[1] & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void load4<float>(const float* p, float* f) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int c = 0; c < 4; ++c) f[c] = __uint_as_float(v[c]);
}

// Unit u of the G * K/32 * N/4 units: column block u % (N/4) of the group row u / (N/4).
template <typename S>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const S* __restrict__ w, int64_t units,
                                                          int N, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int nb = N / kMxCols;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int64_t row = u / nb;   // g * (K/32) + group
  const int col = (int)(u - row * nb) * kMxCols;
  const S* src = w + row * kMxGroup * N + col;
  float v[kMxGroup][kMxCols];
#pragma unroll
  for (int i = 0; i < kMxGroup; ++i) load4<S>(src + (int64_t)i * N, v[i]);
  uint32_t bytes = 0;
#pragma unroll
  for (int c = 0; c < kMxCols; ++c) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < kMxGroup; ++i) big = fmaxf(big, fabsf(v[i][c]));
    // exponent field of the largest magnitude, less the exponent of the
    // largest code; at least 1, so that 2^(b-127) is a normal float
    const int b = max(1, (int)(__float_as_uint(big) >> 23) - 2);
    const float s = __uint_as_float((uint32_t)b << 23);
    u32x4 q;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t r = 0;
      const int i = 8 * d;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[i][c], v[i + 1][c], s, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[i + 2][c], v[i + 3][c], s, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[i + 4][c], v[i + 5][c], s, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[i + 6][c], v[i + 7][c], s, 3);
      q[d] = r;
    }
    st16(codes + (row * N + col + c) * kMxCodeBytes, q);
    bytes |= (uint32_t)b << (8 * c);
  }
  *reinterpret_cast<uint32_t*>(scales + row * N + col) = bytes;
}

template <typename S> __device__ __forceinline__ void store4(S* p, const float* f);
template <> __device__ __forceinline__ void store4<uint16_t>(uint16_t* p, const float* f) {
  u32x2 v;
  v[0] = pack_bf16x2(f[0], f[1]);
  v[1] = pack_bf16x2(f[2], f[3]);
  *reinterpret_cast<u32x2*>(p) = v;
}
template <> __device__ __forceinline__ void store4<float>(float* p, const float* f) {
  u32x4 v;
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = __float_as_uint(f[c]);
  st16(p, v);
}

template <int B>
__device__ __forceinline__ void mx_pair(uint32_t word, float s, float& lo, float& hi) {
  const float __attribute__((ext_vector_type(2))) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, B);
  lo = p[0];
  hi = p[1];
}

template <typename S>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t units, int N, S* __restrict__ w) {
  const int nb = N / kMxCols;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int64_t row = u / nb;
  const int col = (int)(u - row * nb) * kMxCols;
  u32x4 q[kMxCols];
#pragma unroll
  for (int c = 0; c < kMxCols; ++c) q[c] = ld16(codes + (row * N + col + c) * kMxCodeBytes);
  const uint32_t bytes = *reinterpret_cast<const uint32_t*>(scales + row * N + col);
  S* dst = w + row * kMxGroup * N + col;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    float v[8][kMxCols];
#pragma unroll
    for (int c = 0; c < kMxCols; ++c) {
      const float s = __uint_as_float(((bytes >> (8 * c)) & 0xFFu) << 23);
      mx_pair<0>(q[c][d], s, v[0][c], v[1][c]);
      mx_pair<1>(q[c][d], s, v[2][c], v[3][c]);
      mx_pair<2>(q[c][d], s, v[4][c], v[5][c]);
      mx_pair<3>(q[c][d], s, v[6][c], v[7][c]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) store4<S>(dst + (int64_t)(8 * d + i) * N, v[i]);
  }
}

hipError_t launch_mx_quantize(bool is_bf16, int64_t G, int K, int N, const void* w, void* mx,
                              hipStream_t st) {
  const int64_t rows = G * (K / kMxGroup), units = rows * (N / kMxCols);
  uint8_t* codes = static_cast<uint8_t*>(mx);
  uint8_t* scales = codes + rows * N * kMxCodeBytes;
  const dim3 grid((unsigned)((units + 255) / 256));
  if (is_bf16)
    mx_quantize_kernel<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(w), units, N, codes, scales);
  else
    mx_quantize_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(w), units, N, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(bool is_bf16, int64_t G, int K, int N, const void* mx, void* w,
                                hipStream_t st) {
  const int64_t rows = G * (K / kMxGroup), units = rows * (N / kMxCols);
  const uint8_t* codes = static_cast<const uint8_t*>(mx);
  const uint8_t* scales = codes + rows * N * kMxCodeBytes;
  const dim3 grid((unsigned)((units + 255) / 256));
  if (is_bf16)
    mx_dequantize_kernel<uint16_t><<<grid, 256, 0, st>>>(codes, scales, units, N, static_cast<uint16_t*>(w));
  else
    mx_dequantize_kernel<float><<<grid, 256, 0, st>>>(codes, scales, units, N, static_cast<float*>(w));
  return hipGetLastError();
}

}  // namespace moe
