// Newton-Schulz products of stacked matrices, and the update of weights built on them.
//
// Per step, for X [s, l] with s <= l (the transpose of a tall matrix, taken while it is read):
//   A = X X^T           symmetric: tiles on and above the diagonal, mirrored
//   B = b A + c A A     symmetric, too
//   X <- a X + B X      the last one writes the result (transposed back) or updates the weights
// so 3 s^2 l + s^3 multiply-adds a step of 4 s^2 l + 2 s^3: bound by the matrix cores where the
// matrices are large, by the chain of launches where they are small.
//
// Numbers.  X is kept in fp16, scaled by 2^10 (|x| <= 64 fits, an element of 1e-5 still has all
// its bits), at first as two parts hi + lo (22 bits).  The products take the upper parts (11 bits)
// with f32 sums, a is part of B's diagonal, and what that leaves of X, a times the lower part, is
// added in f32.  The roundings of a product then act on X
// from the left only, inside its row space, while a rounding of X itself has null directions, which
// every later step makes |a| times larger.  So X drops its lower part when what the steps left
// can make of it is small (kDropLow).  That is 1e-3 (full rank) to 4e-3 (rank 1) of the result's norm with the
// default steps, and with others what they make of changes of 2^-12 (no lower parts at all: 2e-2 for rank 64 of 352,
// 7e-2 for rank 4; everything in bf16: 1e-2 for a full rank and 0.2, 0.6 for those), with 40 % fewer bytes for X than two parts all the way.
// The exact form takes three products, lo hi + hi lo + hi hi, of X, A and a I + B in two parts each.
//
// Matrices of few rows (or columns) have a form of their own, on [s, s] in 64 bits: see newton_few_gram_kernel.
#include "muon.hpp"

#include "gemm_tile.hpp"

namespace moe {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kXScale = 1024.f;   // of stored X
constexpr float kAScale = 256.f;    // of stored A and B (of the last step's B: see last_scale)

// kAdd: kStep that adds a times the lower part of X
enum NewtonKind { kGram, kPoly, kStep, kAdd, kOut, kUpdate };

// One product of a batch of matrices.  Operands and results are [batch][rows][ld] fp16 planes.
struct Product {
  const uint16_t *ah, *al, *bh, *bl;
  int64_t a_mat, b_mat;     // elements of a matrix
  int lda, ldb, k_len;
  int m_len, n_len;         // padded sizes of the result
  int mt, nt, per, tiles;   // tile grid, tiles of a matrix and of all
  const uint16_t *ch, *cl;  // what the epilogue adds: A (kPoly), the lower part of X (kAdd: ch)
  uint16_t *oh, *ol;        // kGram, kPoly, kStep, kAdd; ol NULL: upper parts only
  uint16_t *th, *tl;        // small tiles, kStep and kAdd: the result's transpose
  int64_t o_mat;
  int ldo, ldt;             // of ch, cl, oh, ol; of th, tl
  float a, b, c;
  // kOut, kUpdate
  float undo;               // of the scales of B and X
  bool tall, bf16;
  int R, C, g0;
  void* out;
  float* master;
  uint16_t* w;
  const float* lr_dev;
  float lr, weight_decay, scale;
};

template <int BM_, int BN_, int WGM_, int WGN_, int BK_, int STAGES_, bool B_MN_>
struct NsCfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, BK = BK_, STAGES = STAGES_;
  static constexpr bool B_MN = B_MN_;
  static constexpr int NW = WGM * WGN, NT = NW * kWave;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MI = WM / 32, NJ = WN / 32;
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
  static_assert(NJ % 2 == 0, "the epilogue takes two 32-column blocks at a time");
};

// Four or eight values as two fp16 parts.
__device__ __forceinline__ void split16(const float* v, u32x2& hi, u32x2& lo) {
  f16x4 h, l;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = (_Float16)v[e];
    l[e] = (_Float16)(v[e] - (float)h[e]);
  }
  hi = __builtin_bit_cast(u32x2, h);
  lo = __builtin_bit_cast(u32x2, l);
}
__device__ __forceinline__ void join16(const u32x2& hi, const u32x2* lo, float* v) {
  const f16x4 h = __builtin_bit_cast(f16x4, hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)h[e];
  if (lo) {
    const f16x4 l = __builtin_bit_cast(f16x4, *lo);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (float)l[e];
  }
}

__device__ __forceinline__ void split16(const float* v, u32x4& hi, u32x4& lo) {
  u32x2 h0, h1, l0, l1;
  split16(v, h0, l0);
  split16(v + 4, h1, l1);
  hi = u32x4{h0[0], h0[1], h1[0], h1[1]};
  lo = u32x4{l0[0], l0[1], l1[0], l1[1]};
}
__device__ __forceinline__ void join16(const u32x4& hi, const u32x4* lo, float* v) {
  const u32x2 h0 = {hi[0], hi[1]}, h1 = {hi[2], hi[3]};
  u32x2 l0, l1;
  if (lo) {
    l0 = u32x2{(*lo)[0], (*lo)[1]};
    l1 = u32x2{(*lo)[2], (*lo)[3]};
  }
  join16(h0, lo ? &l0 : nullptr, v);
  join16(h1, lo ? &l1 : nullptr, v + 4);
}

// master <- keep master - gain O, and its bf16 copy.
struct UpdateScale { float keep, gain; };
__device__ __forceinline__ void update4(const Product& p, const UpdateScale& u, int64_t at, const f32x4& m, const float* v) {
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = u.keep * m[e] - u.gain * v[e];
  *reinterpret_cast<f32x4*>(p.master + at) = f32x4{x[0], x[1], x[2], x[3]};
  if (p.w) st_bf16x4(p.w + at, x);
}

// Four results of row `row` from column `col` on, of matrix g of the user's tensors.  m: the four
// elements of master, if they were loaded ahead.
template <int KIND>
__device__ __forceinline__ void emit4(const Product& p, int64_t g, int row, int col, const float* v,
                                      const UpdateScale& u, const f32x4* m = nullptr) {
  if (row >= p.R || col >= p.C) return;
  const int64_t at = (g * p.R + row) * p.C + col;
  if (p.C % 4 == 0) {   // aligned: 16-byte f32, 8-byte bf16
    if constexpr (KIND == kOut) {
      if (p.bf16) st_bf16x4(static_cast<uint16_t*>(p.out) + at, v);
      else *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      update4(p, u, at, m ? *m : *reinterpret_cast<const f32x4*>(p.master + at), v);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (col + e >= p.C) break;
    if constexpr (KIND == kOut) {
      if (p.bf16) static_cast<uint16_t*>(p.out)[at + e] = (uint16_t)f32_to_bf16(v[e]);
      else static_cast<float*>(p.out)[at + e] = v[e];
    } else {
      const float x = u.keep * p.master[at + e] - u.gain * v[e];
      p.master[at + e] = x;
      if (p.w) p.w[at + e] = (uint16_t)f32_to_bf16(x);
    }
  }
}
__device__ __forceinline__ UpdateScale update_scale(const Product& p) {
  const float lr = p.lr_dev ? *p.lr_dev : p.lr;
  return {1.f - lr * p.weight_decay, lr * p.scale};
}

// Result of four elements of row m from column n on: their sums s and the values x that are added.
template <int KIND>
__device__ __forceinline__ void finish4(const Product& p, int m, int n, const float* s, const float* x, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (KIND == kGram) v[e] = s[e] * (kAScale / (kXScale * kXScale));
    else if constexpr (KIND == kPoly)
      v[e] = p.b * x[e] + p.c * (s[e] * (1.f / kAScale)) + (m == n + e ? p.a * kAScale : 0.f);
    else if constexpr (KIND == kAdd) v[e] = p.a * x[e] + s[e] * (1.f / kAScale);
    else if constexpr (KIND == kStep) v[e] = s[e] * (1.f / kAScale);
    else v[e] = s[e] * p.undo;
  }
}

// The transpose of a 32 x 64 block of fp16 that lies in LDS (rows of kTurnPitch bytes), to 64 rows of 32
// at dst.  The LDS transpose read hands a lane 4 consecutive rows of one column; with row groups 8 g and 8 g + 4
// for the lanes of group g, 4 lanes store 64 bytes of a row.
constexpr int kTurnPitch = 144;
__device__ __forceinline__ void store_turned(const uint8_t* block, uint16_t* dst, int64_t ld, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const uint8_t* const at = block + (8 * g + (i >> 2)) * kTurnPitch + 8 * (i & 3);
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) {
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(at + 32 * cb));
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(at + 4 * kTurnPitch + 32 * cb));
    const i16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    *reinterpret_cast<u32x4*>(dst + (int64_t)(16 * cb + i) * ld + 8 * g) = __builtin_bit_cast(u32x4, v);
  }
}

// Accumulators to results: 32 x 64 blocks through the wave's LDS region, 8 columns of a row for each
// lane.  What is added is loaded one block ahead (unconditional loads, clamped into the matrix: a branch
// for each would make the waits conservative).  All LDS accesses are of words: a block of fp16 is
// written over floats that were read before it.
template <int KIND, bool EXACT, class C>
__device__ __forceinline__ void newton_epilogue(const Product& p, int64_t g, int m0, int n0, bool mirror,
                                                const f32x16 (&acc)[C::MI][C::NJ],
                                                uint8_t* const (&stages)[4], int wm, int wn, int wave,
                                                int lane) {
  constexpr int kRps = C::STAGE_BYTES / kEpiRegionBytes;
  static_assert(kRps >= 1 && (C::NW + kRps - 1) / kRps <= C::STAGES, "epilogue regions fit in the slices");
  constexpr int kBlocks = C::MI * (C::NJ / 2);
  constexpr bool kSym = KIND == kGram || KIND == kPoly, kLast = KIND == kOut || KIND == kUpdate;
  constexpr bool kAux = KIND == kPoly || KIND == kAdd, kAuxLow = KIND == kPoly && EXACT;
  const int rs = wave / kRps;
  uint8_t* const rbase = rs == 0 ? stages[0] : rs == 1 ? stages[1] : rs == 2 ? stages[2] : stages[3];
  uint8_t* const region = rbase + (wave - rs * kRps) * kEpiRegionBytes;
  uint32_t* const reg = reinterpret_cast<uint32_t*>(region);
  UpdateScale scale = {};
  if constexpr (KIND == kUpdate) scale = update_scale(p);
  const int64_t obase = g * p.o_mat;
  const bool turn = kSym ? mirror : kLast && p.tall;
  const int q0 = lane >> 3, c8 = 8 * (lane & 7);
  u32x4 aux_h[2][kAux ? 4 : 1], aux_l[2][kAuxLow ? 4 : 1];
  auto load_aux = [&](int blk, int buf) {
    const int mb = m0 + wm * C::WM + 32 * (blk / (C::NJ / 2)), nb = n0 + wn * C::WN + 64 * (blk % (C::NJ / 2));
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int m = min(mb, p.m_len - 32) + pass * 8 + q0, n = min(nb, p.n_len - 64) + c8;
      const int64_t at = obase + (int64_t)m * p.ldo + n;
      aux_h[buf][pass] = ld16(p.ch + at);
      if constexpr (kAuxLow) aux_l[buf][pass] = ld16(p.cl + at);
    }
  };
  // master, likewise (a load behind the stores of the block before would wait for them): rows as they are
  // stored below, clamped into the matrix
  f32x4 mst[2][KIND == kUpdate ? 8 : 1];
  const bool ahead = KIND == kUpdate && p.C % 4 == 0;
  auto load_master = [&](int blk, int buf) {
    const int mb = m0 + wm * C::WM + 32 * (blk / (C::NJ / 2)), nb = n0 + wn * C::WN + 64 * (blk % (C::NJ / 2));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = turn ? nb + j * 8 + (lane >> 3) : mb + (j >> 1) * 8 + q0;
      const int col = turn ? mb + 4 * (lane & 7) : nb + c8 + 4 * (j & 1);
      const int64_t at = ((p.g0 + g) * p.R + min(row, p.R - 1)) * p.C + min(col, p.C - 4);
      mst[buf][j] = *reinterpret_cast<const f32x4*>(p.master + at);
    }
  };
  if constexpr (kAux) load_aux(0, 0);
  if constexpr (KIND == kUpdate) {
    if (ahead) load_master(0, 0);
  }
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
#pragma unroll
    for (int hc = 0; hc < C::NJ / 2; ++hc) {
      const int blk = i * (C::NJ / 2) + hc;
      if constexpr (kAux) {
        if (blk + 1 < kBlocks) load_aux(blk + 1, (blk + 1) & 1);
      }
      if constexpr (KIND == kUpdate) {
        if (ahead && blk + 1 < kBlocks) load_master(blk + 1, (blk + 1) & 1);
      }
      const int mb = m0 + wm * C::WM + 32 * i, nb = n0 + wn * C::WN + 64 * hc;
      if (mb >= p.m_len || nb >= p.n_len) continue;   // the sizes are whole blocks
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        reg[row * kEpiPitch + (lane & 31)] = __float_as_uint(acc[i][2 * hc][r]);
        reg[row * kEpiPitch + 32 + (lane & 31)] = __float_as_uint(acc[i][2 * hc + 1][r]);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the wave's own region is written
      // a block of bf16 results inside the matrix, rows of whole 16 bytes
      const bool turn16 = KIND == kOut && p.bf16 && p.C % 8 == 0 && mb + 32 <= p.C && nb + 64 <= p.R;
      u32x4 low[kSym && EXACT ? 4 : 1];
#pragma unroll
      for (int pass = 0; pass < 4; ++pass) {
        const int q = pass * 8 + q0, m = mb + q, n = nb + c8;
        float s[8], v[8], x[8];
        Elem<float>::unpack(*reinterpret_cast<const u32x4*>(reg + q * kEpiPitch + c8), s);
        Elem<float>::unpack(*reinterpret_cast<const u32x4*>(reg + q * kEpiPitch + c8 + 4), s + 4);
        if constexpr (kAux) join16(aux_h[blk & 1][pass], kAuxLow ? &aux_l[blk & 1][pass] : nullptr, x);
        finish4<KIND>(p, m, n, s, x, v);
        finish4<KIND>(p, m, n + 4, s + 4, x + 4, v + 4);
        if constexpr (!kLast) {
          const int64_t at = obase + (int64_t)m * p.ldo + n;
          u32x4 hi, lo;
          split16(v, hi, lo);
          st16(p.oh + at, hi);
          if (EXACT || (!kSym && p.ol)) st16(p.ol + at, lo);
          if constexpr (kSym) {
            if (turn) *reinterpret_cast<u32x4*>(region + q * kTurnPitch + 2 * c8) = hi;
            if constexpr (EXACT) low[pass] = lo;
          }
        } else if (!turn) {
          constexpr bool kUp = KIND == kUpdate;
          emit4<KIND>(p, p.g0 + g, m, n, v, scale, kUp ? &mst[blk & 1][2 * pass] : nullptr);
          emit4<KIND>(p, p.g0 + g, m, n + 4, v + 4, scale, kUp ? &mst[blk & 1][2 * pass + 1] : nullptr);
        } else if (KIND == kOut && turn16) {
          *reinterpret_cast<u32x4*>(region + q * kTurnPitch + 2 * c8) = Elem<uint16_t>::pack(v);
        } else {
          *reinterpret_cast<u32x4*>(reg + q * kEpiPitch + c8) = Elem<float>::pack(v);
          *reinterpret_cast<u32x4*>(reg + q * kEpiPitch + c8 + 4) = Elem<float>::pack(v + 4);
        }
      }
      if ((kSym || kLast) && turn) {   // the block's transpose: 64 rows of 32
        __builtin_amdgcn_s_waitcnt(0xC07F);
        if constexpr (kSym) {
          const int64_t at = obase + (int64_t)nb * p.ldo + mb;
          store_turned(region, p.oh + at, p.ldo, lane);
          if constexpr (EXACT) {
            __builtin_amdgcn_s_waitcnt(0xC07F);
#pragma unroll
            for (int pass = 0; pass < 4; ++pass)
              *reinterpret_cast<u32x4*>(region + (pass * 8 + q0) * kTurnPitch + 2 * c8) = low[pass];
            __builtin_amdgcn_s_waitcnt(0xC07F);
            store_turned(region, p.ol + at, p.ldo, lane);
          }
        } else if (KIND == kOut && turn16) {
          store_turned(region, static_cast<uint16_t*>(p.out) + ((p.g0 + g) * p.R + nb) * p.C + mb, p.C, lane);
        } else if constexpr (kLast) {
#pragma unroll
          for (int pass = 0; pass < 8; ++pass) {
            const int n = pass * 8 + (lane >> 3), m4 = 4 * (lane & 7);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(reg[(m4 + e) * kEpiPitch + n]);
            emit4<KIND>(p, p.g0 + g, nb + n, mb + m4, v, scale, KIND == kUpdate ? &mst[blk & 1][pass] : nullptr);
          }
        }
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);   // region reads done before it is rewritten
    }
  }
}

// Tile r of the upper triangle (tm <= tn), column by column.
__device__ __forceinline__ void triangle(int r, int& tm, int& tn) {
  tn = (int)((sqrtf(8.f * (float)r + 1.f) - 1.f) * 0.5f);
  while (tn * (tn + 1) / 2 > r) --tn;
  while ((tn + 1) * (tn + 2) / 2 <= r) ++tn;
  tm = r - tn * (tn + 1) / 2;
}

// Tile of this block.  Consecutive blocks go to different XCDs; each XCD takes a run of tiles, which
// share operands in its L2.  (The edge tiles of all matrices at the end of the run, to even out its last
// round, read their operands anew: 64 [2048, 1408] matrices 6.5 -> 6.8 ms.  The last round in half tiles: no
// change, the clock rises as CUs fall idle.)
template <bool kSym>
__device__ __forceinline__ bool tile_of(const Product& p, int64_t& g, int& tm, int& tn) {
  const int xcd = blockIdx.x % kXcds, first = (int)((int64_t)p.tiles * xcd / kXcds);
  const int L = first + blockIdx.x / kXcds;
  if (L >= (int)((int64_t)p.tiles * (xcd + 1) / kXcds)) return false;
  g = L / p.per;
  const int r = L - (int)g * p.per;
  if constexpr (kSym) triangle(r, tm, tn);
  else band_order(r, p.mt, p.nt, 8, tm, tn);
  return true;
}

// One tile of a product; same ring of LDS slices and order of instructions as the layer's tiles
// (run_tile_bf16), on fp16.
template <int KIND, bool EXACT, class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
void newton_kernel(Product p) {
  MOE_LDS_RING(C, ring);
  constexpr bool kSym = KIND == kGram || KIND == kPoly;
  constexpr int MI = C::MI, NJ = C::NJ, BK = C::BK, S = C::STAGES, KS = BK / 16;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int64_t g;
  int tm, tn;
  if (!tile_of<kSym>(p, g, tm, tn)) return;
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int m_valid = min(C::BM, p.m_len - m0), n_valid = min(C::BN, p.n_len - n0);
  const int64_t a0 = g * p.a_mat + (int64_t)m0 * p.lda;
  const int64_t b0 = g * p.b_mat + (C::B_MN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
  // a tile with half of its columns valid keeps a wave with work on every SIMD (see wave_block)
  const bool spread = C::WGM == 2 && C::WGN == 4 && n_valid <= C::BN / 2 && m_valid > C::BM / 2;
  const int wm = spread ? wave % C::WGM : wave / C::WGN, wn = spread ? wave / C::WGM : wave % C::WGN;

  DmaOperand<C::BM, C::NW, false, 1, false, BK> da;
  DmaOperand<C::BN, C::NW, C::B_MN, 1, false, BK> db;
  da.init(p.lda, m_valid, wave, lane);
  db.init(p.ldb, n_valid, wave, lane);
  const int nk1 = p.k_len / BK, nk = EXACT ? 3 * nk1 : nk1;
  auto issue = [&](uint8_t* st, int kt) {
    int seg = 2, k = kt;      // exact: lo hi, hi lo, then hi hi (the small products first)
    if constexpr (EXACT) {
      seg = (kt >= nk1) + (kt >= 2 * nk1);
      k = kt - seg * nk1;
    }
    const uint16_t* a = (EXACT && seg == 0 ? p.al : p.ah) + a0 + k * BK;
    const uint16_t* b = (EXACT && seg == 1 ? p.bl : p.bh) + b0 + (C::B_MN ? (int64_t)k * BK * p.ldb : (int64_t)k * BK);
    da.issue(st, a, nullptr, 0, kt < nk, wave);
    db.issue(st + C::A_BYTES, b, nullptr, 0, kt < nk, wave);
  };

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  constexpr int kLoads = decltype(da)::kPerWave + decltype(db)::kPerWave;
  const int nk_pad = (nk + S - 1) / S * S;
  auto wait_slices = [&](int pending) {   // at most `pending` later slices outstanding
    if (S >= 4 && pending >= 2) wait_vmcnt<(S >= 4 ? 2 : 0) * kLoads>();
    else if (S >= 3 && pending >= 1) wait_vmcnt<(S >= 3 ? 1 : 0) * kLoads>();
    else wait_vmcnt<0>();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(ring[i], i);

  auto loop = [&](auto na_c) {
    constexpr int NA = decltype(na_c)::value;
    constexpr int kReads = NA == 0 ? 0 : NA + NJ * (C::B_MN ? 2 : 1);
    auto frags = [&](const uint8_t* st, int ks, bf16x8 (&av)[MI], bf16x8 (&bv)[NJ]) {
      if constexpr (NA > 0) {
        auto fa = [&](int i) {
          av[i] = kc_frag<BK>(st, wm * C::WM + 32 * i + (lane & 31), 2 * ks + (lane >> 5));
        };
        auto fb = [&](int j) {
          if constexpr (C::B_MN)
            bv[j] = mn_frag(st + C::A_BYTES, C::BN, wn * C::WN + 32 * j, ks, lane);
          else
            bv[j] = kc_frag<BK>(st + C::A_BYTES, wn * C::WN + 32 * j + (lane & 31), 2 * ks + (lane >> 5));
        };
        fb(0);
        fa(0);
#pragma unroll
        for (int j = 1; j < NJ; ++j) fb(j);
#pragma unroll
        for (int i = 1; i < NA; ++i) fa(i);
      }
    };
    auto mfma_step = [&](const bf16x8 (&av)[MI], const bf16x8 (&bv)[NJ]) {
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, av[i]),
                                                            __builtin_bit_cast(f16x8, bv[j]), acc[i][j], 0, 0, 0);
    };
    bf16x8 av[2][MI], bv[2][NJ];
    const bf16x8 zero = {};
#pragma unroll
    for (int i = 0; i < MI; ++i) av[1][i] = zero;   // "previous step" of slice 0: adds zeros
#pragma unroll
    for (int j = 0; j < NJ; ++j) bv[1][j] = zero;
    wait_slices(S - 2);
    lds_barrier();
    for (int kt0 = 0; kt0 < nk_pad; kt0 += S) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          frags(ring[i], ks, av[ks & 1], bv[ks & 1]);
          if (ks == 0) issue(ring[(i + S - 1) % S], kt0 + i + S - 1);
          mfma_step(av[(ks + 1) & 1], bv[(ks + 1) & 1]);
          if (ks == 0)
            interleave_step<0, NA * NJ, kReads, kLoads>();
          else
            interleave_step<0, NA * NJ, kReads, 0>();
          __builtin_amdgcn_sched_barrier(0);
        }
        wait_slices(min(S - 2, nk_pad - 2 - (kt0 + i)));
        lds_barrier();
      }
    }
    mfma_step(av[1], bv[1]);   // last step of the last slice
  };
  const int na = wn * C::WN >= n_valid ? 0 : max(0, min(MI, (m_valid - wm * C::WM + 31) / 32));
  with_count<MI>(__builtin_amdgcn_readfirstlane(na), loop);
  __syncthreads();
  newton_epilogue<KIND, EXACT, C>(p, g, m0, n0, kSym && tm != tn, acc, ring, wm, wn, wave, lane);
}

// Tiles of few or small matrices, where a launch is over in microseconds and the time is that of its
// longest chain: T x T tiles for many blocks, k split over the block's four waves (slices of 64 k in
// turn).  Each wave copies its own slices to LDS, with no barrier, one or two ahead; copies of whole
// 128-byte row pieces, as fragments read from memory touch 32 rows at 32 bytes each and take twice
// the time.  Both operands lie along k (X is kept with its transpose); the waves' sums meet in LDS in a fixed
// order.
template <int KIND, bool EXACT, int T, int D>   // D: slices of a wave in LDS
__global__ __launch_bounds__(256) void newton_small_kernel(Product p) {
  constexpr bool kSym = KIND == kGram || KIND == kPoly, kLast = KIND == kOut || KIND == kUpdate;
  constexpr bool kAux = KIND == kPoly || KIND == kAdd, kAuxLow = KIND == kPoly && EXACT;
  constexpr int B = T / 32;                       // 32-wide blocks of a side
  constexpr int P = EXACT ? 2 : 1;                // parts of a factor
  constexpr int kPlane = T * 64 * 2, kSlice = 2 * P * kPlane, kPart = 4 * T * (T + 1) * 4;
  // separate LDS objects, so that the copies into one do not hold up reads of the other
  __shared__ __align__(16) uint8_t ring0[4 * kSlice > kPart ? 4 * kSlice : kPart];
  __shared__ __align__(16) uint8_t ring1[D > 1 ? 4 * kSlice : 16];
  float (*const part)[T][T + 1] = reinterpret_cast<float (*)[T][T + 1]>(ring0);   // after the products
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int64_t g;
  int tm, tn;
  if (!tile_of<kSym>(p, g, tm, tn)) return;
  const int m0 = tm * T, n0 = tn * T;

  f32x16 acc[B][B];
#pragma unroll
  for (int i = 0; i < B; ++i)
#pragma unroll
    for (int j = 0; j < B; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  DmaOperand<T, 1, false, 1, false, 64> da, db;
  da.init(p.lda, T, 0, lane);
  db.init(p.ldb, T, 0, lane);
  constexpr int kLoads = P * (decltype(da)::kPerWave + decltype(db)::kPerWave);
  const int64_t a0 = g * p.a_mat + (int64_t)m0 * p.lda, b0 = g * p.b_mat + (int64_t)n0 * p.ldb;
  const int n_slices = p.k_len / 64;
  auto issue = [&](uint8_t* st, int c) {
    da.issue(st, p.ah + a0 + c * 64, nullptr, 0, true, 0);
    db.issue(st + P * kPlane, p.bh + b0 + c * 64, nullptr, 0, true, 0);
    if constexpr (EXACT) {
      da.issue(st + kPlane, p.al + a0 + c * 64, nullptr, 0, true, 0);
      db.issue(st + 3 * kPlane, p.bl + b0 + c * 64, nullptr, 0, true, 0);
    }
  };
  auto multiply = [&](const uint8_t* st) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      f16x8 av[P][B], bv[P][B];
#pragma unroll
      for (int h = 0; h < P; ++h)
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int row = 32 * i + (lane & 31), ch = 2 * ks + (lane >> 5);
          av[h][i] = __builtin_bit_cast(f16x8, kc_frag<64>(st + h * kPlane, row, ch));
          bv[h][i] = __builtin_bit_cast(f16x8, kc_frag<64>(st + (P + h) * kPlane, row, ch));
        }
#pragma unroll
      for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j) {
          if constexpr (EXACT) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[1][i], bv[0][j], acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[0][i], bv[1][j], acc[i][j], 0, 0, 0);
          }
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[0][i], bv[0][j], acc[i][j], 0, 0, 0);
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slice is read before it is refilled
    __builtin_amdgcn_sched_barrier(0);
  };
  uint8_t* const st0 = ring0 + wave * kSlice;
  uint8_t* const st1 = ring1 + (D > 1 ? wave * kSlice : 0);
  if (wave < n_slices) issue(st0, wave);
  if (D > 1 && wave + 4 < n_slices) issue(st1, wave + 4);
  for (int c = wave; c < n_slices; c += 4 * D) {
    if (D > 1 && c + 4 < n_slices) wait_vmcnt<kLoads>(); else wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
    multiply(st0);
    if (c + 4 * D < n_slices) issue(st0, c + 4 * D);
    if (D > 1 && c + 4 < n_slices) {
      if (c + 8 < n_slices) wait_vmcnt<kLoads>(); else wait_vmcnt<0>();
      __builtin_amdgcn_sched_barrier(0);
      multiply(st1);
      if (c + 12 < n_slices) issue(st1, c + 12);
    }
  }
  // what is added: loaded before the sums meet
  constexpr int kTurns = T * T / 1024, kCols = T / 4;
  const int64_t obase = g * p.o_mat;
  u32x2 aux_h[kAux ? kTurns : 1], aux_l[kAuxLow ? kTurns : 1];
#pragma unroll
  for (int it = 0; it < kTurns; ++it) {
    const int64_t at = obase + (int64_t)(m0 + it * (1024 / T) + tid / kCols) * p.ldo + n0 + 4 * (tid % kCols);
    if constexpr (kAux) aux_h[it] = *reinterpret_cast<const u32x2*>(p.ch + at);
    if constexpr (kAuxLow) aux_l[it] = *reinterpret_cast<const u32x2*>(p.cl + at);
  }
  __syncthreads();                                // every wave is done with its slices
#pragma unroll
  for (int i = 0; i < B; ++i)
#pragma unroll
    for (int j = 0; j < B; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        part[wave][32 * i + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)][32 * j + (lane & 31)] = acc[i][j][q];
  __syncthreads();
  UpdateScale scale = {};
  if constexpr (KIND == kUpdate) scale = update_scale(p);
  const bool turn = kSym ? tm != tn : kLast ? p.tall : true;   // a step writes X and its transpose
#pragma unroll
  for (int it = 0; it < kTurns; ++it) {
    const int row = it * (1024 / T) + tid / kCols, col = 4 * (tid % kCols);
    const int m = m0 + row, n = n0 + col;
    float s[4], x[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[e] = (part[0][row][col + e] + part[1][row][col + e]) + (part[2][row][col + e] + part[3][row][col + e]);
    if constexpr (kAux) join16(aux_h[it], kAuxLow ? &aux_l[it] : nullptr, x);
    finish4<KIND>(p, m, n, s, x, v);
    if constexpr (!kLast) {
      const int64_t at = obase + (int64_t)m * p.ldo + n;
      u32x2 hi, lo;
      split16(v, hi, lo);
      *reinterpret_cast<u32x2*>(p.oh + at) = hi;
      if (EXACT || (!kSym && p.ol)) *reinterpret_cast<u32x2*>(p.ol + at) = lo;
    } else if (!turn) {
      emit4<KIND>(p, p.g0 + g, m, n, v, scale);
    }
    if (turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) part[0][row][col + e] = v[e];   // read by this thread alone so far
    }
  }
  if (!turn) return;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kTurns; ++it) {
    const int n = it * (1024 / T) + tid / kCols, m4 = 4 * (tid % kCols);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = part[0][m4 + e][n];
    if constexpr (!kLast) {
      u32x2 hi, lo;
      split16(v, hi, lo);
      uint16_t* const th = kSym ? p.oh + obase : p.th + g * p.o_mat;
      uint16_t* const tl = kSym ? p.ol + obase : p.tl + g * p.o_mat;
      const int64_t at = (int64_t)(n0 + n) * (kSym ? p.ldo : p.ldt) + m0 + m4;
      *reinterpret_cast<u32x2*>(th + at) = hi;
      if (EXACT) *reinterpret_cast<u32x2*>(tl + at) = lo;
    } else {
      emit4<KIND>(p, p.g0 + g, n0 + n, m0 + m4, v, scale);
    }
  }
}

// --------------------------------------------------------- before the products

struct Source {
  const float* g;
  float* mom;         // NULL: the matrices themselves
  float momentum;
  bool nesterov;
  int R, C, g0;
  int parts;
  double* sums;       // [batch][kNormParts]
};

__device__ __forceinline__ float direction(const Source& s, float grad, float mom) {
  return s.nesterov ? fmaf(s.momentum, mom, grad) : mom;
}

// Sums of squares of part `blockIdx.x` of matrix blockIdx.y, in 64 bits (no scale of the entries
// overflows or vanishes); with momentum, its update on the way.
template <int V>
__global__ __launch_bounds__(256) void newton_squares_kernel(Source s) {
  __shared__ double red[4];
  const int tid = threadIdx.x;
  const int64_t n = (int64_t)s.R * s.C / V, base = (int64_t)(s.g0 + blockIdx.y) * s.R * s.C;
  double sum = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < n; i += (int64_t)s.parts * 256) {
    float v[V];
    const float* gp = s.g + base + i * V;
    if constexpr (V == 4) Elem<float>::unpack(ld16(gp), v);
    else v[0] = *gp;
    if (s.mom) {
      float m[V];
      float* mp = s.mom + base + i * V;
      if constexpr (V == 4) Elem<float>::unpack(ld16(mp), m);
      else m[0] = *mp;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        m[e] = fmaf(s.momentum, m[e], v[e]);
        v[e] = direction(s, v[e], m[e]);
      }
      if constexpr (V == 4) st16(mp, Elem<float>::pack(m));
      else *mp = m[0];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sum = fma((double)v[e], (double)v[e], sum);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if ((tid & 63) == 0) red[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) s.sums[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X = U / |U| in fp16 parts, zeros in the padding: one 64 x 64 tile of the matrix for each block.  Its
// own orientation goes straight from registers, the other one through LDS: X is the transpose of a
// tall matrix; th and tl (small matrices) take the transpose of X.
struct Start {
  bool tall;
  int sp, lp;
  uint16_t *xh, *xl, *th, *tl;   // xl, tl NULL: upper parts only; th NULL: X alone
};
template <int V>
__global__ __launch_bounds__(256) void newton_start_kernel(Source s, Start d) {
  __shared__ float tile[64][65];
  const int tid = threadIdx.x, lane = tid & 63;
  const int rp = d.tall ? d.lp : d.sp, cp = d.tall ? d.sp : d.lp;
  const int ct = cp / 64, per = ct * (rp / 64);
  const int64_t b = blockIdx.x / per;
  const int rem = (int)(blockIdx.x - b * per);
  const int r0 = rem / ct * 64, c0 = rem % ct * 64;
  const int64_t base = (s.g0 + b) * s.R * s.C;
  float u[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + (tid >> 4) + 16 * j, c = c0 + 4 * (tid & 15);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[j][e] = 0.f;
    if (r < s.R && c < s.C) {
      const int64_t at = base + (int64_t)r * s.C + c;
      float m[4] = {0.f, 0.f, 0.f, 0.f};
      const bool grad = !s.mom || s.nesterov;
      if constexpr (V == 4) {
        if (grad) Elem<float>::unpack(ld16(s.g + at), u[j]);
        if (s.mom) Elem<float>::unpack(ld16(s.mom + at), m);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < s.C) {
            if (grad) u[j][e] = s.g[at + e];
            if (s.mom) m[e] = s.mom[at + e];
          }
      }
      if (s.mom) {
#pragma unroll
        for (int e = 0; e < 4; ++e) u[j][e] = direction(s, u[j][e], m[e]);
      }
    }
  }
  double sum = 0.0;
  for (int i = lane; i < s.parts; i += kWave) sum += s.sums[b * kNormParts + i];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  // zeros stay zeros; an infinity or NaN anywhere makes the whole matrix NaN
  const double inv = sum == 0.0 ? 0.0 : sum < (double)INFINITY ? (double)kXScale / sqrt(sum) : (double)NAN;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) u[j][e] = (float)((double)u[j][e] * inv);
  auto store = [&](uint16_t* hp, uint16_t* lp, int rows, int ld, int x0, int y0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x2 hi, lo;
      split16(u[j], hi, lo);
      const int64_t at = (b * rows + x0 + (tid >> 4) + 16 * j) * ld + y0 + 4 * (tid & 15);
      *reinterpret_cast<u32x2*>(hp + at) = hi;
      if (lp) *reinterpret_cast<u32x2*>(lp + at) = lo;
    }
  };
  uint16_t *const own_h = d.tall ? d.th : d.xh, *const own_l = d.tall ? d.tl : d.xl;
  uint16_t *const turned_h = d.tall ? d.xh : d.th, *const turned_l = d.tall ? d.xl : d.tl;
  if (own_h) store(own_h, own_l, rp, cp, r0, c0);
  if (!turned_h) return;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[(tid >> 4) + 16 * j][4 * (tid & 15) + e] = u[j][e];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) u[j][e] = tile[4 * (tid & 15) + e][(tid >> 4) + 16 * j];
  store(turned_h, turned_l, cp, rp, c0, r0);
}

// ---------------------------------------------------------------------- few rows
//
// With few rows the iteration runs on the rows alone.  Every X_k is a polynomial of A_0 = U U^T / |U|^2 times
// X_0, so with P_0 = I
//   B_k = a + b A_k + c A_k^2,   P_k+1 = P_k B_k,   A_k+1 = B_k A_k B_k,   result = P U / |U|:
// two passes over U and products of [s, s] between them, three launches for 17.  All of these matrices are
// symmetric and commute.  What a rounding puts into a null direction of A_0 grows by a^2 with every step, as X's
// own does by a, but nothing keeps it from turning negative: hence 64 bits throughout, and only as long as
// the product of a^2 leaves 1e-8 of that (kFewGrow).  |U|^2 is the trace.  Bound by the matrix cores' rate in
// 64 bits (a [64, 64] product 3 us on its CU) and, for fewer rows, by the chain of loads, barriers and launches: of
// 64 [32, 1000] 8.2 + 14.9 + 9.0 us, of 1 [12, 14336] 5.2 + 11.1 + 4.0, of 64 [64, 14336] 150 + 52 + 303.

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kFewPitch = 4;          // of a row in LDS, beyond its doubles: rows 8 banks apart
constexpr double kFewGrow = 4096.0;   // largest product of |a|

// Rows of a result: register r of a lane holds row 4 r + lane / 16 of column lane % 16.
__device__ __forceinline__ f64x4 mfma64(double a, double b, const f64x4& c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

struct Few {
  Source u;
  bool tall;
  int s, l, chunk, chunks;
  double *parts, *poly;   // [G][chunks][tiles][256], [G][16 NB][16 NB]
};

// Sums of products of rows over `chunk` of l (a quarter to each wave), tiles on and above the diagonal; with
// momentum, its update on the way.  A lane's element is both operands': X[16 i + lane % 16][k + lane / 16].
template <int NB>
__global__ __launch_bounds__(256) void newton_few_gram_kernel(Few f) {
  constexpr int NT = NB * (NB + 1) / 2;
  __shared__ double sums[3][NT][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
  const int64_t g = blockIdx.x / f.chunks;
  const int c = (int)(blockIdx.x - g * f.chunks);
  const int64_t base = (f.u.g0 + g) * f.s * f.l;
  f64x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f64x4{0, 0, 0, 0};
  const int k1 = min(f.l, (c + 1) * f.chunk), per = f.chunk / 4;
  const int w0 = c * f.chunk + wave * per, w1 = min(k1, w0 + per);
  for (int k0 = w0; k0 < w1; k0 += 16) {
    float x[4][NB], m[4][NB];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        // rows are contiguous along k, or (tall) along the rows of X: a lane's four k, or 16 lanes' rows
        const int r = 16 * i + i16, k = f.tall ? k0 + 4 * e + q : k0 + 4 * q + e;
        const bool in = r < f.s && k < w1;
        const int64_t at = base + (f.tall ? (int64_t)k * f.s + r : (int64_t)r * f.l + k);
        x[e][i] = in ? f.u.g[at] : 0.f;
        m[e][i] = in && f.u.mom ? f.u.mom[at] : 0.f;
      }
    if (f.u.mom) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int r = 16 * i + i16, k = f.tall ? k0 + 4 * e + q : k0 + 4 * q + e;
          m[e][i] = fmaf(f.u.momentum, m[e][i], x[e][i]);
          if (r < f.s && k < w1) f.u.mom[base + (f.tall ? (int64_t)k * f.s + r : (int64_t)r * f.l + k)] = m[e][i];
          x[e][i] = direction(f.u, x[e][i], m[e][i]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int t = 0;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i <= j; ++i, ++t) acc[t] = mfma64((double)x[e][i], (double)x[e][j], acc[t]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave - 1][t][r][lane] = acc[t][r];
  }
  __syncthreads();
  if (wave > 0) return;
  double* const out = f.parts + (int64_t)blockIdx.x * NT * 256 + lane;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      out[t * 256 + r * 64] = (acc[t][r] + sums[0][t][r][lane]) + (sums[1][t][r][lane] + sums[2][t][r][lane]);
}

struct FewCoef { int steps; float c[16][3]; };

// The iteration on [16 NB, 16 NB], one block for each matrix: the tiles of a product shared out to the waves (up to
// four on a SIMD, to overlap their chains: 8 [64, 64] 72 us with one, 64 with four), mirrored when they are
// written.
template <int NB>
struct FewWaves { static constexpr int N = NB == 1 ? 2 : NB == 2 ? 4 : 16; };
template <int NB>
__global__ __launch_bounds__(64 * FewWaves<NB>::N) void newton_few_steps_kernel(Few f, FewCoef coef) {
  constexpr int N = 16 * NB, NT = NB * (NB + 1) / 2, W = N + kFewPitch, NW = FewWaves<NB>::N, TW = (2 * NT + NW - 1) / NW;
  __shared__ double A[N * W], B[N * W], T[N * W], P[N * W];
  __shared__ double trace;
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t g = blockIdx.x;
  struct Tile { int i, j; };
  auto tile = [](int t) {   // column by column
    const int j = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
    return Tile{t - j * (j + 1) / 2, j};
  };
  auto product = [&](const double* x, const double* y, Tile t) {   // symmetric ones: both operands by rows
    f64x4 s = {0, 0, 0, 0};
    const double* const xr = x + (16 * t.i + i16) * W + q;
    const double* const yr = y + (16 * t.j + i16) * W + q;
#pragma unroll
    for (int k = 0; k < N; k += 4) s = mfma64(xr[k], yr[k], s);
    return s;
  };
  auto store = [&](double* z, Tile t, const f64x4& v) {
    const int col = 16 * t.j + i16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * t.i + 4 * r + q;
      if (row > col) continue;          // a diagonal tile's lower half mirrors its upper one
      z[row * W + col] = v[r];
      z[col * W + row] = v[r];
    }
  };
  const double* const parts = f.parts + g * f.chunks * NT * 256 + lane;
  for (int t = wave; t < NT; t += NW) {
    f64x4 v = {0, 0, 0, 0};
    for (int c0 = 0; c0 < f.chunks; c0 += 8) {   // eight at a time, the last ones, too: each wait is a trip to memory
      double x[8][4];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[u][r] = parts[((int64_t)min(c0 + u, f.chunks - 1) * NT + t) * 256 + r * 64];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += c0 + u < f.chunks ? x[u][r] : 0.0;
    }
    store(A, tile(t), v);
  }
  __syncthreads();
  if (wave == 0) {
    double d = lane < N ? A[lane * W + lane] : 0.0;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) d += __shfl_xor(d, o, kWave);
    if (lane == 0) trace = d;
  }
  __syncthreads();
  const double total = trace;
  // zeros stay zeros; an infinity or NaN makes the whole matrix NaN
  const double inv = total == 0.0 ? 0.0 : total < (double)INFINITY ? 1.0 / total : (double)NAN;
  for (int e = tid; e < N * N; e += 64 * NW) A[e / N * W + e % N] *= inv;
  __syncthreads();
  for (int k = 0; k < coef.steps; ++k) {
    const double a = coef.c[k][0], b = coef.c[k][1], c = coef.c[k][2];
    for (int t = wave; t < NT; t += NW) {
      const Tile at = tile(t);
      f64x4 s = product(A, A, at);
      const int col = 16 * at.j + i16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * at.i + 4 * r + q;
        s[r] = (row == col ? a : 0.0) + b * A[row * W + col] + c * s[r];
      }
      store(B, at, s);
      if (k == 0) store(P, at, s);
    }
    __syncthreads();
    // B A and P B, which waits in registers until P is read
    const bool last = k + 1 == coef.steps;
    f64x4 next[TW];
#pragma unroll
    for (int n = 0; n < TW; ++n) {
      const int t = wave + n * NW;
      if (t < NT && !last) store(T, tile(t), product(B, A, tile(t)));
      if (t >= NT && t < 2 * NT && k > 0) next[n] = product(P, B, tile(t - NT));
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < TW; ++n) {
      const int t = wave + n * NW;
      if (t >= NT && t < 2 * NT && k > 0) store(P, tile(t - NT), next[n]);
    }
    if (!last)
      for (int t = wave; t < NT; t += NW) store(A, tile(t), product(T, B, tile(t)));
    __syncthreads();
  }
  const double scale = sqrt(inv);
  for (int e = tid; e < N * N; e += 64 * NW) f.poly[g * N * N + e] = P[e / N * W + e % N] * scale;
}

// Result P U, 16 columns to a wave at a time.  The order of the operands is that of the result in memory.
template <int NB, int KIND>
__global__ __launch_bounds__(256) void newton_few_apply_kernel(Few f, Product p, int blocks) {
  constexpr int N = 16 * NB, W = N + kFewPitch;
  __shared__ double P[N * W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i16 = lane & 15, q = lane >> 4;
  const int64_t g = blockIdx.x / blocks, base = (f.u.g0 + g) * f.s * f.l;
  for (int e = tid; e < N * N; e += 256) P[e / N * W + e % N] = f.poly[g * N * N + e];
  __syncthreads();
  UpdateScale scale = {};
  if constexpr (KIND == kUpdate) scale = update_scale(p);
  const bool grad = !f.u.mom || f.u.nesterov;
  for (int64_t n0 = ((blockIdx.x - g * blocks) * 4 + wave) * 16; n0 < f.l; n0 += (int64_t)blocks * 64) {
    const int64_t n = n0 + i16;
    f64x4 acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = f64x4{0, 0, 0, 0};
    float x[4 * NB];
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
      const int k = f.tall ? e / 4 * 16 + 4 * q + e % 4 : 4 * e + q;
      const bool in = k < f.s && n < f.l;
      const int64_t at = base + (f.tall ? n * f.s + k : k * (int64_t)f.l + n);
      float u = in && grad ? f.u.g[at] : 0.f;
      if (f.u.mom) u = direction(f.u, u, in ? f.u.mom[at] : 0.f);
      x[e] = u;
    }
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
      const int k = f.tall ? e / 4 * 16 + 4 * q + e % 4 : 4 * e + q;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const double pe = P[(16 * i + i16) * W + k], xe = x[e];
        acc[i] = f.tall ? mfma64(xe, pe, acc[i]) : mfma64(pe, xe, acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // tall: rows of the result are columns of X
        const int64_t row = f.tall ? n0 + 4 * r + q : 16 * i + 4 * r + q, col = f.tall ? 16 * i + i16 : n;
        if (row >= p.R || col >= p.C) continue;
        const int64_t at = ((p.g0 + g) * p.R + row) * p.C + col;
        const float v = (float)acc[i][r];
        if constexpr (KIND == kOut) {
          if (p.bf16) static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_to_bf16(v);
          else static_cast<float*>(p.out)[at] = v;
        } else {
          const float m = scale.keep * p.master[at] - scale.gain * v;
          p.master[at] = m;
          if (p.w) p.w[at] = (uint16_t)f32_to_bf16(m);
        }
      }
  }
}

// ---------------------------------------------------------------------- host

// Up to so many 64 x 64 tiles a product takes small tiles (for X, which then is kept with its transpose: whole
// calls of 32 [256, 256] 119 us with small tiles and 139 without).
constexpr int kSmallTiles = 512;

inline int up(int v, int to) { return (v + to - 1) / to * to; }

unsigned xcd_grid(int tiles) { return (unsigned)kXcds * ((tiles + kXcds - 1) / kXcds); }

template <int KIND, bool EXACT, class C>
hipError_t product_with(Product p, int batch, hipStream_t st) {
  p.mt = (p.m_len + C::BM - 1) / C::BM;
  p.nt = (p.n_len + C::BN - 1) / C::BN;
  p.per = KIND == kGram || KIND == kPoly ? p.mt * (p.mt + 1) / 2 : p.mt * p.nt;
  p.tiles = p.per * batch;
  newton_kernel<KIND, EXACT, C><<<xcd_grid(p.tiles), C::NT, 0, st>>>(p);
  return hipGetLastError();
}

template <int KIND, bool EXACT, int T, int D>
hipError_t product_small(Product p, int batch, hipStream_t st) {
  p.mt = p.m_len / T;
  p.nt = p.n_len / T;
  p.per = KIND == kGram || KIND == kPoly ? p.mt * (p.mt + 1) / 2 : p.mt * p.nt;
  p.tiles = p.per * batch;
  newton_small_kernel<KIND, EXACT, T, D><<<xcd_grid(p.tiles), 256, 0, st>>>(p);
  return hipGetLastError();
}

// Time of a product in rounds of tiles over 256 CUs: the last round counts in full as long as there are
// few.  One 256 x 256 tile of a CU takes 1.65 (us for each 64 k), two 128 x 128 ones 1.25, a single one 0.75.
double rounds(int64_t tiles, int at_once) {
  return tiles <= 4 * at_once ? (double)((tiles + at_once - 1) / at_once) : (double)tiles / at_once;
}
double big_rounds(int64_t tiles) { return 1.65 * rounds(tiles, 256); }
double mid_rounds(int64_t tiles) { return tiles <= 256 ? 0.75 : 1.25 * rounds(tiles, 512); }

// Tiles by their number.  A and B of 1 [1024, 8192] (us; 256 x 256, 128 x 128 and small tiles): 405, 213, 60 and
// 66, 34, 15 (f32); of 20 [300, 2000] 38, 23, 16 and 15, 9, 8; of 4 [1000, 1000] 26, 15, 17; of 6 [1100, 1100] 30, 21,
// 28; of 1 [4096, 4096] the whole call 1476 with 256 x 256, 1800 with 128 x 128.  X of 8 [512, 1024] 17, 10, 16; of
// 20 [300, 2000] 28, 20, 39; of 3 [700, 5000] f32 56, 60, 113.  By those of `part` matrices, a whole part of the
// stack, also where the last part holds fewer: small tiles sum in another order, and a matrix's bits may not depend
// on its place in the stack.
template <int KIND, bool EXACT>
hipError_t product(const Product& p, bool small, int part, int batch, hipStream_t st) {
  constexpr bool kMn = KIND != kGram && KIND != kPoly;
  using Big = NsCfg<256, 256, 2, 4, 64, 2, kMn>;
  using Mid = NsCfg<128, 128, 2, 2, 64, 2, kMn>;
  auto tiles = [&](int t) {
    const int64_t mt = (p.m_len + t - 1) / t, nt = (p.n_len + t - 1) / t;
    return part * (kMn ? mt * nt : mt * (mt + 1) / 2);
  };
  if (!kMn) small = tiles(64) <= kSmallTiles;   // both operands lie along k in any case
  // 32 x 32 tiles until there are two for each CU: whole calls of [512, 512] 95 us with them and 148
  // with 64 x 64 ones (f32), of [1024, 1024] 296 and 223.  Two slices of two parts take a CU's LDS, so they
  // are for one tile on a CU: 5 [264, 416] 128 us with two, 110 with one; [64, 14336] 246 and 293.
  if (small) {
    if (tiles(32) > 512) return product_small<KIND, EXACT, 64, 1>(p, batch, st);
    if constexpr (EXACT) {
      if (tiles(32) > 256) return product_small<KIND, EXACT, 32, 1>(p, batch, st);
    }
    return product_small<KIND, EXACT, 32, 2>(p, batch, st);
  }
  return big_rounds(tiles(256)) <= mid_rounds(tiles(128)) ? product_with<KIND, EXACT, Big>(p, batch, st)
                                                          : product_with<KIND, EXACT, Mid>(p, batch, st);
}
template <int KIND>
hipError_t product(const Product& q, const NewtonPlan& p, int batch, hipStream_t st) {
  if constexpr (KIND != kAdd) {   // the exact form has a in B's diagonal
    if (p.exact) return product<KIND, true>(q, p.small, p.batch, batch, st);
  }
  return product<KIND, false>(q, p.small, p.batch, batch, st);
}

// Whether X keeps its lower part for step k: a rounding of X (2^-12 of an element) has null
// directions, which the steps from k on make up to |a_k a_k+1 ...| times larger.  Up to
// kDropLow that stays at 3e-3 of the norm, next to 1e-3 to 3e-3 of the products' own roundings (default steps); for
// the last step it is only its own |a|.
constexpr float kDropLow = 12.f;
bool keeps_low(const NewtonCall& c, int k) {
  if (c.p.exact) return true;
  if (k == c.steps - 1) return false;
  float grow = 1.f;
  for (int j = k; j < c.steps; ++j) grow *= fmaxf(1.f, fabsf(c.coef[j][0]));
  return grow > kDropLow;
}

// The power of two that the last step's B is stored by, on top of kAScale.  A step before the last leaves singular
// values of at most 15, so its |B| = |a + b s^2 + c s^4| is at most 15 / s where s is large, and below fp16's 255
// where s is not (coefficients are at most 32: s < 1.4).  The last step may leave any value, and its B be up to
// 32 (1 + 15^2 + 15^4).  The largest s that can enter it follows from the coefficients (1 at the start, then the
// extremes of a s + b s^3 + c s^5), and from that the largest |B|, which takes half of fp16's range: a sum that its
// roundings enlarge still fits.  1 where |B| stays within 128, as in every iteration that tends to 1.
float last_scale(const NewtonCall& c) {
  double s = 1.0;
  for (int k = 0; k + 1 < c.steps; ++k) {
    const double a = c.coef[k][0], b = c.coef[k][1], q = c.coef[k][2];
    const double h = -0.5 * (3.0 * b + copysign(sqrt(fmax(0.0, 9.0 * b * b - 20.0 * a * q)), b));
    double most = 0.0;
    for (const double t : {s * s, h / (5.0 * q), a / h})   // s^2: the end, and where a + 3 b t + 5 q t^2 = 0
      if (t > 0.0 && t <= s * s) most = fmax(most, fabs(a + t * (b + t * q)) * sqrt(t));
    s = fmin(15.0, most);
  }
  const float* const f = c.coef[c.steps - 1];
  const double a = f[0], b = f[1], q = f[2];
  double most = fabs(a);
  for (const double t : {s * s, -b / (2.0 * q)})
    if (t > 0.0 && t <= s * s) most = fmax(most, fabs(a + t * (b + t * q)));
  float scale = 1.f;
  while (most * kAScale * scale > 32768.0) scale *= 0.5f;
  return scale;
}

// What the last launch of a call writes.
void results(const NewtonCall& c, Product& q) {
  q.tall = c.p.tall; q.bf16 = c.bf16;
  q.R = c.p.R; q.C = c.p.C;
  q.out = c.out; q.master = c.master; q.w = c.w;
  q.lr_dev = c.lr_dev; q.lr = c.lr; q.weight_decay = c.weight_decay; q.scale = c.scale;
}

bool few_steps(const NewtonCall& c) {
  double grow = 1.0;
  for (int k = 0; k < c.steps; ++k) grow *= fmax(1.0, fabs((double)c.coef[k][0]));
  return c.p.few && grow <= kFewGrow;
}

template <int NB>
hipError_t launch_few(const NewtonCall& c, Source u, hipStream_t st) {
  const NewtonPlan& p = c.p;
  Few f{};
  f.tall = p.tall;
  f.s = p.s; f.l = p.l; f.chunk = p.chunk; f.chunks = p.chunks;
  f.parts = static_cast<double*>(c.ws);
  f.poly = f.parts + (int64_t)p.few_batch * p.chunks * (NB * (NB + 1) / 2) * 256;
  FewCoef coef;
  coef.steps = c.steps;
  for (int k = 0; k < c.steps; ++k)
    for (int i = 0; i < 3; ++i) coef.c[k][i] = c.coef[k][i];
  Product q{};
  results(c, q);
  for (int g0 = 0; g0 < p.G; g0 += p.few_batch) {
    const int batch = p.G - g0 < p.few_batch ? p.G - g0 : p.few_batch;
    // Blocks of 64 columns, about 1024 in all.  By their registers a CU holds eight of them at a time for 16 rows, four for
    // 32, three for 48 and two for 64.
    const int64_t want = (p.l + 63) / 64, most = 1024 / batch + 1;
    const int blocks = (int)(want < most ? want : most);
    u.g0 = q.g0 = g0;
    f.u = u;
    newton_few_gram_kernel<NB><<<batch * p.chunks, 256, 0, st>>>(f);
    newton_few_steps_kernel<NB><<<batch, 64 * FewWaves<NB>::N, 0, st>>>(f, coef);
    if (c.out) newton_few_apply_kernel<NB, kOut><<<batch * blocks, 256, 0, st>>>(f, q, blocks);
    else newton_few_apply_kernel<NB, kUpdate><<<batch * blocks, 256, 0, st>>>(f, q, blocks);
  }
  return hipGetLastError();
}

}  // namespace

NewtonPlan newton_plan(int G, int R, int C, bool exact) {
  NewtonPlan p{};
  p.G = G; p.R = R; p.C = C;
  p.tall = R > C;
  p.s = p.tall ? C : R;
  p.l = p.tall ? R : C;
  p.sp = up(p.s, kNewtonPad);
  p.lp = up(p.l, kNewtonPad);
  p.exact = exact || p.s < kNewtonFewRows;
  p.small = (int64_t)G * (p.sp / 64) * (p.lp / 64) <= kSmallTiles;
  // About 2048 tiles of 256 x 256 to a launch: 8 rounds over the 256 CUs, of which the last one
  // is partly empty; more would only take memory (at most 2^30 elements of X, or one matrix).
  const int64_t t = (p.sp + 255) / 256, tiles = t * (t + 1) / 2;
  const int64_t fit = ((int64_t)1 << 30) / ((int64_t)p.sp * p.lp);
  int64_t most = (2048 + tiles - 1) / tiles;
  if (most > fit) most = fit > 1 ? fit : 1;
  const int64_t batches = (G + most - 1) / most;
  p.batch = (int)((G + batches - 1) / batches);
  const size_t x = (size_t)p.batch * p.sp * p.lp * 2, a = (size_t)p.batch * p.sp * p.sp * 2;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.parts = take((size_t)p.batch * kNormParts * sizeof(double));
  for (int i = 0; i < 2; ++i) {
    p.xh[i] = take(x);
    p.xl[i] = take(x);
    p.th[i] = take(p.small ? x : 0);
    p.tl[i] = take(p.small && p.exact ? x : 0);
  }
  p.ah = take(a);
  p.bh = take(a);
  p.al = take(p.exact ? a : 0);
  p.bl = take(p.exact ? a : 0);
  // On the rows alone: 56 to 248 us without, 13 to 20 with (1 [8, 8], 1 [12, 14336]); 64 [48, 14336] 751 (bf16) and
  // 1076 (f32), 268 and 280.  Products of 64 rows in 64 bits take 50 us: 8 [64, 500] 57 and 66, 68; 1 [64, 2000]
  // 70 and 84, 74; 64 [64, 3000] 180 and 230, 162.
  p.few = p.s <= 48 || (p.s <= 64 && p.l >= 2048);
  if (p.few) {
    p.few_batch = G < kNewtonFewBatch ? G : kNewtonFewBatch;
    // a chunk costs its length (18 ns a column for 64 rows) and its sums' reading (0.13 us): about sqrt(l) / 3
    const int nb = (p.s + 15) / 16;
    int64_t chunks = (int64_t)(0.375 * sqrt((double)p.l)) + 1;
    if (chunks > 1024 / p.few_batch + 1) chunks = 1024 / p.few_batch + 1;
    p.chunk = up((int)((p.l + chunks - 1) / chunks), 64);
    p.chunks = (p.l + p.chunk - 1) / p.chunk;
    const size_t each = (size_t)p.chunks * (nb * (nb + 1) / 2) * 256 + (size_t)nb * nb * 256;
    const size_t need = (size_t)p.few_batch * each * sizeof(double);
    if (off < need) off = (need + 255) / 256 * 256;
  }
  p.total = off;
  return p;
}

hipError_t launch_newton(const NewtonCall& c, hipStream_t st) {
  const NewtonPlan& p = c.p;
  auto at = [&](size_t off) { return reinterpret_cast<uint16_t*>(static_cast<char*>(c.ws) + off); };
  uint16_t *const ah = at(p.ah), *const al = at(p.al), *const bh = at(p.bh), *const bl = at(p.bl);
  const int64_t n = (int64_t)p.R * p.C;
  if (few_steps(c)) {
    Source s{};
    s.g = c.g;
    s.mom = c.mom;
    s.momentum = c.momentum;
    s.nesterov = c.nesterov;
    switch ((p.s + 15) / 16) {
      case 1: return launch_few<1>(c, s, st);
      case 2: return launch_few<2>(c, s, st);
      case 3: return launch_few<3>(c, s, st);
      default: return launch_few<4>(c, s, st);
    }
  }
  const float last_b = last_scale(c);
  for (int g0 = 0; g0 < p.G; g0 += p.batch) {
    const int batch = p.G - g0 < p.batch ? p.G - g0 : p.batch;
    Source s{};
    s.g = c.g;
    s.mom = c.mom;
    s.momentum = c.momentum;
    s.nesterov = c.nesterov;
    s.R = p.R; s.C = p.C; s.g0 = g0;
    s.sums = reinterpret_cast<double*>(at(p.parts));
    const int64_t want = (n + 4095) / 4096;   // 16 elements or more to a thread
    s.parts = (int)(want < kNormParts ? want : kNormParts);
    const unsigned tiles = (unsigned)((int64_t)batch * (p.sp / 64) * (p.lp / 64));
    Start d{p.tall, p.sp, p.lp, at(p.xh[0]), keeps_low(c, 0) ? at(p.xl[0]) : nullptr,
            p.small ? at(p.th[0]) : nullptr, p.small && p.exact ? at(p.tl[0]) : nullptr};
    const dim3 sq(s.parts, batch);
    if (n % 4 == 0) newton_squares_kernel<4><<<sq, 256, 0, st>>>(s);
    else newton_squares_kernel<1><<<sq, 256, 0, st>>>(s);
    if (p.C % 4 == 0) newton_start_kernel<4><<<tiles, 256, 0, st>>>(s, d);
    else newton_start_kernel<1><<<tiles, 256, 0, st>>>(s, d);
    for (int k = 0; k < c.steps; ++k) {
      const uint16_t *xh = at(p.xh[k & 1]), *xl = at(p.xl[k & 1]);
      const int64_t x_mat = (int64_t)p.sp * p.lp, a_mat = (int64_t)p.sp * p.sp;
      const bool last = k + 1 == c.steps, add = !p.exact && keeps_low(c, k);
      Product q{};
      const float bs = last ? last_b : 1.f;   // of the stored B
      q.a = c.coef[k][0] * bs; q.b = c.coef[k][1] * bs; q.c = c.coef[k][2] * bs;
      q.ah = xh; q.al = xl; q.bh = xh; q.bl = xl;
      q.a_mat = q.b_mat = x_mat;
      q.lda = q.ldb = q.k_len = p.lp;
      q.m_len = q.n_len = p.sp;
      q.oh = ah; q.ol = al; q.o_mat = a_mat; q.ldo = p.sp;
      hipError_t e = product<kGram>(q, p, batch, st);
      if (e != hipSuccess) return e;
      q.ah = ah; q.al = al; q.bh = ah; q.bl = al;
      q.a_mat = q.b_mat = a_mat;
      q.lda = q.ldb = q.k_len = p.sp;
      q.ch = ah; q.cl = al;
      q.oh = bh; q.ol = bl;
      e = product<kPoly>(q, p, batch, st);
      if (e != hipSuccess) return e;
      q.ah = bh; q.al = bl;
      q.bh = p.small ? at(p.th[k & 1]) : xh;
      q.bl = p.small ? at(p.tl[k & 1]) : xl;
      q.a_mat = a_mat; q.b_mat = x_mat;
      q.lda = q.k_len = p.sp; q.ldb = p.small ? p.sp : p.lp;
      q.n_len = p.lp;
      q.ch = xl;
      q.o_mat = x_mat; q.ldo = p.lp;
      if (!last) {
        q.oh = at(p.xh[(k + 1) & 1]);
        q.ol = keeps_low(c, k + 1) ? at(p.xl[(k + 1) & 1]) : nullptr;
        q.th = at(p.th[(k + 1) & 1]);
        q.tl = at(p.tl[(k + 1) & 1]);
        q.ldt = p.sp;
        e = add ? product<kAdd>(q, p, batch, st) : product<kStep>(q, p, batch, st);
      } else {
        results(c, q);
        q.undo = 1.f / (kAScale * kXScale * bs);
        q.g0 = g0;
        e = c.out ? product<kOut>(q, p, batch, st) : product<kUpdate>(q, p, batch, st);
      }
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace moe
