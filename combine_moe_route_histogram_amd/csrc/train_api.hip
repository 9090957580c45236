// C entry points of include/moe_train.h: argument checks, workspace layout, launches.
#include <cmath>

#include "api.hpp"
#include "balance.hpp"
#include "muon.hpp"

using namespace moe;

namespace {

int check_ws_bytes(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(MOE_EWORKSPACE, "workspace is NULL (need %zu bytes)", need);
  if (reinterpret_cast<uintptr_t>(ws) % kAlign)
    return fail(MOE_EWORKSPACE, "workspace must be %zu-byte aligned", kAlign);
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, need %zu", ws_bytes, need);
  return MOE_OK;
}

// ---- router losses

constexpr int kBalanceMaxTokens = 1 << 28;   // a launch holds less than 2^32 threads

int check_balance(const moe_dims* d, int seq_len) {
  MOE_TRY(check_dims(d));
  if (d->T > kBalanceMaxTokens)
    return fail(MOE_EUNSUPPORTED, "the router's losses take at most %d tokens (T=%d)", kBalanceMaxTokens, d->T);
  if (seq_len < 1 || seq_len > d->T)
    return fail(MOE_EINVAL, "seq_len must be in [1, T] (got seq_len=%d, T=%d)", seq_len, d->T);
  return MOE_OK;
}

int sequences(const moe_dims* d, int seq_len) { return d->T / seq_len + (d->T % seq_len != 0); }

// Workspace sections (byte offsets).
struct BalanceLayout {
  int S, by, chunk, cps, eb, entries;
  size_t part_p, part_c, part_z, part_n, seq_loss, seq_z, seq_n, seq_some, ticket, total;
};
BalanceLayout balance_layout(const moe_dims* d, int seq_len) {
  BalanceLayout L;
  L.S = sequences(d, seq_len);
  // a lane group or a wave for a sequence, or blocks for chunks of it
  L.by = seq_len <= kBalanceFew ? kByGroup
       : seq_len <= kBalanceShort || (seq_len <= kBalanceShortMany && L.S >= kBalanceMany) ? kByWave : kByChunk;
  // Chunks of up to 64 tokens for each of 8 waves where that makes two blocks for each CU, else smaller ones (a
  // wave's tokens are one chain): 131072 tokens, 256 experts 50 us with 256 chunks, 40 with 512, 51 with 2048,
  // as the joining launch has more to read.  Not where there are many sequences, each with joining blocks of its
  // own (30000 tokens, 256 experts in sequences of 70: 18 us, 66 in two chunks each).
  L.chunk = seq_len < kBalanceChunk ? (seq_len + 7) / 8 * 8 : kBalanceChunk;
  L.cps = 1;
  if (L.by == kByChunk) {
    while (L.chunk > 64 && L.S < 64 && (int64_t)L.S * ((seq_len + L.chunk - 1) / L.chunk) < 512) L.chunk = (L.chunk / 2 + 7) / 8 * 8;
    L.cps = (seq_len + L.chunk - 1) / L.chunk;
  }
  L.eb = (d->E + 31) / 32;
  L.entries = L.S;
  if (L.by != kByChunk) {
    const int per = seq_len <= kBalanceFew ? 4 * (64 / balance_lanes(d->E)) : 4;
    const int blocks = L.S / per + (L.S % per != 0);
    L.entries = blocks < kBalanceShortBlocks ? blocks : kBalanceShortBlocks;
  }
  const size_t chunks = L.cps > 1 ? (size_t)L.S * L.cps : 0;
  size_t off = 0;
  L.part_p = off;   off = align_up(off + chunks * d->E * 4);
  L.part_c = off;   off = align_up(off + chunks * d->E * 4);
  L.part_z = off;   off = align_up(off + chunks * 4);
  L.part_n = off;   off = align_up(off + chunks * 4);
  L.seq_loss = off; off = align_up(off + (size_t)L.entries * (L.cps > 1 ? L.eb : 1) * 4);
  L.seq_z = off;    off = align_up(off + (size_t)L.entries * 4);
  L.seq_n = off;    off = align_up(off + (size_t)L.entries * 4);
  L.seq_some = off; off = align_up(off + (size_t)L.entries * 4);
  L.ticket = off;   off = align_up(off + 4);
  L.total = off;
  return L;
}

template <typename T>
T* ws_at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// ---- update of stacked weights

const float kDefaultCoef[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kDefaultSteps = 5;

int check_stack(int G, int R, int C, int dtype) {
  if (G < 1) return fail(MOE_EINVAL, "G must be >= 1 (got %d)", G);
  if (G > kNewtonMaxStack) return fail(MOE_EUNSUPPORTED, "G must be at most %d (got %d)", kNewtonMaxStack, G);
  if (R < 1 || R > kNewtonMaxDim)
    return fail(MOE_EUNSUPPORTED, "R must be in [1, %d] (got %d)", kNewtonMaxDim, R);
  if (C < 1 || C > kNewtonMaxDim)
    return fail(MOE_EUNSUPPORTED, "C must be in [1, %d] (got %d)", kNewtonMaxDim, C);
  if ((int64_t)R * C > kNewtonMaxMatrix)
    return fail(MOE_EUNSUPPORTED, "R*C must be at most 2^32 (R=%d, C=%d)", R, C);
  if ((double)G * R * C > 549755813888.0)
    return fail(MOE_EUNSUPPORTED, "G*R*C must be at most 2^39 (G=%d, R=%d, C=%d)", G, R, C);
  if ((dtype & ~MOE_EXACT) != MOE_F32 && (dtype & ~MOE_EXACT) != MOE_BF16)
    return fail(MOE_EUNSUPPORTED, "dtype must be MOE_F32 or MOE_BF16, with or without MOE_EXACT (got %d)", dtype);
  return MOE_OK;
}
bool is_bf16(int dtype) { return (dtype & ~MOE_EXACT) == MOE_BF16; }
bool is_exact(int dtype) { return dtype != MOE_BF16; }

// The iteration's coefficients: the caller's, or the default ones in `own`.
int check_newton(const moe_newton* n, moe_newton* own, const moe_newton** out) {
  if (!n) {
    own->steps = kDefaultSteps;
    for (int k = 0; k < kDefaultSteps; ++k)
      for (int i = 0; i < 3; ++i) own->coef[k][i] = kDefaultCoef[i];
    *out = own;
    return MOE_OK;
  }
  if (n->steps < 1 || n->steps > MOE_NEWTON_MAX_STEPS)
    return fail(MOE_EINVAL, "steps must be in [1, %d] (got %d)", MOE_NEWTON_MAX_STEPS, n->steps);
  for (int k = 0; k < n->steps; ++k)
    for (int i = 0; i < 3; ++i)
      if (!(std::fabs(n->coef[k][i]) <= 32.f))
        return fail(MOE_EINVAL, "coefficients must be finite and at most 32 (step %d: %g)", k, (double)n->coef[k][i]);
  *out = n;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(const moe_dims* d, int seq_len) {
  if (check_balance(d, seq_len) != MOE_OK) return 0;
  return balance_layout(d, seq_len).total;
}

int moe_balance(const moe_dims* d, int seq_len, const float* logits, const int32_t* topk_idx,
                const uint8_t* mask, int32_t* counts, int32_t* tokens, float* probs, float* loss,
                void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_balance(d, seq_len));
  MOE_TRY(check_ptr(logits, "logits"));
  MOE_TRY(check_ptr(topk_idx, "topk_idx"));
  MOE_TRY(check_ptr(counts, "counts"));
  MOE_TRY(check_ptr(tokens, "tokens"));
  MOE_TRY(check_ptr(probs, "probs"));
  MOE_TRY(check_ptr(loss, "loss"));
  const BalanceLayout L = balance_layout(d, seq_len);
  MOE_TRY(check_ws_bytes(ws, ws_bytes, L.total));
  BalanceArgs a{};
  a.T = d->T; a.E = d->E; a.K = d->K; a.seq_len = seq_len; a.S = L.S; a.chunk = L.chunk;
  a.cps = L.cps; a.eb = L.eb; a.entries = L.entries;
  a.logits = logits; a.topk_idx = topk_idx; a.mask = mask;
  a.counts = counts; a.tokens = tokens; a.probs = probs; a.loss = loss;
  a.part_p = ws_at<float>(ws, L.part_p);
  a.part_c = ws_at<int32_t>(ws, L.part_c);
  a.part_z = ws_at<float>(ws, L.part_z);
  a.part_n = ws_at<int32_t>(ws, L.part_n);
  a.seq_loss = ws_at<float>(ws, L.seq_loss);
  a.seq_z = ws_at<float>(ws, L.seq_z);
  a.by = L.by;
  a.seq_n = L.by != kByChunk ? ws_at<int32_t>(ws, L.seq_n) : tokens;
  a.seq_some = L.by != kByChunk ? ws_at<int32_t>(ws, L.seq_some) : nullptr;
  a.ticket = ws_at<int32_t>(ws, L.ticket);
  return hip_status(launch_balance(a, as_stream(stream)), "moe_balance");
}

int moe_balance_bwd(const moe_dims* d, int seq_len, const float* logits, const uint8_t* mask,
                    const int32_t* counts, const int32_t* tokens, const float* dloss,
                    const float* dtopk_w, const float* topk_w, const int32_t* topk_idx,
                    float* dlogits, void* stream) {
  MOE_TRY(check_balance(d, seq_len));
  MOE_TRY(check_ptr(logits, "logits"));
  MOE_TRY(check_ptr(counts, "counts"));
  MOE_TRY(check_ptr(tokens, "tokens"));
  MOE_TRY(check_ptr(dloss, "dloss"));
  if (dtopk_w || topk_w || topk_idx) {
    MOE_TRY(check_ptr(dtopk_w, "dtopk_w"));
    MOE_TRY(check_ptr(topk_w, "topk_w"));
    MOE_TRY(check_ptr(topk_idx, "topk_idx"));
  }
  MOE_TRY(check_ptr(dlogits, "dlogits"));
  BalanceBwdArgs a{};
  a.T = d->T; a.E = d->E; a.K = d->K; a.S = sequences(d, seq_len);
  a.seq = DivBy((uint32_t)seq_len);
  a.logits = logits; a.mask = mask; a.counts = counts; a.tokens = tokens; a.dloss = dloss;
  a.dtopk_w = dtopk_w; a.topk_w = topk_w; a.topk_idx = topk_idx; a.dlogits = dlogits;
  return hip_status(launch_balance_bwd(a, as_stream(stream)), "moe_balance_bwd");
}

size_t moe_muon_workspace_bytes(int G, int R, int C, int dtype) {
  if (check_stack(G, R, C, dtype) != MOE_OK) return 0;
  return newton_plan(G, R, C, is_exact(dtype)).total;
}

int moe_orthogonalize(int G, int R, int C, int dtype, const moe_newton* n, const float* g, void* out,
                      void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_stack(G, R, C, dtype));
  moe_newton own;
  MOE_TRY(check_newton(n, &own, &n));
  MOE_TRY(check_ptr(g, "g"));
  MOE_TRY(check_ptr(out, "out"));
  NewtonCall c{};
  c.p = newton_plan(G, R, C, is_exact(dtype));
  MOE_TRY(check_ws_bytes(ws, ws_bytes, c.p.total));
  c.ws = ws;
  c.steps = n->steps;
  c.coef = n->coef;
  c.bf16 = is_bf16(dtype);
  c.g = g;
  c.out = out;
  return hip_status(launch_newton(c, as_stream(stream)), "moe_orthogonalize");
}

int moe_muon(int G, int R, int C, int dtype, const moe_newton* n, const moe_muon_params* p,
             const float* lr, const float* grad, float* mom, float* master, void* w, void* ws,
             size_t ws_bytes, void* stream) {
  MOE_TRY(check_stack(G, R, C, dtype));
  moe_newton own;
  MOE_TRY(check_newton(n, &own, &n));
  if (!p) return fail(MOE_EINVAL, "params is NULL");
  if (reinterpret_cast<uintptr_t>(lr) % 4) return fail(MOE_EINVAL, "lr is not 4-byte aligned");
  MOE_TRY(check_ptr(grad, "grad"));
  MOE_TRY(check_ptr(mom, "mom"));
  MOE_TRY(check_ptr(master, "master"));
  if (is_bf16(dtype)) MOE_TRY(check_ptr(w, "w"));
  else if (w) return fail(MOE_EINVAL, "w must be NULL for MOE_F32: master is the weight itself");
  NewtonCall c{};
  c.p = newton_plan(G, R, C, is_exact(dtype));
  MOE_TRY(check_ws_bytes(ws, ws_bytes, c.p.total));
  c.ws = ws;
  c.steps = n->steps;
  c.coef = n->coef;
  c.bf16 = is_bf16(dtype);
  c.g = grad;
  c.mom = mom;
  c.master = master;
  c.w = static_cast<uint16_t*>(w);
  c.lr_dev = lr;
  c.lr = p->lr;
  c.momentum = p->momentum;
  c.weight_decay = p->weight_decay;
  c.scale = p->scale;
  c.nesterov = p->nesterov != 0;
  return hip_status(launch_newton(c, as_stream(stream)), "moe_muon");
}

}  // extern "C"
