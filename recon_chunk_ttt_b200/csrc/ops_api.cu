// C-ABI boundary of the operators around the layer (include/ttt.h): the gated
// delta rule, rotary positions and layer norm.  Everything is checked on the
// host before anything is enqueued.

#include <cuda_runtime.h>

#include <cmath>

#include "../../include/ttt.h"
#include "common.cuh"
#include "internal.h"
#include "ops_internal.h"

using ttt::DeltaArgs;
using ttt::NormArgs;
using ttt::RopeArgs;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxSeqs = 65535;  // a launch's third grid axis

ttt_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA; }
cudaStream_t cs(ttt_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool precision_ok(int32_t p) { return p == TTT_PREC_BF16_TC || p == TTT_PREC_FP32_CHECK; }

ttt_status check_delta_cfg(const ttt_delta_config* c) {
  if (c == nullptr) return TTT_ERR_INVALID_ARG;
  if (c->heads < 1 || c->heads > 4096 || c->qk_heads < 1 || c->heads % c->qk_heads != 0)
    return TTT_ERR_INVALID_ARG;
  if (!precision_ok(c->precision) || !std::isfinite(c->scale)) return TTT_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return TTT_ERR_UNSUPPORTED_SHAPE;
  return TTT_OK;
}

// The arguments of a valid config and its tokens; pointers are checked where
// there are tokens.
ttt_status delta_args(const ttt_delta_config* c, const ttt_delta_tokens* t, DeltaArgs* a) {
  const ttt_status s = check_delta_cfg(c);
  if (s != TTT_OK) return s;
  if (t == nullptr || t->n < 0 || t->n > kMaxTokens) return TTT_ERR_INVALID_ARG;
  if (t->seqs < 0 || t->seqs > kMaxSeqs) return TTT_ERR_INVALID_ARG;
  a->H = c->heads;
  a->Hk = c->qk_heads;
  a->d = c->d;
  a->bf16 = c->precision == TTT_PREC_BF16_TC;
  a->scale = c->scale;
  a->Q = t->Q, a->K = t->K, a->V = t->V;
  a->g = t->log_decay, a->b = t->beta;
  a->ldq = t->ldq, a->ldk = t->ldk, a->ldv = t->ldv;
  a->n = t->n;
  a->offsets = t->offsets;
  a->seqs = t->seqs;
  a->brief = -1;
  if (t->n > 0) {
    if (!t->Q || !t->K || !t->V || !t->log_decay || !t->beta) return TTT_ERR_INVALID_ARG;
    const int64_t qk = (int64_t)a->Hk * a->d, v = (int64_t)a->H * a->d;
    if (t->ldq < qk || t->ldk < qk || t->ldv < v) return TTT_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 32;
    if (t->ldq > most || t->ldk > most || t->ldv > most) return TTT_ERR_INVALID_ARG;
    const int64_t unit = a->bf16 ? 8 : 4;
    if (t->ldq % unit || t->ldk % unit || t->ldv % unit) return TTT_ERR_ALIGNMENT;
    if (!aligned(t->Q, 16) || !aligned(t->K, 16) || !aligned(t->V, 16) ||
        !aligned(t->log_decay, 4) || !aligned(t->beta, 4))
      return TTT_ERR_ALIGNMENT;
  }
  return TTT_OK;
}

// The forms over sequences: with no offsets there is one.
ttt_status check_sequences(const DeltaArgs& a) {
  if (a.offsets == nullptr) return a.seqs == 1 ? TTT_OK : TTT_ERR_INVALID_ARG;
  return aligned(a.offsets, 8) ? TTT_OK : TTT_ERR_ALIGNMENT;
}

// Which sequences go in chunks of 64 tokens on the tensor cores (two kernels, and a whole
// chunk's work for any part of one) and which token after token (about 0.6 us a token).
//  - Alone, the two meet at 20 to 24 tokens (16 heads of 128: 14.4 us against 11.1 us for
//    16 tokens, 15.8 us for 24): calls of up to 16 tokens go by token.
//  - Sequences shorter than a chunk on average are mixed, single tokens beside long ones:
//    those of up to 16 tokens go by token, then the others in chunks (256 single tokens
//    and four sequences of 1,000: 254 us; all in chunks 651 us).
//  - Where the average is 4 tokens at most and the call small, all go by token: the longest
//    sequence costs 77 us then, and 17 sequences of 4 tokens take 18 us against 29 us mixed.
constexpr int64_t kBrief = 16, kMixed = 64, kSmall = 128;
bool by_token(const DeltaArgs& a) {
  return !a.bf16 || a.n <= kBrief || (a.n <= 4 * a.seqs && a.n <= kSmall);
}

size_t delta_bytes(const DeltaArgs& a, bool backward) {
  if (backward) return a.bf16 ? ttt::delta_grad_bytes(a) : ttt::delta_tokens_backward_bytes(a);
  return by_token(a) ? 0 : ttt::delta_tc_bytes(a);
}

}  // namespace

extern "C" {

size_t ttt_delta_workspace_bytes(const ttt_delta_config* cfg, int64_t n, int64_t seqs,
                                 int32_t backward) {
  if (check_delta_cfg(cfg) != TTT_OK || n < 0 || n > kMaxTokens || seqs < 0 || seqs > kMaxSeqs)
    return 0;
  DeltaArgs a = {};
  a.H = cfg->heads, a.Hk = cfg->qk_heads, a.d = cfg->d;
  a.bf16 = cfg->precision == TTT_PREC_BF16_TC;
  a.n = n, a.seqs = seqs;
  return delta_bytes(a, backward != 0);
}

ttt_status ttt_delta_chunk(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                           const float* S_in, float* S_out, void* O, void* workspace,
                           size_t workspace_bytes, ttt_stream_t stream) {
  DeltaArgs a;
  ttt_status s = delta_args(cfg, tok, &a);
  if (s != TTT_OK) return s;
  s = check_sequences(a);
  if (s != TTT_OK) return s;
  if (a.n > 0 && !O) return TTT_ERR_INVALID_ARG;
  const void* ptrs[] = {S_in, S_out, O, workspace};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TTT_ERR_ALIGNMENT;
  const size_t need = delta_bytes(a, false);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  if (a.seqs == 0) return TTT_OK;
  if (by_token(a)) return cuda_status(ttt::delta_tokens(a, INT64_MAX, S_in, S_out, O, cs(stream)));
  if (a.offsets != nullptr && a.n <= kMixed * a.seqs) {
    a.brief = kBrief;
    const cudaError_t e = ttt::delta_tokens(a, a.brief, S_in, S_out, O, cs(stream));
    if (e != cudaSuccess) return cuda_status(e);
  }
  return cuda_status(ttt::delta_tc(a, S_in, S_out, O, workspace, cs(stream)));
}

ttt_status ttt_delta_step(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                          const int32_t* slots, int64_t pool, const float* S, float* S_out,
                          void* O, ttt_stream_t stream) {
  DeltaArgs a;
  const ttt_status s = delta_args(cfg, tok, &a);
  if (s != TTT_OK) return s;
  if (a.offsets != nullptr || a.seqs != a.n || pool < 0) return TTT_ERR_INVALID_ARG;
  if (slots == nullptr && pool < a.n) return TTT_ERR_INVALID_ARG;
  if (a.n == 0) return TTT_OK;
  if (!O || (pool > 0 && (!S || !S_out))) return TTT_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(S, 16) || !aligned(S_out, 16) || !aligned(O, 16))
    return TTT_ERR_ALIGNMENT;
  return cuda_status(ttt::delta_step(a, slots, pool, S, S_out, O, cs(stream)));
}

ttt_status ttt_delta_backward(const ttt_delta_config* cfg, const ttt_delta_tokens* tok,
                              const float* S_in, const void* dO, const float* dS_out, void* dQ,
                              void* dK, void* dV, float* dlog_decay, float* dbeta, float* dS_in,
                              void* workspace, size_t workspace_bytes, ttt_stream_t stream) {
  DeltaArgs a;
  ttt_status s = delta_args(cfg, tok, &a);
  if (s != TTT_OK) return s;
  s = check_sequences(a);
  if (s != TTT_OK) return s;
  if (a.n > 0 && (!dO || !dQ || !dK || !dV || !dlog_decay || !dbeta)) return TTT_ERR_INVALID_ARG;
  const void* ptrs[] = {S_in, dO, dS_out, dQ, dK, dV, dS_in, workspace};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TTT_ERR_ALIGNMENT;
  if (!aligned(dlog_decay, 4) || !aligned(dbeta, 4)) return TTT_ERR_ALIGNMENT;
  const size_t need = delta_bytes(a, true);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  if (a.seqs == 0) return TTT_OK;
  if (a.bf16)
    return cuda_status(ttt::delta_grad(a, S_in, dO, dS_out, dQ, dK, dV, dlog_decay, dbeta, dS_in,
                                       workspace, cs(stream)));
  return cuda_status(ttt::delta_tokens_backward(a, S_in, dO, dS_out, dQ, dK, dV, dlog_decay, dbeta,
                                                dS_in, workspace, cs(stream)));
}

ttt_status ttt_rope(const ttt_rope_config* cfg, const void* Q, int64_t ldq, int32_t q_heads,
                    const void* K, int64_t ldk, int32_t k_heads, const float* positions,
                    int64_t n, void* Q_out, int64_t ldq_out, void* K_out, int64_t ldk_out,
                    int32_t inverse, ttt_stream_t stream) {
  if (cfg == nullptr || !precision_ok(cfg->precision)) return TTT_ERR_INVALID_ARG;
  if (cfg->layout != TTT_ROPE_HALF && cfg->layout != TTT_ROPE_PAIRS) return TTT_ERR_INVALID_ARG;
  if (cfg->freq != TTT_ROPE_FREQ_AXIS && cfg->freq != TTT_ROPE_FREQ_HEAD)
    return TTT_ERR_INVALID_ARG;
  if (cfg->d != 64 && cfg->d != 128 && cfg->d != 256) return TTT_ERR_UNSUPPORTED_SHAPE;
  int64_t total = 0;
  for (int x = 0; x < 3; ++x) {
    if (cfg->rot[x] < 0 || cfg->rot[x] % 2 != 0) return TTT_ERR_INVALID_ARG;
    if (!std::isfinite(cfg->base[x]) || !(cfg->base[x] >= 1.f)) return TTT_ERR_INVALID_ARG;
    total += cfg->rot[x];
  }
  if (total < 2 || total > cfg->d) return TTT_ERR_INVALID_ARG;
  if (n < 0 || n > kMaxTokens || q_heads < 1 || q_heads > 4096 || k_heads < 0 || k_heads > 4096)
    return TTT_ERR_INVALID_ARG;
  if (k_heads == 0 && (K || K_out)) return TTT_ERR_INVALID_ARG;
  if (n == 0) return TTT_OK;
  if (!Q || !Q_out || !positions || (k_heads > 0 && (!K || !K_out))) return TTT_ERR_INVALID_ARG;
  const int64_t lq = (int64_t)q_heads * cfg->d, lk = (int64_t)k_heads * cfg->d;
  const int64_t most = (int64_t)1 << 32;
  if (ldq < lq || ldq_out < lq || ldq > most || ldq_out > most) return TTT_ERR_INVALID_ARG;
  if (k_heads > 0 && (ldk < lk || ldk_out < lk || ldk > most || ldk_out > most))
    return TTT_ERR_INVALID_ARG;
  // in place only row on row: any other distance would overwrite rows unread
  if ((Q_out == Q && ldq_out != ldq) || (k_heads > 0 && K_out == K && ldk_out != ldk))
    return TTT_ERR_INVALID_ARG;
  const bool bf16 = cfg->precision == TTT_PREC_BF16_TC;
  const int64_t unit = bf16 ? 8 : 4;
  if (ldq % unit || ldq_out % unit || (k_heads > 0 && (ldk % unit || ldk_out % unit)))
    return TTT_ERR_ALIGNMENT;
  const void* ptrs[] = {Q, K, Q_out, K_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TTT_ERR_ALIGNMENT;
  if (!aligned(positions, 4)) return TTT_ERR_ALIGNMENT;
  RopeArgs a = {};
  a.d = cfg->d;
  for (int x = 0; x < 3; ++x) a.rot[x] = cfg->rot[x], a.base[x] = cfg->base[x];
  a.pairs = cfg->layout == TTT_ROPE_PAIRS;
  a.head_freq = cfg->freq == TTT_ROPE_FREQ_HEAD;
  a.bf16 = bf16;
  a.inverse = inverse != 0;
  a.Q = Q, a.K = K, a.Qo = Q_out, a.Ko = K_out;
  a.ldq = ldq, a.ldk = ldk, a.ldqo = ldq_out, a.ldko = ldk_out;
  a.Hq = q_heads, a.Hk = k_heads;
  a.pos = positions;
  a.n = n;
  return cuda_status(ttt::rope(a, cs(stream)));
}

static ttt_status norm_args(const ttt_norm_config* cfg, int64_t rows, NormArgs* a) {
  if (cfg == nullptr || !precision_ok(cfg->precision)) return TTT_ERR_INVALID_ARG;
  if (!std::isfinite(cfg->eps) || cfg->eps < 0.f) return TTT_ERR_INVALID_ARG;
  if (cfg->dim < 1 || cfg->dim > 65536) return TTT_ERR_UNSUPPORTED_SHAPE;
  if (rows < 0 || rows > kMaxTokens) return TTT_ERR_INVALID_ARG;
  *a = {cfg->dim, rows, cfg->eps, cfg->precision == TTT_PREC_BF16_TC};
  return TTT_OK;
}

size_t ttt_norm_workspace_bytes(const ttt_norm_config* cfg, int64_t rows) {
  NormArgs a;
  if (norm_args(cfg, rows, &a) != TTT_OK) return 0;
  return ttt::norm_workspace_bytes(a);
}

ttt_status ttt_layer_norm(const ttt_norm_config* cfg, const void* X, int64_t ldx, int64_t rows,
                          const float* weight, const float* bias, void* Y, float* stats,
                          ttt_stream_t stream) {
  NormArgs a;
  const ttt_status s = norm_args(cfg, rows, &a);
  if (s != TTT_OK) return s;
  if (rows == 0) return TTT_OK;
  if (!X || !Y || ldx < a.dim || ldx > (int64_t)1 << 32) return TTT_ERR_INVALID_ARG;
  if (Y == X && ldx != a.dim) return TTT_ERR_INVALID_ARG;
  const void* ptrs[] = {X, weight, bias, Y};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TTT_ERR_ALIGNMENT;
  if (!aligned(stats, 4)) return TTT_ERR_ALIGNMENT;
  return cuda_status(ttt::norm_forward(a, X, ldx, weight, bias, Y, stats, cs(stream)));
}

ttt_status ttt_layer_norm_backward(const ttt_norm_config* cfg, const void* X, int64_t ldx,
                                   const void* dY, int64_t lddy, int64_t rows,
                                   const float* weight, const float* stats, void* dX,
                                   float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, ttt_stream_t stream) {
  NormArgs a;
  const ttt_status s = norm_args(cfg, rows, &a);
  if (s != TTT_OK) return s;
  if (!dX && !dweight && !dbias) return TTT_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!X || !dY || !stats) return TTT_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 32;
    if (ldx < a.dim || ldx > most || lddy < a.dim || lddy > most) return TTT_ERR_INVALID_ARG;
    if ((dX == X && ldx != a.dim) || (dX == dY && lddy != a.dim)) return TTT_ERR_INVALID_ARG;
  }
  const void* ptrs[] = {X, dY, weight, dX, dweight, dbias, workspace};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TTT_ERR_ALIGNMENT;
  if (!aligned(stats, 4)) return TTT_ERR_ALIGNMENT;
  if (rows > 0 && (dweight || dbias) &&
      (workspace == nullptr || workspace_bytes < ttt::norm_workspace_bytes(a)))
    return TTT_ERR_WORKSPACE;
  return cuda_status(ttt::norm_backward(a, X, ldx, dY, lddy, weight, stats, dX, dweight, dbias,
                                        workspace, cs(stream)));
}

}  // extern "C"
