// Internal host-side interface of the operators around the layer (delta rule,
// rotary positions, layer norm) between ops_api.cu and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ttt {

// Tokens of the delta rule after validation.
struct DeltaArgs {
  int H, Hk, d;
  bool bf16;
  float scale;
  const void *Q, *K, *V;
  const float *g, *b;  // log decay, beta: [n][H]
  int64_t ldq, ldk, ldv;
  int64_t n;
  const int64_t* offsets;  // [seqs + 1] or nullptr: one sequence of n tokens
  int64_t seqs;
  int64_t brief;  // forward: sequences of at most so many tokens are not taken in chunks
};

// ---- CUDA cores, token by token (kernels_delta.cu) ---------------------------
// The sequences of at most `longest` tokens.
cudaError_t delta_tokens(const DeltaArgs& a, int64_t longest, const float* S_in, float* S_out,
                         void* O, cudaStream_t st);
cudaError_t delta_step(const DeltaArgs& a, const int32_t* slots, int64_t pool, const float* S,
                       float* S_out, void* O, cudaStream_t st);
size_t delta_tokens_backward_bytes(const DeltaArgs& a);
cudaError_t delta_tokens_backward(const DeltaArgs& a, const float* S_in, const void* dO,
                                  const float* dS_out, void* dQ, void* dK, void* dV, float* dg,
                                  float* db, float* dS_in, void* ws, cudaStream_t st);
// out[n][Hk*d] = sum over the H / Hk heads that share a key head, in head order,
// of part[n][H*d] (both dQ and dK: two arrays each).
cudaError_t delta_share(const DeltaArgs& a, const float* part_q, const float* part_k, void* dQ,
                        void* dK, cudaStream_t st);

// ---- tensor cores, chunks of 64 tokens (kernels_delta_tc.cu): bf16 tokens ---------
// The sequences of more than a.brief tokens.
size_t delta_tc_bytes(const DeltaArgs& a);
cudaError_t delta_tc(const DeltaArgs& a, const float* S_in, float* S_out, void* O, void* ws,
                     cudaStream_t st);

// Its gradient (kernels_delta_grad.cu).
size_t delta_grad_bytes(const DeltaArgs& a);
cudaError_t delta_grad(const DeltaArgs& a, const float* S_in, const void* dO, const float* dS_out,
                       void* dQ, void* dK, void* dV, float* dg, float* db, float* dS_in, void* ws,
                       cudaStream_t st);

// ---- rotary positions (kernels_rope.cu) --------------------------------------
struct RopeArgs {
  int d, rot[3];
  float base[3];
  bool pairs, head_freq, bf16, inverse;
  const void *Q, *K;
  void *Qo, *Ko;
  int64_t ldq, ldk, ldqo, ldko;
  int Hq, Hk;
  const float* pos;
  int64_t n;
};
cudaError_t rope(const RopeArgs& a, cudaStream_t st);

// ---- layer norm (kernels_norm.cu) ---------------------------------------------
struct NormArgs {
  int64_t dim, rows;
  float eps;
  bool bf16;
};
size_t norm_workspace_bytes(const NormArgs& a);
cudaError_t norm_forward(const NormArgs& a, const void* X, int64_t ldx, const float* w,
                         const float* b, void* Y, float* stats, cudaStream_t st);
cudaError_t norm_backward(const NormArgs& a, const void* X, int64_t ldx, const void* dY,
                          int64_t lddy, const float* w, const float* stats, void* dX, float* dw,
                          float* db, void* ws, cudaStream_t st);

}  // namespace ttt
