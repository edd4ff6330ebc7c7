// Gated delta rule on CUDA cores, token after token: the one-token form, the
// fp32 check mode, and its gradient.  Per head, S in R^{d x d} (row = output):
//   S' = e^g S,  u = b (v - S' k),  S <- S' + u k^T,  o = scale S q.
// Every row of S goes its own way (row i needs v_i, k, q, g, b alone), so rows
// are spread over the lanes of the whole GPU and stay in registers.

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "ops_internal.h"

namespace ttt {
namespace {

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four consecutive values (16- or 8-byte aligned).
__device__ __forceinline__ void ld4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The tokens of sequence i, and its first slot when every sequence gets one
// slot for each `step` tokens begun: start / step + i leaves room for all
// sequences before it (ceil(len / step) <= end/step - start/step + 1) and
// needs no scan.  Offsets that are no offsets are cut to 0..n and reported.
struct Seq {
  int64_t t0, t1, slot;
};
__device__ __forceinline__ Seq sequence(const int64_t* offsets, int64_t n, int64_t i, int step,
                                        int* err) {
  if (offsets == nullptr) return {0, n, 0};
  const int64_t a = offsets[i], b = offsets[i + 1];
  if (a < 0 || b < a || b > n) atomicExch(err, (int)kErrOffsets);
  Seq s;
  s.t0 = a < 0 ? 0 : (a > n ? n : a);
  s.t1 = b < s.t0 ? s.t0 : (b > n ? n : b);
  s.slot = s.t0 / step + i;
  return s;
}

constexpr int kRows = 4;    // rows of S a group of lanes holds
constexpr int kWarps = 4;
constexpr int kKeep = 16;   // tokens between the states kept for the gradient

struct TokArgs {
  const void *Q, *K, *V;
  const float *g, *b;
  int64_t ldq, ldk, ldv, n;
  const int64_t* offsets;
  const int32_t* slots;
  int64_t pool;
  int H, Hk;
  float scale;
  int* err;
  int64_t longest;  // sequences of more tokens are left alone
};

// grid (d / rows of a block, H, sequences or requests), 128 threads.  A row of
// S lies over LPR lanes, 4 or 8 columns each; a group of LPR lanes holds
// kRows rows, so a step has kRows independent 16-byte loads a lane in flight
// (8 KB a block): one-token calls are bound by the states' traffic, reading
// and writing them once (96 requests, 32 heads of 128: 77 us, 81% of the measured copy
// rate).  S' k and S' q come from the same pass over S (o = scale (S' q + u (k.q))), so a
// token has one reduction over lanes.
// STEP: request i and every later one of the same slot, in order.
// KEEP: the state before every kKeep-th token is written to `keep`.
template <typename T, int D, bool STEP, bool KEEP>
__global__ void __launch_bounds__(32 * kWarps)
    delta_tokens_kernel(TokArgs a, const float* S_in, float* S_out, T* O, float* keep) {
  constexpr int LPR = D == 64 ? 16 : 32, NC = D / LPR / 4, G = 32 / LPR;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % LPR;
  const int r0 = ((blockIdx.x * kWarps + warp) * G + lane / LPR) * kRows;
  const int h = blockIdx.y, hk = h / (a.H / a.Hk);
  const int64_t i = blockIdx.z;
  const size_t DD = (size_t)D * D;

  Seq sq{i, i + 1, 0};
  size_t at = (size_t)i;
  bool live = true;
  if (STEP) {
    if (a.slots != nullptr) {
      const int32_t s = a.slots[i];
      live = s >= 0 && s < a.pool;
      at = live ? (size_t)s : 0;
    }
    if (!live) {  // padding: a row of zeros
      if (l == 0)
        for (int r = 0; r < kRows; ++r) put(O + i * (int64_t)a.H * D + h * D + r0 + r, 0.f);
      return;
    }
  } else {
    sq = sequence(a.offsets, a.n, i, kKeep, a.err);
    if (sq.t1 - sq.t0 > a.longest) return;
  }

  float s[kRows][4 * NC];
  const size_t sbase = (at * a.H + h) * DD + (size_t)r0 * D + l * 4;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (S_in != nullptr)
        ld4(S_in + sbase + (size_t)r * D + c * 4 * LPR, &s[r][4 * c]);
      else
        s[r][4 * c] = s[r][4 * c + 1] = s[r][4 * c + 2] = s[r][4 * c + 3] = 0.f;
    }

  if (STEP && a.slots != nullptr) {  // an earlier request of this slot takes this one with it
    bool seen = false;
    for (int64_t j = lane; j < i; j += 32) seen |= a.slots[j] == (int32_t)at;
    if (__any_sync(0xffffffffu, seen)) return;
  }

  for (int64_t t = sq.t0; STEP || t < sq.t1;) {
    if (KEEP && (t - sq.t0) % kKeep == 0) {
      float* kp = keep + ((sq.slot + (t - sq.t0) / kKeep) * a.H + h) * DD + (size_t)r0 * D + l * 4;
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(kp + (size_t)r * D + c * 4 * LPR) = make_float4(
              s[r][4 * c], s[r][4 * c + 1], s[r][4 * c + 2], s[r][4 * c + 3]);
    }
    float k[4 * NC], q[4 * NC], v[kRows];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      ld4(static_cast<const T*>(a.K) + t * a.ldk + hk * D + c * 4 * LPR + l * 4, &k[4 * c]);
      ld4(static_cast<const T*>(a.Q) + t * a.ldq + hk * D + c * 4 * LPR + l * 4, &q[4 * c]);
    }
    ld4(static_cast<const T*>(a.V) + t * a.ldv + h * D + r0, v);
    const float eg = expf(a.g[t * a.H + h]), b = a.b[t * a.H + h];
    float sk[kRows] = {}, sq_[kRows] = {}, kq = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) {
      kq = fmaf(k[c], q[c], kq);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        s[r][c] *= eg;
        sk[r] = fmaf(s[r][c], k[c], sk[r]);
        sq_[r] = fmaf(s[r][c], q[c], sq_[r]);
      }
    }
#pragma unroll
    for (int m = LPR / 2; m > 0; m /= 2) {
      kq += __shfl_xor_sync(0xffffffffu, kq, m);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        sk[r] += __shfl_xor_sync(0xffffffffu, sk[r], m);
        sq_[r] += __shfl_xor_sync(0xffffffffu, sq_[r], m);
      }
    }
    float o[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float u = b * (v[r] - sk[r]);
      o[r] = a.scale * fmaf(u, kq, sq_[r]);
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) s[r][c] = fmaf(u, k[c], s[r][c]);
    }
    if (O != nullptr && l == 0)
#pragma unroll
      for (int r = 0; r < kRows; ++r) put(O + t * (int64_t)a.H * D + h * D + r0 + r, o[r]);
    if (STEP && a.slots != nullptr) {  // the next request of this slot
      int64_t next = a.n;
      for (int64_t j0 = t + 1; j0 < a.n; j0 += 32) {
        const bool same = j0 + lane < a.n && a.slots[j0 + lane] == (int32_t)at;
        const unsigned m = __ballot_sync(0xffffffffu, same);
        if (m != 0) {
          next = j0 + __ffs(m) - 1;
          break;
        }
      }
      if (next >= a.n) break;
      t = next;
    } else {
      if (STEP) break;
      ++t;
    }
  }
  if (S_out != nullptr)
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4*>(S_out + sbase + (size_t)r * D + c * 4 * LPR) =
            make_float4(s[r][4 * c], s[r][4 * c + 1], s[r][4 * c + 2], s[r][4 * c + 3]);
}

// Gradient, token after token from the last (fp32 check mode; one block a
// sequence and head, its speed is not the point).  With A the gradient of the
// state after token t (dS_out at first) and S' its faded state:
//   A += scale do q^T;  du = A k;  dv = b du;  db = du.(v - S'k);
//   dq = scale S^T do;  dk = A^T u - S'^T dv;  A -= dv k^T;  dg = <A, S'>;  A *= e^g.
// The states come again from those kept every kKeep tokens, one stretch at a
// time (`hist`).  Rows of S and A stay with one warp; sums over rows are taken
// in a warp first, then over the warps in order.
constexpr int kBW = 16;  // warps
template <int D>
__global__ void __launch_bounds__(32 * kBW)
    delta_tokens_backward_kernel(TokArgs a, const float* dO, const float* dS_out, const float* keep,
                                 float* hist, float* A, float* dq_out, float* dk_out, float* dV,
                                 float* dg_out, float* db_out) {
  constexpr int NC = D / 32;
  __shared__ float red[kBW][2][D];
  __shared__ float red2[kBW][2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.x, hk = h / (a.H / a.Hk);
  const int64_t i = blockIdx.y;
  const size_t DD = (size_t)D * D;
  const Seq sq = sequence(a.offsets, a.n, i, kKeep, a.err);
  float* Ah = A + (i * a.H + h) * DD;
  float* hs = hist + (i * a.H + h) * DD * kKeep;
  for (int row = warp; row < D; row += kBW)
    for (int c = 0; c < NC; ++c) {
      const size_t e = (size_t)row * D + c * 32 + lane;
      Ah[e] = dS_out != nullptr ? dS_out[(i * a.H + h) * DD + e] : 0.f;
    }
  const int64_t len = sq.t1 - sq.t0;
  for (int64_t blk = (len + kKeep - 1) / kKeep - 1; blk >= 0; --blk) {
    const int64_t b0 = sq.t0 + blk * kKeep, b1 = b0 + kKeep < sq.t1 ? b0 + kKeep : sq.t1;
    for (int row = warp; row < D; row += kBW) {  // hist[j]: the state before token b0 + j
      float s[NC];
      for (int c = 0; c < NC; ++c)
        s[c] = keep[((sq.slot + blk) * a.H + h) * DD + (size_t)row * D + c * 32 + lane];
      for (int64_t t = b0; t < b1; ++t) {
        const float eg = expf(a.g[t * a.H + h]), b = a.b[t * a.H + h];
        const float* kp = static_cast<const float*>(a.K) + t * a.ldk + hk * D;
        float sk = 0.f;
        for (int c = 0; c < NC; ++c) {
          hs[(t - b0) * DD + (size_t)row * D + c * 32 + lane] = s[c];
          s[c] *= eg;
          sk = fmaf(s[c], kp[c * 32 + lane], sk);
        }
        for (int m = 16; m > 0; m /= 2) sk += __shfl_xor_sync(0xffffffffu, sk, m);
        const float u = b * (static_cast<const float*>(a.V)[t * a.ldv + h * D + row] - sk);
        for (int c = 0; c < NC; ++c) s[c] = fmaf(u, kp[c * 32 + lane], s[c]);
      }
    }
    for (int64_t t = b1 - 1; t >= b0; --t) {
      const float eg = expf(a.g[t * a.H + h]), b = a.b[t * a.H + h];
      float k[NC], q[NC], dq[NC] = {}, dk[NC] = {}, dg = 0.f, db = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        k[c] = static_cast<const float*>(a.K)[t * a.ldk + hk * D + c * 32 + lane];
        q[c] = static_cast<const float*>(a.Q)[t * a.ldq + hk * D + c * 32 + lane];
      }
      for (int row = warp; row < D; row += kBW) {
        const float go = a.scale * dO[t * (int64_t)a.H * D + h * D + row];
        const float v = static_cast<const float*>(a.V)[t * a.ldv + h * D + row];
        float s[NC], A_[NC], du = 0.f, sk = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const size_t e = (size_t)row * D + c * 32 + lane;
          s[c] = eg * hs[(t - b0) * DD + e];
          A_[c] = fmaf(go, q[c], Ah[e]);
          sk = fmaf(s[c], k[c], sk);
          du = fmaf(A_[c], k[c], du);
        }
        for (int m = 16; m > 0; m /= 2) {
          sk += __shfl_xor_sync(0xffffffffu, sk, m);
          du += __shfl_xor_sync(0xffffffffu, du, m);
        }
        const float u = b * (v - sk), dv = b * du;
        if (lane == 0) dV[t * (int64_t)a.H * D + h * D + row] = dv;
        db = fmaf(du, v - sk, db);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          dq[c] = fmaf(go, fmaf(u, k[c], s[c]), dq[c]);
          dk[c] = fmaf(A_[c], u, fmaf(-s[c], dv, dk[c]));
          A_[c] = fmaf(-dv, k[c], A_[c]);
          dg = fmaf(A_[c], s[c], dg);
          Ah[(size_t)row * D + c * 32 + lane] = eg * A_[c];
        }
      }
      for (int m = 16; m > 0; m /= 2) dg += __shfl_xor_sync(0xffffffffu, dg, m);
      __syncthreads();  // the sums of the token before have been read
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        red[warp][0][c * 32 + lane] = dq[c];
        red[warp][1][c * 32 + lane] = dk[c];
      }
      if (lane == 0) red2[warp][0] = dg, red2[warp][1] = db;
      __syncthreads();
      for (int e = threadIdx.x; e < 2 * D; e += 32 * kBW) {
        float x = 0.f;
        for (int w = 0; w < kBW; ++w) x += red[w][e / D][e % D];
        (e < D ? dq_out : dk_out)[t * (int64_t)a.H * D + h * D + e % D] = x;
      }
      if (threadIdx.x < 2) {
        float x = 0.f;
        for (int w = 0; w < kBW; ++w) x += red2[w][threadIdx.x];
        (threadIdx.x == 0 ? dg_out : db_out)[t * a.H + h] = x;
      }
    }
  }
}

// Sum over the heads that share a key head, rounded once.  Rows that belong
// to no sequence are left as they are, as everywhere.
template <typename T>
__global__ void __launch_bounds__(256)
    delta_share_kernel(const float* pq, const float* pk, T* dQ, T* dK, int64_t n, int H, int Hk,
                       int D, const int64_t* offsets, int64_t seqs) {
  const int64_t total = n * Hk * D;
  const int64_t first = offsets == nullptr ? 0 : offsets[0];
  const int64_t last = offsets == nullptr ? n : offsets[seqs];
  const int grp = H / Hk;
  for (int64_t e = (blockIdx.x * (int64_t)256 + threadIdx.x) * 4; e < total;
       e += (int64_t)gridDim.x * 1024) {
    const int64_t t = e / (Hk * D);
    if (t < first || t >= last) continue;
    const int c = (int)(e % (Hk * D)), hk = c / D;
    const size_t src = (size_t)t * H * D + (size_t)hk * grp * D + c % D;
    float x[4] = {}, y[4] = {}, z[4];
    for (int m = 0; m < grp; ++m) {
      ld4(pq + src + (size_t)m * D, z);
#pragma unroll
      for (int w = 0; w < 4; ++w) x[w] += z[w];
      ld4(pk + src + (size_t)m * D, z);
#pragma unroll
      for (int w = 0; w < 4; ++w) y[w] += z[w];
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) put(dQ + e + w, x[w]), put(dK + e + w, y[w]);
  }
}

TokArgs pack(const DeltaArgs& a, int* err) {
  return {a.Q, a.K, a.V, a.g, a.b, a.ldq, a.ldk, a.ldv, a.n, a.offsets, nullptr, 0,
          a.H, a.Hk, a.scale, err, INT64_MAX};
}

// One block's rows of S.
constexpr int block_rows(int d) { return kRows * kWarps * (d == 64 ? 2 : 1); }

template <typename T, int D, bool STEP, bool KEEP>
cudaError_t launch_tokens(const TokArgs& k, int64_t blocks, const float* S_in, float* S_out,
                          void* O, float* keep, cudaStream_t st) {
  const dim3 grid((unsigned)(D / block_rows(D)), (unsigned)k.H, (unsigned)blocks);
  TraceScope ts(STEP ? "delta_step" : "delta_tokens", st);
  delta_tokens_kernel<T, D, STEP, KEEP>
      <<<grid, 32 * kWarps, 0, st>>>(k, S_in, S_out, static_cast<T*>(O), keep);
  return cudaGetLastError();
}

template <bool STEP, bool KEEP>
cudaError_t by_type(const DeltaArgs& a, const TokArgs& k, int64_t blocks, const float* S_in,
                    float* S_out, void* O, float* keep, cudaStream_t st) {
  using B = __nv_bfloat16;
  if constexpr (!KEEP) {  // states are kept for the fp32 gradient alone
    if (a.bf16) {
      if (a.d == 64) return launch_tokens<B, 64, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
      if (a.d == 128) return launch_tokens<B, 128, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
      return launch_tokens<B, 256, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
    }
  }
  if (a.d == 64) return launch_tokens<float, 64, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
  if (a.d == 128) return launch_tokens<float, 128, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
  return launch_tokens<float, 256, STEP, KEEP>(k, blocks, S_in, S_out, O, keep, st);
}

struct BackPlan {
  size_t keep, hist, A, pq, pk, total;  // byte offsets, and the whole
};
BackPlan back_plan(const DeltaArgs& a) {
  const size_t DD = (size_t)a.d * a.d * 4;
  BackPlan p;
  size_t o = 0;
  p.keep = o;
  o += align_up((size_t)(a.n / kKeep + a.seqs) * a.H * DD, 1024);
  p.hist = o;
  o += align_up((size_t)a.seqs * a.H * DD * kKeep, 1024);
  p.A = o;
  o += align_up((size_t)a.seqs * a.H * DD, 1024);
  p.pq = o;
  o += align_up((size_t)a.n * a.H * a.d * 4, 1024);
  p.pk = o;
  o += align_up((size_t)a.n * a.H * a.d * 4, 1024);
  p.total = o;
  return p;
}

template <int D>
cudaError_t launch_backward(const DeltaArgs& a, const TokArgs& k, const void* dO,
                            const float* dS_out, void* dV, float* dg, float* db, char* w,
                            const BackPlan& p, cudaStream_t st) {
  TraceScope ts("delta_tokens_backward", st);
  delta_tokens_backward_kernel<D><<<dim3((unsigned)a.H, (unsigned)a.seqs), 32 * kBW, 0, st>>>(
      k, static_cast<const float*>(dO), dS_out, reinterpret_cast<const float*>(w + p.keep),
      reinterpret_cast<float*>(w + p.hist), reinterpret_cast<float*>(w + p.A),
      reinterpret_cast<float*>(w + p.pq), reinterpret_cast<float*>(w + p.pk), static_cast<float*>(dV),
      dg, db);
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_tokens(const DeltaArgs& a, int64_t longest, const float* S_in, float* S_out,
                         void* O, cudaStream_t st) {
  int* err = device_error_ptr();
  if (err == nullptr) return cudaErrorInvalidDevice;
  TokArgs k = pack(a, err);
  k.longest = longest;
  return by_type<false, false>(a, k, a.seqs, S_in, S_out, O, nullptr, st);
}

cudaError_t delta_step(const DeltaArgs& a, const int32_t* slots, int64_t pool, const float* S,
                       float* S_out, void* O, cudaStream_t st) {
  TokArgs k = pack(a, nullptr);
  k.slots = slots;
  k.pool = pool;
  return by_type<true, false>(a, k, a.n, S, S_out, O, nullptr, st);
}

cudaError_t delta_share(const DeltaArgs& a, const float* pq, const float* pk, void* dQ, void* dK,
                        cudaStream_t st) {
  const int64_t vecs = a.n * a.Hk * a.d / 4;
  const unsigned grid = (unsigned)((vecs + 255) / 256 < 148 * 8 ? (vecs + 255) / 256 : 148 * 8);
  TraceScope ts("delta_share", st);
  if (a.bf16)
    delta_share_kernel<<<grid, 256, 0, st>>>(pq, pk, static_cast<__nv_bfloat16*>(dQ),
                                             static_cast<__nv_bfloat16*>(dK), a.n, a.H, a.Hk, a.d,
                                             a.offsets, a.seqs);
  else
    delta_share_kernel<<<grid, 256, 0, st>>>(pq, pk, static_cast<float*>(dQ),
                                             static_cast<float*>(dK), a.n, a.H, a.Hk, a.d,
                                             a.offsets, a.seqs);
  return cudaGetLastError();
}

size_t delta_tokens_backward_bytes(const DeltaArgs& a) { return back_plan(a).total; }

cudaError_t delta_tokens_backward(const DeltaArgs& a, const float* S_in, const void* dO,
                                  const float* dS_out, void* dQ, void* dK, void* dV, float* dg,
                                  float* db, float* dS_in, void* ws, cudaStream_t st) {
  int* err = device_error_ptr();
  if (err == nullptr) return cudaErrorInvalidDevice;
  const TokArgs k = pack(a, err);
  const BackPlan p = back_plan(a);
  char* w = static_cast<char*>(ws);
  cudaError_t e = by_type<false, true>(a, k, a.seqs, S_in, nullptr, nullptr,
                                       reinterpret_cast<float*>(w + p.keep), st);
  if (e != cudaSuccess) return e;
  e = a.d == 64    ? launch_backward<64>(a, k, dO, dS_out, dV, dg, db, w, p, st)
      : a.d == 128 ? launch_backward<128>(a, k, dO, dS_out, dV, dg, db, w, p, st)
                   : launch_backward<256>(a, k, dO, dS_out, dV, dg, db, w, p, st);
  if (e != cudaSuccess) return e;
  if (dS_in != nullptr) {
    e = cudaMemcpyAsync(dS_in, w + p.A, (size_t)a.seqs * a.H * a.d * a.d * 4,
                        cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
  }
  if (a.n == 0) return cudaSuccess;
  return delta_share(a, reinterpret_cast<const float*>(w + p.pq),
                     reinterpret_cast<const float*>(w + p.pk), dQ, dK, st);
}

}  // namespace ttt
