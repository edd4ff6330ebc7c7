// Gated delta rule in chunks of 64 tokens on the tensor cores.
//
// Inside a chunk, with G the running sum of the log decays, gamma = e^G,
// Gamma_ij = e^(G_i - G_j) and S the state before the chunk (rows = outputs):
//   (I + L) U = beta (V - gamma K S^T),  L = strictly lower part of beta Gamma (K K^T)
//   O = scale gamma (Q S^T) + P U,       P = lower part of scale Gamma (Q K^T)
//   S <- gamma_64 S + U^T (rest K),      rest_j = e^(G_64 - G_j)
// T = (I + L)^-1 and P need no state: delta_chunk_kernel forms them for all
// chunks at once.  What is left is a chain over the chunks of a sequence, and
// delta_state_chain (delta_state.cuh) makes its step short.
//
// Bound by that chain, not by memory or by the tensor cores: a step of 64 tokens takes
// 3.0 us at d = 256 (2.7 us at 128), of which the products are 1.2 us; the rest is the
// latency of one product's result on its way to be the next one's operand.  (137,400
// tokens, 4 heads of 256: 2,147 steps, 6.4 ms; the bytes alone would be 0.18 ms.)

#include "delta_state.cuh"

namespace ttt {
namespace {

// ----------------------------------------------------------------------------
// delta_chunk_kernel: T, P and the gates of one chunk and head.  The inverse is fp32 on
// CUDA cores (its entries multiply up, so L's rounding would too).  Bound by its own
// instructions and shared memory, about a third in the decays and triangles, a fifth each
// in the substitution and the two products: 95 us for 4,320 chunks and heads of d = 128
// (0.15 GB, 23 us); it is 4% of a long sequence's time and a fifth of a packed batch's.
// ----------------------------------------------------------------------------
constexpr int kChunkThreads = 128;
constexpr int kLS = 36;  // row length of the 32 x 32 fp32 blocks: 16-byte rows, spread over banks

struct ChunkArgs {
  const __nv_bfloat16 *Q, *K;
  const float *g, *b;
  int64_t ldq, ldk, n;
  const int64_t* offsets;
  int64_t seqs;
  int H, Hk;
  float scale;
  uint8_t* blocks;
  int64_t slots;
  int64_t brief;   // chunks of sequences of at most so many tokens are left out
  int32_t* order;  // written where it is not nullptr
};

// The sequences from the longest to the shortest, equal ones as they come: a chain's
// time is its length, so the longest has to start first (16,411 tokens in 13 sequences, the
// longest last, 16 heads of 128: 602 us as they come, 512 us from the longest).
__device__ __forceinline__ void rank_sequences(const ChunkArgs& a, int64_t* len, int tid) {
  for (int i = tid; i < a.seqs; i += kChunkThreads) {
    const SeqRange s = seq_range(a.offsets, a.n, i);
    len[i] = s.t1 - s.t0;
  }
  __syncthreads();
  for (int i = tid; i < a.seqs; i += kChunkThreads) {
    int rank = 0;
    for (int j = 0; j < a.seqs; ++j) rank += len[j] > len[i] || (len[j] == len[i] && j < i);
    a.order[rank] = i;
  }
}

template <int D, bool GRAD>
// (five blocks an SM, for d = 256 the three that its tiles allow: 95 us against 100 us for four)
__global__ void __launch_bounds__(kChunkThreads, D == 256 ? 0 : 5)
    delta_chunk_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *sK = smem, *sQ = smem + kC * D * 2;
  // fp32 blocks over the tiles once the products are taken: L21, and the
  // transposes of L11, L22; T11, T22, L21 T11, T21
  float* fb = reinterpret_cast<float*>(smem);
  __shared__ float2 G[kC];
  __shared__ float beta[kC];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t slot = blockIdx.x;
  const int h = blockIdx.y, hk = h / (a.H / a.Hk);
  if (slot == a.slots) {  // one block more: it ranks the sequences
    if (h == 0) rank_sequences(a, reinterpret_cast<int64_t*>(smem_raw), tid);
    return;
  }
  const ChunkRange c = chunk_range(a.offsets, a.n, a.seqs, slot);
  if (c.len == 0 || c.sequence <= a.brief) return;

  for (int e = tid; e < kC * D / 8; e += kChunkThreads) {
    const int row = e / (D / 8), col = e % (D / 8) * 8;
    const bool ok = row < c.len;
    const int64_t t = c.t0 + (ok ? row : 0);
    cp16(smem_u32(sK) + sw(kC, row, col), a.K + t * a.ldk + hk * D + col, ok);
    cp16(smem_u32(sQ) + sw(kC, row, col), a.Q + t * a.ldq + hk * D + col, ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (warp == 0) {
    sum_decays(a.g, c.t0, c.len, a.H, h, lane, G);
  } else if (warp == 1) {
    for (int j = lane; j < kC; j += 32) {
      float b = j < c.len ? a.b[(c.t0 + j) * a.H + h] : 0.f;
      // The gradient divides U by beta.  A beta of nothing becomes 2^-64: the
      // token's U is then that small (its part in any sum rounds away), but
      // U / beta has all its digits.
      if (GRAD && j < c.len && fabsf(b) <= kNoBeta) b = kNoBeta;
      beta[j] = b;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // K K^T and Q K^T: a warp takes 16 rows, up to the diagonal
  float kk[8][4] = {}, qk[8][4] = {};
  const int m0 = warp * 16;
  for (int k = 0; k < D / 16; ++k) {
    uint32_t ak[4], aq[4], b[4];
    const int ar = m0 + (lane % 16), ac = k * 16 + (lane / 16) * 8;
    ldsm4(smem_u32(sK) + sw(kC, ar, ac), ak);
    ldsm4(smem_u32(sQ) + sw(kC, ar, ac), aq);
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if (p <= warp) {
        ldsm4(smem_u32(sK) + sw(kC, p * 16 + (lane / 16) * 8 + lane % 8,
                                k * 16 + (lane / 8 % 2) * 8), b);
        mma(kk[2 * p], ak, b[0], b[1]);
        mma(kk[2 * p + 1], ak, b[2], b[3]);
        mma(qk[2 * p], aq, b[0], b[1]);
        mma(qk[2 * p + 1], aq, b[2], b[3]);
      }
  }
  __syncthreads();  // the tiles are free

  uint8_t* out = a.blocks + (slot * a.H + h) * (int64_t)chunk_bytes(GRAD ? 3 : 1);
  uint8_t* outP = out + 3 * kTri;
  float *L21 = fb, *Lt1 = fb + 32 * kLS, *Lt2 = fb + 2 * 32 * kLS, *T1 = fb + 3 * 32 * kLS,
        *T2 = fb + 4 * 32 * kLS, *Z = fb + 5 * 32 * kLS;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    if (nt > 2 * warp + 1) break;  // above the diagonal
    const int j = nt * 8 + 2 * (lane % 4);
    const float2 Gj[2] = {G[j], G[j + 1]};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = m0 + lane / 4 + 8 * half;
      const float2 Gi = G[i];
      const float b = beta[i];
      float p[2], l[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float e = j + x <= i ? decay(Gi, Gj[x]) : 0.f;
        p[x] = j + x <= i ? a.scale * e * qk[nt][2 * half + x] : 0.f;
        l[x] = j + x < i ? b * e * kk[nt][2 * half + x] : 0.f;
      }
      if (nt < 4 && warp >= 2) {
        *reinterpret_cast<float2*>(L21 + (i - 32) * kLS + j) = make_float2(l[0], l[1]);
      } else {
        float* to = nt < 4 ? Lt1 + j * kLS + i : Lt2 + (j - 32) * kLS + i - 32;
        to[0] = l[0], to[kLS] = l[1];
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(outP + tri(i, j));
      if (GRAD) {
        uint32_t hi, mid, lo;
        split3(p[0], p[1], hi, mid, lo);
        dst[0] = hi;
        dst[kTri / 4] = mid;
        dst[2 * kTri / 4] = lo;
      } else {
        dst[0] = pack_bf16x2(p[0], p[1]);
      }
    }
  }
  __syncthreads();

  // (I + L)^-1 by halves: the two diagonal blocks by substitution (a thread
  // holds a column), then T21 = -T22 L21 T11.
  if (warp < 2) {
    const float* Lt = warp == 0 ? Lt1 : Lt2;
    float* T = warp == 0 ? T1 : T2;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < 31; ++k)
#pragma unroll
      for (int i4 = (k + 1) / 4; i4 < 8; ++i4) {
        const float4 l = *reinterpret_cast<const float4*>(Lt + k * kLS + i4 * 4);
        const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (i4 * 4 + q > k) x[i4 * 4 + q] = fmaf(-lv[q], x[k], x[i4 * 4 + q]);
      }
#pragma unroll
    for (int i = 0; i < 32; ++i) T[i * kLS + lane] = x[i];
  } else if (warp == 2) {  // gates
    float* gates = reinterpret_cast<float*>(out + (3 + (GRAD ? 3 : 1)) * kTri);
    for (int j = lane; j < kC; j += 32) {
      gates[j] = decay(G[j]);
      gates[kC + j] = decay(G[kC - 1], G[j]);
      gates[2 * kC + j] = beta[j];
    }
  }
  __syncthreads();
  // a thread takes two rows of 4 columns
  const auto product = [&](const float* x, const float* y, float* to, float sign) {
    const int i = tid / 8 * 2, j = tid % 8 * 4;
    float z[2][4] = {};
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float xv[2][4], yv[4][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4*>(xv[q]) = *reinterpret_cast<const float4*>(x + (i + q) * kLS + k);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(yv[q]) = *reinterpret_cast<const float4*>(y + (k + q) * kLS + j);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int w = 0; w < 4; ++w) z[p][w] = fmaf(xv[p][q], yv[q][w], z[p][w]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *reinterpret_cast<float4*>(to + (i + p) * kLS + j) =
          make_float4(sign * z[p][0], sign * z[p][1], sign * z[p][2], sign * z[p][3]);
  };
  product(L21, T1, Z, 1.f);
  __syncthreads();
  product(T2, Z, L21, -1.f);  // T21
  __syncthreads();
  // rows r and r + 32 of T, 8 columns of each half, as 16-byte units
  const int r = tid / 4, cb = tid % 4 * 8;
  const float* src[3] = {T1 + r * kLS + cb, L21 + r * kLS + cb, T2 + r * kLS + cb};
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int i = r + (q > 0 ? 32 : 0), j = cb + (q == 2 ? 32 : 0);
    if (j / 16 > i / 16) continue;
    uint32_t w[3][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      split3(src[q][2 * x], src[q][2 * x + 1], w[0][x], w[1][x], w[2][x]);
#pragma unroll
    for (int x = 0; x < 3; ++x)
      *reinterpret_cast<uint4*>(out + x * kTri + tri(i, j)) =
          make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
  }
}

// ----------------------------------------------------------------------------
template <int D, int KS, int RG, int ST>
__global__ void __launch_bounds__(SK<D, KS, RG, ST, false>::THREADS, ST == 1 ? 2 : 1)
    delta_state_kernel(const __grid_constant__ CUtensorMap mQ,
                       const __grid_constant__ CUtensorMap mK,
                       const __grid_constant__ CUtensorMap mV, const __grid_constant__ StateArgs a) {
  extern __shared__ uint8_t smem_raw[];
  delta_state_chain<D, KS, RG, ST, false>(mQ, mK, mV, mV, a, smem_raw, blockIdx.x, blockIdx.y,
                                          blockIdx.z);
}

template <int D, bool GRAD>
cudaError_t launch_chunks(const DeltaArgs& a, uint8_t* blocks, cudaStream_t st) {
  const int need = 2 * kC * D * 2, fp = 6 * 32 * kLS * 4;
  const int smem = (need > fp ? need : fp) + 1024;
  const cudaError_t e = ensure_smem_attr(delta_chunk_kernel<D, GRAD>, smem);
  if (e != cudaSuccess) return e;
  const ChunkArgs k = {static_cast<const __nv_bfloat16*>(a.Q), static_cast<const __nv_bfloat16*>(a.K),
                       a.g, a.b, a.ldq, a.ldk, a.n, a.offsets, a.seqs, a.H, a.Hk, a.scale, blocks,
                       chunk_slots(a), a.brief, order_of(a, blocks)};
  TraceScope ts("delta_chunk", st);
  delta_chunk_kernel<D, GRAD>
      <<<dim3((unsigned)(chunk_slots(a) + (k.order != nullptr)), (unsigned)a.H), kChunkThreads, smem,
         st>>>(k);
  return cudaGetLastError();
}

template <int D, int KS, int RG, int ST>
cudaError_t launch_state(const DeltaArgs& a, const float* S_in, float* S_out, void* O,
                         const uint8_t* blocks, cudaStream_t st) {
  using L = SK<D, KS, RG, ST, false>;
  int* err = device_error_ptr();
  if (err == nullptr) return cudaErrorInvalidDevice;
  CUtensorMap mQ, mK, mV;
  if (!head_map(&mQ, a.Q, a.n, a.ldq, a.Hk * D, D) || !head_map(&mK, a.K, a.n, a.ldk, a.Hk * D, D) ||
      !strip_map(&mV, a.V, a.n, a.ldv, a.H * D))
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_attr(delta_state_kernel<D, KS, RG, ST>, L::SMEM);
  if (e != cudaSuccess) return e;
  const StateArgs k = {a.n,   a.offsets, a.H, a.Hk, a.scale, blocks, order_of(a, blocks), S_in,
                       S_out, static_cast<__nv_bfloat16*>(O), a.brief, DeltaKept{}, err};
  // no more sequences than this have more than a.brief tokens, and they come first
  const int64_t most = k.order == nullptr || a.brief < 0 ? a.seqs : a.n / (a.brief + 1);
  const unsigned seqs = (unsigned)(most < a.seqs ? most : a.seqs);
  TraceScope ts("delta_state", st);
  delta_state_kernel<D, KS, RG, ST><<<dim3(D / (16 * RG), (unsigned)a.H, seqs), L::THREADS, L::SMEM,
                                      st>>>(mQ, mK, mV, k);
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_prepare(const DeltaArgs& a, bool gradient, uint8_t* blocks, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  if (gradient)
    return a.d == 64    ? launch_chunks<64, true>(a, blocks, st)
           : a.d == 128 ? launch_chunks<128, true>(a, blocks, st)
                        : launch_chunks<256, true>(a, blocks, st);
  return a.d == 64    ? launch_chunks<64, false>(a, blocks, st)
         : a.d == 128 ? launch_chunks<128, false>(a, blocks, st)
                      : launch_chunks<256, false>(a, blocks, st);
}

size_t delta_tc_bytes(const DeltaArgs& a) { return blocks_bytes(a, 1); }

cudaError_t delta_tc(const DeltaArgs& a, const float* S_in, float* S_out, void* O, void* ws,
                     cudaStream_t st) {
  uint8_t* blocks = static_cast<uint8_t*>(ws) + kOrderBytes;
  const cudaError_t e = delta_prepare(a, false, blocks, st);
  if (e != cudaSuccess) return e;
  // Groups of 16 rows of S.  Where there are no more of them than SMs, four warps share each,
  // one on each quarter of an SM (1,374 tokens, 4 heads of 128: 60 us against 95 us); else two
  // do, with half the exchange for each product, and four groups share an SM (16,411 tokens in
  // 13 sequences, 16 heads of 128: 511 us against 551 us; 14,000 tokens in 20 sequences, 16
  // heads of 64: 142 us against 220 us).
  const bool few = a.seqs * a.H * (a.d / 16) <= num_sms();
  if (a.d == 64)
    return few ? launch_state<64, 4, 1, 2>(a, S_in, S_out, O, blocks, st)
               : launch_state<64, 2, 2, 1>(a, S_in, S_out, O, blocks, st);
  if (a.d == 128)
    return few ? launch_state<128, 4, 1, 2>(a, S_in, S_out, O, blocks, st)
               : launch_state<128, 2, 2, 1>(a, S_in, S_out, O, blocks, st);
  return launch_state<256, 4, 1, 2>(a, S_in, S_out, O, blocks, st);
}

}  // namespace ttt
