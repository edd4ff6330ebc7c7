// Rotary positions over three axes: each pair of a head's values turns by
// position * frequency, (x, y) -> (x cos - y sin, y cos + x sin).
//
// Bound by memory: q and k are read and written once.  The angles depend on
// the token and the pair alone, so a block forms the d/2 sines and cosines of
// each of its tokens once, in shared memory, and all heads of q and k use
// them.  Angles are taken in turns (position * frequency / 2 pi) in fp64 and
// reduced there (t - rint(t)), so far positions keep all of fp32's bits; the
// reduced angle goes through sincospi in fp32.

#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "ops_internal.h"

namespace ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kTok = 8;  // tokens of a block, at most: 8 KB of angles

struct RopeParams {
  double turns[kMaxPairs];   // turns per unit of position, by pair
  unsigned char axis[kMaxPairs];
  const void* X[2];  // q, k
  void* Y[2];
  int64_t ld[2], ldo[2];
  int heads[2];
  const float* pos;
  int64_t n;
  int pairs;  // rotated pairs (R / 2)
  float sign;
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ uint4 pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

__device__ __forceinline__ float2 turn(float2 cs, float x, float y) {
  return make_float2(x * cs.x - y * cs.y, y * cs.x + x * cs.y);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// PAIRS: values 2j, 2j+1; a 16-byte vector holds whole pairs.  Otherwise (HALF)
// a thread takes the vector at j and the one at j + pairs; where the half is
// no multiple of the vector (VEC = false) it takes single values.
template <typename T, int D, bool PAIRS, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p,
                                                        int tok) {
  __shared__ float2 cs[kTok][D / 2];
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int m = p.n - t0 < tok ? (int)(p.n - t0) : tok;
  for (int e = threadIdx.x; e < m * p.pairs; e += kThreads) {
    const int t = e / p.pairs, j = e % p.pairs;
    const double a = (double)p.pos[(t0 + t) * 3 + p.axis[j]] * p.turns[j];
    float s, c;
    sincospif((float)(2.0 * (a - rint(a))), &s, &c);
    cs[t][j] = make_float2(c, p.sign * s);
  }
  __syncthreads();
  constexpr int N = Vec<T>::N;
  const int half = p.pairs;
  // items of a head: PAIRS d/N vectors; HALF half/N pairs of vectors, then the
  // vectors (or single values) that pass
  const int per = PAIRS ? D / N : VEC ? half / N + (D - 2 * half) / N : half + (D - 2 * half);
  const int heads = p.heads[0] + p.heads[1];
  for (int e = threadIdx.x; e < m * heads * per; e += kThreads) {
    const int i = e % per, hh = e / per % heads, t = e / per / heads;
    const int w = hh >= p.heads[0], h = w ? hh - p.heads[0] : hh;
    const T* x = static_cast<const T*>(p.X[w]) + (t0 + t) * p.ld[w] + h * D;
    T* y = static_cast<T*>(p.Y[w]) + (t0 + t) * p.ldo[w] + h * D;
    if (PAIRS) {
      const uint4 in = *reinterpret_cast<const uint4*>(x + i * N);
      float a[N];
      Vec<T>::unpack(in, a);
#pragma unroll
      for (int c = 0; c < N; c += 2)
        if (i * (N / 2) + c / 2 < half) {
          const float2 r = turn(cs[t][i * (N / 2) + c / 2], a[c], a[c + 1]);
          a[c] = r.x, a[c + 1] = r.y;
        }
      *reinterpret_cast<uint4*>(y + i * N) = Vec<T>::pack(a);
    } else if (VEC) {
      if (i < half / N) {
        const uint4 lo = *reinterpret_cast<const uint4*>(x + i * N);
        const uint4 hi = *reinterpret_cast<const uint4*>(x + half + i * N);
        float a[N], b[N];
        Vec<T>::unpack(lo, a);
        Vec<T>::unpack(hi, b);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float2 r = turn(cs[t][i * N + c], a[c], b[c]);
          a[c] = r.x, b[c] = r.y;
        }
        *reinterpret_cast<uint4*>(y + i * N) = Vec<T>::pack(a);
        *reinterpret_cast<uint4*>(y + half + i * N) = Vec<T>::pack(b);
      } else {
        const int c = 2 * half + (i - half / N) * N;
        *reinterpret_cast<uint4*>(y + c) = *reinterpret_cast<const uint4*>(x + c);
      }
    } else {
      if (i < half) {
        const float2 r = turn(cs[t][i], ld1(x + i), ld1(x + half + i));
        st1(y + i, r.x);
        st1(y + half + i, r.y);
      } else {
        y[half + i] = x[half + i];
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch(const RopeParams& p, bool pairs, cudaStream_t st) {
  // tokens of a block: enough values for four vectors a thread, but blocks
  // for the whole GPU first
  const int64_t vecs = (int64_t)(p.heads[0] + p.heads[1]) * D / Vec<T>::N;
  int64_t tok = 4 * kThreads / vecs;
  if (tok > p.n / (148 * 4)) tok = p.n / (148 * 4);
  tok = tok < 1 ? 1 : tok > kTok ? kTok : tok;
  const unsigned grid = (unsigned)((p.n + tok - 1) / tok);
  TraceScope ts("rope", st);
  const bool vec = p.pairs % Vec<T>::N == 0;
  if (pairs)
    rope_kernel<T, D, true, true><<<grid, kThreads, 0, st>>>(p, (int)tok);
  else if (vec)
    rope_kernel<T, D, false, true><<<grid, kThreads, 0, st>>>(p, (int)tok);
  else
    rope_kernel<T, D, false, false><<<grid, kThreads, 0, st>>>(p, (int)tok);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rope(const RopeArgs& a, cudaStream_t st) {
  if (a.n == 0 || a.Hq + a.Hk == 0) return cudaSuccess;
  RopeParams p;
  const int total = a.rot[0] + a.rot[1] + a.rot[2];
  int j = 0;
  for (int x = 0; x < 3; ++x)
    for (int i = 0; i < a.rot[x] / 2; ++i, ++j) {
      const double e = a.head_freq ? 2.0 * j / total : 2.0 * i / a.rot[x];
      p.turns[j] = std::pow((double)a.base[x], -e) / 6.283185307179586476925;
      p.axis[j] = (unsigned char)x;
    }
  p.X[0] = a.Q, p.X[1] = a.K, p.Y[0] = a.Qo, p.Y[1] = a.Ko;
  p.ld[0] = a.ldq, p.ld[1] = a.ldk, p.ldo[0] = a.ldqo, p.ldo[1] = a.ldko;
  p.heads[0] = a.Hq, p.heads[1] = a.Hk;
  p.pos = a.pos;
  p.n = a.n;
  p.pairs = total / 2;
  p.sign = a.inverse ? -1.f : 1.f;
  using B = __nv_bfloat16;
  if (a.bf16)
    return a.d == 64    ? launch<B, 64>(p, a.pairs, st)
           : a.d == 128 ? launch<B, 128>(p, a.pairs, st)
                        : launch<B, 256>(p, a.pairs, st);
  return a.d == 64    ? launch<float, 64>(p, a.pairs, st)
         : a.d == 128 ? launch<float, 128>(p, a.pairs, st)
                      : launch<float, 256>(p, a.pairs, st);
}

}  // namespace ttt
