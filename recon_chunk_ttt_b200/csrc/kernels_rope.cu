// Rotary positions over three axes: each pair of a head's values turns by
// position * frequency, (x, y) -> (x cos - y sin, y cos + x sin).
//
// Bound by memory: q and k are read and written once.  The angles depend on
// the token and the pair alone, so a block forms the sines and cosines of its
// tokens once, in shared memory, and all heads of q and k use them; a thread's
// first loads are on their way meanwhile.  Angles are taken in turns (position
// * frequency / 2 pi) in fixed point: a position is a 24-bit integer times a
// power of two, a frequency 62 bits of a turn; of their product the whole turns
// fall off and the next 32 bits stay (off by 2^-32 + |position| 2^-62 turns at
// most: 1.5e-9 turns up to positions of 2^28).  The angle goes through sincospi in fp32.  (137,400 tokens of
// 10 heads of 128 in bf16, 0.70 GB: 144 us, 76% of the measured copy rate.)

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
  uint64_t turns[kMaxPairs];  // by pair: turns per unit of position * 2^64; the axis in the last 2 bits
  const void* X[2];  // q, k
  void* Y[2];
  int64_t ld[2], ldo[2];
  int heads[2];
  const float* pos;
  int64_t n;
  int pairs;  // rotated pairs (R / 2)
  int per;    // items of a head: what a thread takes at a time
  // 2^32 / x + 1 of per, heads * per (0 where a block has one token), pairs (from 2 on): for e / x
  uint32_t per_inv, row_inv, pair_inv;
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

__device__ __forceinline__ float2 turn(float c, float s, float x, float y) {
  return make_float2(x * c - y * s, y * c + x * s);
}
// N angles' values from shared memory, 16 bytes at a time where there are as many: lanes
// side by side read side by side (cosines and sines interleaved would not).
template <int N>
__device__ __forceinline__ void angles(const float* p, float* x) {
  if (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A value of the parameters by a lane's own index, through its generic address: as a
// constant, 32 indexes would be 32 reads one after another (84% of that unit's time
// before; 194 us against 142 us for 137,400 tokens of 10 heads of 128).
__device__ __forceinline__ uint64_t table(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.u64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}

// position * turns, reduced to [-1/2, 1/2) turns, times 2.
__device__ __forceinline__ float half_turns(float pos, uint64_t turns) {
  const uint32_t bits = __float_as_uint(pos), ex = bits >> 23 & 255;
  if (ex == 255) return __int_as_float(0x7fffffff);  // infinity, NaN
  const uint32_t m = (bits & 0x7fffff) | (ex != 0 ? 0x800000 : 0);
  const int e = (ex != 0 ? (int)ex : 1) - 150;  // |pos| = m 2^e
  // m * turns = (b 2^32 + low) 2^-64 turns
  const uint64_t a = (uint64_t)m * (uint32_t)turns;
  const uint64_t b = (uint64_t)m * (uint32_t)(turns >> 32) + (a >> 32);
  uint32_t f;
  if (e <= 0)
    f = e > -64 ? (uint32_t)(b >> -e) : 0;
  else
    f = e < 64 ? (uint32_t)(((b << 32 | (uint32_t)a) << e) >> 32) : 0;
  if (bits >> 31) f = 0u - f;
  return (float)(int32_t)f * 0x1p-31f;
}

// An item is PAIRS: a 16-byte vector (whole pairs); else (HALF) the vector at j
// and the one at j + pairs, then vectors that pass; where the half is no multiple of
// the vector (VEC = false) the same with single values.
template <typename T, int D, bool PAIRS, bool VEC>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeParams p, int tok) {
  constexpr int N = Vec<T>::N, BATCH = 4;
  __shared__ __align__(16) float cosines[kTok][D / 2], sines[kTok][D / 2];
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int m = p.n - t0 < tok ? (int)(p.n - t0) : tok;
  const int half = p.pairs, row = (p.heads[0] + p.heads[1]) * p.per, total = m * row;

  struct Item {
    int t, i;  // token, item of the head (-1: none)
    const T* x;
    T* y;
    uint4 lo, hi;
  };
  const auto load = [&](Item& it, int e) {
    it.i = -1;
    if (e >= total) return;
    it.t = (int)__umulhi((uint32_t)e, p.row_inv);
    const int f = e - it.t * row;
    int hh = (int)__umulhi((uint32_t)f, p.per_inv);
    it.i = f - hh * p.per;
    const int w = hh >= p.heads[0];
    if (w) hh -= p.heads[0];
    it.x = static_cast<const T*>(w ? p.X[1] : p.X[0]) + (t0 + it.t) * (w ? p.ld[1] : p.ld[0]) + hh * D;
    it.y = static_cast<T*>(w ? p.Y[1] : p.Y[0]) + (t0 + it.t) * (w ? p.ldo[1] : p.ldo[0]) + hh * D;
    if (PAIRS) {
      it.lo = *reinterpret_cast<const uint4*>(it.x + it.i * N);
    } else if (VEC) {
      if (it.i < half / N) {
        it.lo = *reinterpret_cast<const uint4*>(it.x + it.i * N);
        it.hi = *reinterpret_cast<const uint4*>(it.x + half + it.i * N);
      } else {
        it.lo = *reinterpret_cast<const uint4*>(it.x + half + it.i * N);
      }
    }
  };
  const auto finish = [&](const Item& it) {
    if (it.i < 0) return;
    if (PAIRS) {
      float a[N], cs[N / 2], sn[N / 2];
      Vec<T>::unpack(it.lo, a);
      if (it.i * (N / 2) < half) {
        angles<N / 2>(&cosines[it.t][it.i * (N / 2)], cs);
        angles<N / 2>(&sines[it.t][it.i * (N / 2)], sn);
#pragma unroll
        for (int c = 0; c < N / 2; ++c)
          if (it.i * (N / 2) + c < half) {
            const float2 r = turn(cs[c], sn[c], a[2 * c], a[2 * c + 1]);
            a[2 * c] = r.x, a[2 * c + 1] = r.y;
          }
      }
      *reinterpret_cast<uint4*>(it.y + it.i * N) = Vec<T>::pack(a);
    } else if (VEC) {
      if (it.i < half / N) {
        float a[N], b[N], cs[N], sn[N];
        Vec<T>::unpack(it.lo, a);
        Vec<T>::unpack(it.hi, b);
        angles<N>(&cosines[it.t][it.i * N], cs);
        angles<N>(&sines[it.t][it.i * N], sn);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float2 r = turn(cs[c], sn[c], a[c], b[c]);
          a[c] = r.x, b[c] = r.y;
        }
        *reinterpret_cast<uint4*>(it.y + it.i * N) = Vec<T>::pack(a);
        *reinterpret_cast<uint4*>(it.y + half + it.i * N) = Vec<T>::pack(b);
      } else {
        *reinterpret_cast<uint4*>(it.y + half + it.i * N) = it.lo;
      }
    } else if (it.i < half) {
      const float2 r = turn(cosines[it.t][it.i], sines[it.t][it.i], ld1(it.x + it.i),
                            ld1(it.x + half + it.i));
      st1(it.y + it.i, r.x);
      st1(it.y + half + it.i, r.y);
    } else {
      it.y[half + it.i] = it.x[half + it.i];
    }
  };

  Item items[BATCH];
#pragma unroll
  for (int b = 0; b < BATCH; ++b) load(items[b], threadIdx.x + b * kThreads);
  for (int e = threadIdx.x; e < m * half; e += kThreads) {
    // (one pair: its reciprocal does not fit 32 bits)
    const int t = half == 1 ? e : (int)__umulhi((uint32_t)e, p.pair_inv), j = e - t * half;
    float s, c;
    const uint64_t f = table(&p.turns[j]);
    sincospif(half_turns(p.pos[(t0 + t) * 3 + (f & 3)], f), &s, &c);
    cosines[t][j] = c;
    sines[t][j] = p.sign * s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < total; e += BATCH * kThreads) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) finish(items[b]);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) load(items[b], e + (BATCH + b) * kThreads);
  }
}

template <typename T, int D>
cudaError_t launch(RopeParams& p, bool pairs, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const bool vec = p.pairs % N == 0;
  const int unit = pairs || vec ? N : 1;
  p.per = pairs ? D / N : (D - p.pairs) / unit;
  const int64_t row = (int64_t)(p.heads[0] + p.heads[1]) * p.per;
  p.per_inv = (uint32_t)((1ull << 32) / p.per + 1);
  p.pair_inv = p.pairs == 1 ? 0 : (uint32_t)((1ull << 32) / p.pairs + 1);
  // tokens of a block: four items a thread, but blocks for the whole GPU first
  int64_t tok = 4 * kThreads / row;
  if (tok > p.n / (148 * 4)) tok = p.n / (148 * 4);
  tok = tok < 1 ? 1 : tok > kTok ? kTok : tok;
  // Exact: several tokens have e < 2^12 items.  One token may have up to 2^21: e / row is 0,
  // and per <= 255 (d = 256, one pair) keeps the error of e / per below 1 / per.
  p.row_inv = tok == 1 ? 0 : (uint32_t)((1ull << 32) / row + 1);
  const unsigned grid = (unsigned)((p.n + tok - 1) / tok);
  TraceScope ts("rope", st);
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
  for (int x = 0; x < 3; ++x) {
    // a geometric row; with 64 bits of mantissa 128 products keep more than a double has
    if (a.rot[x] == 0) continue;
    const long double size = a.head_freq ? total : a.rot[x];
    const long double ratio = std::pow((long double)a.base[x], -2 / size);
    long double turns = std::pow((long double)a.base[x], a.head_freq ? -2 * j / size : 0) /
                        6.283185307179586476925286766559L;  // base >= 1: less than a sixth of a turn
    for (int i = 0; i < a.rot[x] / 2; ++i, ++j, turns *= ratio)
      p.turns[j] = ((uint64_t)std::ldexp(turns, 62) << 2) | (uint64_t)x;
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
