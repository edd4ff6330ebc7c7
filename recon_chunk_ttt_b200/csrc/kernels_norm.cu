// Layer norm and its gradient.
//   y = (x - mean) rstd w + b;   with xh = (x - mean) rstd, g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx, each once.  A row lies in the registers of a group of threads
// (8 lanes, 1, 4, 8 or 16 warps), so the mean, then the squares about the mean, then
// the result are taken from one read.  In the backward kernel a thread keeps
// its columns' sums of dy and dy xh in registers over all rows of its block;
// the blocks' sums meet in the workspace and a second kernel adds them in
// their order (no atomics).  Of the measured copy rate, bf16 rows of 1,024:
// forward 79%, backward 73% (137,400 rows, 180 us with both kernels); of 4,096 86% and 81%;
// fp32 75 to 100%.
// Rows that are not whole 16-byte vectors go in pairs or one by one: 40 to 62% in bf16, 75 to
// 90% in fp32.  Rows beyond the registers (8,000 of 16,384, backward): 44% in
// bf16, 54% in fp32.

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ops_internal.h"

namespace ttt {
namespace {

template <typename T, int V>
struct Ld;
template <>
struct Ld<float, 4> {
  static __device__ __forceinline__ void get(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  static __device__ __forceinline__ void put(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Ld<float, 1> {
  static __device__ __forceinline__ void put(float* p, const float* x) { *p = x[0]; }
};
template <>
struct Ld<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Ld<__nv_bfloat16, 2> {
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x[0], x[1]);
  }
};
template <>
struct Ld<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    *p = __float2bfloat16_rn(x[0]);
  }
};
// A vector as it lies in memory: what waits in registers for its turn.
template <typename T, int V>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void get(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void none() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float* x) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (V == 8) {
        x[2 * i % V] = __uint_as_float(w[i] << 16);
        x[(2 * i + 1) % V] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void get(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void none() { v = 0; }
  __device__ __forceinline__ void unpack(float* x) const {
    x[0] = __uint_as_float(v << 16), x[1] = __uint_as_float(v & 0xffff0000u);
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void get(const T* p) { v = *p; }
  __device__ __forceinline__ void none() { v = T(0.f); }
  __device__ __forceinline__ void unpack(float* x) const { x[0] = (float)v; }
};
// Two floats that one instruction works on.
struct Two {
  unsigned long long v;
  Two() = default;
  __device__ __forceinline__ Two(float x, float y) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  }
  __device__ __forceinline__ explicit Two(float x) : Two(x, x) {}
  __device__ __forceinline__ float x() const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a;
  }
  __device__ __forceinline__ float y() const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return b;
  }
  __device__ __forceinline__ float sum() const { return x() + y(); }
};
__device__ __forceinline__ Two add(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// The same of one float, where values are loaded one by one.
struct One {
  float v;
  One() = default;
  __device__ __forceinline__ explicit One(float x) : v(x) {}
  __device__ __forceinline__ float x() const { return v; }
  __device__ __forceinline__ float y() const { return 0.f; }
  __device__ __forceinline__ float sum() const { return v; }
};
__device__ __forceinline__ One add(One a, One b) { return One(a.v + b.v); }
__device__ __forceinline__ One mul(One a, One b) { return One(a.v * b.v); }
__device__ __forceinline__ One fma(One a, One b, One c) { return One(fmaf(a.v, b.v, c.v)); }
// Pair c of V values, or the one value.
template <int V>
using Num = std::conditional_t<V == 1, One, Two>;
template <int V>
__device__ __forceinline__ Num<V> pair(const float* x, int c) {
  if constexpr (V == 1)
    return One(x[0]);
  else
    return Two(x[2 * c], x[2 * c + 1]);
}
// w, b: floats, as many as the token vector holds
template <int V>
__device__ __forceinline__ void get_f(const float* p, float* x) {
  if (V == 1) {
    x[0] = *p;
  } else if (V == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[V - 1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) Ld<float, 4>::get(p + i, x + i);
  }
}

// Sum over the G threads of a group (one or more warps of the block), the same
// value in all of them, in a fixed order.  `slot` alternates between sums so
// that one barrier a sum is enough.
template <int G>
__device__ __forceinline__ float group_sum(float x, float* red) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  if (G > 32) {
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w) x += red[w];
  }
  return x;
}

// Threads of a block: 8 rows a block for a warp each, else one row.
constexpr int block_of(int G) { return G <= 32 ? 256 : G; }

// Sums of N values over the G threads of a group at once; one barrier.
constexpr int warps_of(int G) { return G < 32 ? 1 : G / 32; }
// Rows a group takes at once: 32 values a thread; half of that where they are loaded one by
// one (a register each), in the groups whose block has few registers a thread, and where two
// arrays of floats are in flight.  (34,000 rows of 4,096 in bf16, two rows of 256 threads
// instead of one: forward 134 us and 102 us, backward 162 us and 194 us.)
constexpr int rows_at_once(int g, int nv, int v, bool forward, bool floats) {
  const int r = (v == 1 || g > (forward ? 256 : 128) || (!forward && floats) ? 16 : 32) / (nv * v);
  return r < 1 ? 1 : r > 4 ? 4 : r;
}
// Blocks of the backward kernel that an SM holds (128 registers a thread); the grid is
// one wave of them.
constexpr int backward_resident(int G) { return 512 / block_of(G); }
template <int G, int N>
__device__ __forceinline__ void group_sums(float (&x)[N], float (*red)[warps_of(G)]) {
#pragma unroll
  for (int m = (G < 32 ? G : 32) / 2; m > 0; m /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], m);
  if (G > 32) {
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][threadIdx.x / 32] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = 0.f;
#pragma unroll
      for (int w = 0; w < G / 32; ++w) x[i] += red[i][w];
    }
  }
}

// A group takes R rows at a time, whose sums share a barrier; the next R rows are
// loaded meanwhile, and the weight and bias stay in registers.
template <typename T, int V, int G, int NV, int R>
__global__ void __launch_bounds__(block_of(G))
    norm_kernel(const T* X, int64_t ldx, int64_t rows, int dim, float eps,
                const float* __restrict__ w, const float* __restrict__ b, T* Y, float* stats) {
  constexpr int GR = block_of(G) / G;  // groups of a block
  __shared__ float red[2][2][R][warps_of(G)];
  const int l = threadIdx.x % G, nv = dim / V;
  const float inv = 1.f / dim;
  float ww[NV][V], bb[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int c = 0; c < V; ++c) ww[i][c] = 1.f, bb[i][c] = 0.f;
    if (w != nullptr && l + i * G < nv) get_f<V>(w + (l + i * G) * V, ww[i]);
    if (b != nullptr && l + i * G < nv) get_f<V>(b + (l + i * G) * V, bb[i]);
  }
  struct Rows {
    Raw<T, V> x[R][NV];
  };
  const auto load = [&](Rows& n, int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (row + r < rows && l + i * G < nv)
          n.x[r][i].get(X + (row + r) * ldx + (l + i * G) * V);
        else
          n.x[r][i].none();
  };
  const int64_t step = (int64_t)gridDim.x * GR * R;
  int64_t row = ((int64_t)blockIdx.x * GR + threadIdx.x / G) * R;
  Rows now, next;
  load(now, row);
  int turn = 0;
  // the lanes of a warp stay together: groups whose rows have ended go along with nothing
  const int64_t lead = G < 32 ? threadIdx.x % 32 / G * R : 0;
  for (; row - lead < rows; row += step) {
    // in place is in order: Y's rows are this step's, the loads the next one's
    load(next, row + step);
    float mean[R], sq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[V];
        now.x[r][i].unpack(x);
#pragma unroll
        for (int c = 0; c < V; ++c) mean[r] += x[c];  // nothing behind the row's end
      }
    }
    group_sums<G, R>(mean, red[turn][0]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] *= inv;
      sq[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l + i * G < nv) {
          float x[V];
          now.x[r][i].unpack(x);
#pragma unroll
          for (int c = 0; c < V; ++c) sq[r] = fmaf(x[c] - mean[r], x[c] - mean[r], sq[r]);
        }
    }
    group_sums<G, R>(sq, red[turn][1]);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rstd = 1.f / sqrtf(sq[r] * inv + eps);
      if (row + r >= rows) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l + i * G < nv) {
          float x[V];
          now.x[r][i].unpack(x);
#pragma unroll
          for (int c = 0; c < V; ++c) x[c] = fmaf((x[c] - mean[r]) * rstd, ww[i][c], bb[i][c]);
          Ld<T, V>::put(Y + (row + r) * dim + (l + i * G) * V, x);
        }
      if (stats != nullptr && l == 0) stats[2 * (row + r)] = mean[r], stats[2 * (row + r) + 1] = rstd;
    }
    now = next;
  }
}

// Rows wider than the registers of a block: a block of 512 threads reads its row
// three times (from the caches after the first).
template <typename T, int V>
__global__ void __launch_bounds__(512)
    norm_wide_kernel(const T* X, int64_t ldx, int dim, float eps, const float* __restrict__ w,
                     const float* __restrict__ b, T* Y, float* stats) {
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const auto get = [&](int c, float* x) {
    Raw<T, V> r;
    r.get(X + row * ldx + c);
    r.unpack(x);
  };
  float sum = 0.f, sq = 0.f, x[V], ww[V];
#pragma unroll 4
  for (int c = threadIdx.x * V; c < dim; c += 512 * V) {
    get(c, x);
#pragma unroll
    for (int i = 0; i < V; ++i) sum += x[i];
  }
  const float mean = group_sum<512>(sum, red[0]) / dim;
#pragma unroll 4
  for (int c = threadIdx.x * V; c < dim; c += 512 * V) {
    get(c, x);
#pragma unroll
    for (int i = 0; i < V; ++i) sq = fmaf(x[i] - mean, x[i] - mean, sq);
  }
  const float rstd = 1.f / sqrtf(group_sum<512>(sq, red[1]) / dim + eps);
#pragma unroll 2
  for (int c = threadIdx.x * V; c < dim; c += 512 * V) {
    get(c, x);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (x[i] - mean) * rstd;
    if (w != nullptr) {
      get_f<V>(w + c, ww);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] *= ww[i];
    }
    if (b != nullptr) {
      get_f<V>(b + c, ww);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] += ww[i];
    }
    Ld<T, V>::put(Y + row * dim + c, x);
  }
  if (stats != nullptr && threadIdx.x == 0) stats[2 * row] = mean, stats[2 * row + 1] = rstd;
}

// One block's sums over its rows, columns in place: part[2][blocks][dim], dw then db.
// A group takes R rows at a time, whose 2 R sums share a barrier; the next R rows
// are loaded meanwhile.  Rows wait as they lie in memory and are unpacked when
// they are used (twice): registers for rows in flight, not for their conversion.
template <typename T, int V, int G, int NV, int R, bool COLS>
__global__ void __launch_bounds__(block_of(G), backward_resident(G))
    norm_backward_kernel(const T* X, int64_t ldx, const T* dY, int64_t lddy, int64_t rows, int dim,
                         const float* __restrict__ w, const float* __restrict__ stats, T* dX,
                         float* part) {
  constexpr int GR = block_of(G) / G;  // groups of a block
  __shared__ float red[2][2 * R][warps_of(G)];
  extern __shared__ float cols[];  // [GR > 1 ? dim : 0]
  const int l = threadIdx.x % G, nv = dim / V;
  const float inv = 1.f / dim;
  constexpr int P = (V + 1) / 2;  // pairs
  using N = Num<V>;
  N aw[COLS ? NV : 1][P], ab[COLS ? NV : 1][P], ww[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = 1.f;
    if (w != nullptr && l + i * G < nv) get_f<V>(w + (l + i * G) * V, v);
#pragma unroll
    for (int c = 0; c < P; ++c) {
      ww[i][c] = pair<V>(v, c);
      if (COLS) aw[i][c] = ab[i][c] = N(0.f);
    }
  }
  struct Rows {
    Raw<T, V> x[R][NV], g[R][NV];
    float mean[R], rstd[R];
  };
  const auto load = [&](Rows& n, int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row + r < rows;
      n.mean[r] = live ? stats[2 * (row + r)] : 0.f;
      n.rstd[r] = live ? stats[2 * (row + r) + 1] : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live && l + i * G < nv) {
          n.x[r][i].get(X + (row + r) * ldx + (l + i * G) * V);
          n.g[r][i].get(dY + (row + r) * lddy + (l + i * G) * V);
        } else {
          n.x[r][i].none();
          n.g[r][i].none();
        }
    }
  };
  const int64_t step = (int64_t)gridDim.x * GR * R;
  int64_t row = ((int64_t)blockIdx.x * GR + threadIdx.x / G) * R;
  Rows now, next;
  load(now, row);
  int turn = 0;
  // the lanes of a warp stay together: groups whose rows have ended go along with nothing
  const int64_t lead = G < 32 ? threadIdx.x % 32 / G * R : 0;
  for (; row - lead < rows; row += step) {
    // in place is in order: dX's rows are this step's, the loads the next one's
    load(next, row + step);
    // Values go in pairs (one instruction for two where there are two).  With d = x - mean,
    // per row: s1 = sum g w, s2 = sum g w d;  dx = rstd (g w - (rstd s2/n) (d rstd) - s1/n),
    // each factor rstd beside one of the row's size: rstd^3 by itself leaves fp32's range.
    float sums[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const N mean(-now.mean[r]), rstd(now.rstd[r]);
      N s1(0.f), s2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (l + i * G < nv) {
          float xs[V], gs[V];
          now.x[r][i].unpack(xs);
          now.g[r][i].unpack(gs);
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const N d = add(pair<V>(xs, c), mean), g = pair<V>(gs, c);
            if (COLS) {
              aw[i][c] = fma(mul(g, rstd), d, aw[i][c]);
              ab[i][c] = add(ab[i][c], g);
            }
            const N gw = mul(g, ww[i][c]);
            s1 = add(s1, gw);
            s2 = fma(gw, d, s2);
          }
        }
      sums[2 * r] = s1.sum();
      sums[2 * r + 1] = s2.sum();
    }
    if (dX != nullptr) {  // the same for the whole grid
      group_sums<G, 2 * R>(sums, red[turn]);
      turn ^= 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rs = now.rstd[r];
        const N mean(-now.mean[r]), rstd(rs), k1(-(sums[2 * r] * inv)),
            k2(-rs * (sums[2 * r + 1] * inv));
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (row + r < rows && l + i * G < nv) {
            float xs[V], gs[V];
            now.x[r][i].unpack(xs);
            now.g[r][i].unpack(gs);
#pragma unroll
            for (int c = 0; c < P; ++c) {
              const N xh = mul(add(pair<V>(xs, c), mean), rstd);
              const N y = mul(fma(pair<V>(gs, c), ww[i][c], fma(xh, k2, k1)), rstd);
              gs[2 * c] = y.x();
              if (V > 1) gs[(2 * c + 1) % V] = y.y();
            }
            Ld<T, V>::put(dX + (row + r) * dim + (l + i * G) * V, gs);
          }
      }
    }
    now = next;
  }
  if (COLS) {
    float* pw = part + (size_t)blockIdx.x * dim;
    float* pb = pw + (size_t)gridDim.x * dim;
    for (int which = 0; which < 2; ++which) {
      N(&acc)[COLS ? NV : 1][P] = which == 0 ? aw : ab;
      float* out = which == 0 ? pw : pb;
      const auto value = [&](int i, int c) { return c % 2 == 0 ? acc[i][c / 2].x() : acc[i][c / 2].y(); };
      if (GR == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (l + i * G < nv)
#pragma unroll
            for (int c = 0; c < V; ++c) out[(l + i * G) * V + c] = value(i, c);
      } else {  // the block's groups in turn
        for (int r = 0; r < GR; ++r) {
          if ((int)threadIdx.x / G == r)
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (l + i * G < nv)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                  float& z = cols[(l + i * G) * V + c];
                  z = r == 0 ? value(i, c) : z + value(i, c);
                }
          __syncthreads();
        }
        for (int c = threadIdx.x; c < dim; c += block_of(G)) out[c] = cols[c];
        __syncthreads();
      }
    }
  }
}

// dX of wide rows: two reads, the second from the caches.
template <typename T, int V>
__global__ void __launch_bounds__(512)
    norm_backward_wide_kernel(const T* X, int64_t ldx, const T* dY, int64_t lddy, int dim,
                              const float* __restrict__ w, const float* __restrict__ stats, T* dX) {
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const float mean = stats[2 * row], rstd = stats[2 * row + 1];
  const auto get = [&](int c, float* xh, float* g) {  // V normalised values, and dy w
    Raw<T, V> xr, gr;
    xr.get(X + row * ldx + c);
    gr.get(dY + row * lddy + c);
    xr.unpack(xh);
    gr.unpack(g);
    float ww[V];
    if (w != nullptr) get_f<V>(w + c, ww);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xh[i] = (xh[i] - mean) * rstd;
      if (w != nullptr) g[i] *= ww[i];
    }
  };
  float s1 = 0.f, s2 = 0.f, x[V], g[V];
#pragma unroll 2
  for (int c = threadIdx.x * V; c < dim; c += 512 * V) {
    get(c, x, g);
#pragma unroll
    for (int i = 0; i < V; ++i) s1 += g[i], s2 = fmaf(g[i], x[i], s2);
  }
  s1 = group_sum<512>(s1, red[0]) / dim;
  s2 = group_sum<512>(s2, red[1]) / dim;
#pragma unroll 2
  for (int c = threadIdx.x * V; c < dim; c += 512 * V) {
    get(c, x, g);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = rstd * (g[i] - s1 - x[i] * s2);
    Ld<T, V>::put(dX + row * dim + c, g);
  }
}

// Column sums of wide rows: a thread owns V columns, a block a range of rows.
// Runs before dX is written, which may lie over X or dY.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    norm_cols_wide_kernel(const T* X, int64_t ldx, const T* dY, int64_t lddy, int64_t rows,
                          int64_t per, int dim, const float* __restrict__ stats, float* part) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= dim) return;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  float sw[V] = {}, sb[V] = {}, x[V], g[V];
#pragma unroll 4
  for (int64_t row = r0; row < r1; ++row) {
    Raw<T, V> xr, gr;
    xr.get(X + row * ldx + c);
    gr.get(dY + row * lddy + c);
    xr.unpack(x);
    gr.unpack(g);
    const float mean = stats[2 * row], rstd = stats[2 * row + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) sw[i] = fmaf(g[i], (x[i] - mean) * rstd, sw[i]), sb[i] += g[i];
  }
  float* to = part + (size_t)blockIdx.y * dim + c;
#pragma unroll
  for (int i = 0; i < V; ++i) to[i] = sw[i], to[(size_t)gridDim.y * dim + i] = sb[i];
}

// dw, db = the blocks' sums, added in order: 32 columns a block, 32 rows of
// threads take every 32nd block's sum, then their 32 sums in order.
__global__ void __launch_bounds__(1024)
    norm_columns_kernel(const float* __restrict__ part, int blocks, int dim, float* dw, float* db) {
  __shared__ float red[32][33];
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const int x = threadIdx.x % 32, r = threadIdx.x / 32, c = blockIdx.x * 32 + x;
  const float* p = part + (size_t)blockIdx.y * blocks * dim + c;
  float s = 0.f;
  if (c < dim)
#pragma unroll 4
    for (int k = r; k < blocks; k += 32) s += p[(size_t)k * dim];
  red[r][x] = s;
  __syncthreads();
  if (r == 0 && c < dim) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][x];
    out[c] = s;
  }
}

// How a row is laid over threads: G threads, NV vectors of V values each (R rows at
// a time, backward).  G = 0: too wide for registers.
struct Shape {
  int V, G, NV, R;
};
// Values loaded at once: 16 bytes where rows are whole vectors of that and start on them, two
// bf16 values where rows are even, else single ones.
int full_vector(const NormArgs& a) { return a.bf16 ? 8 : 4; }
int vector_of(const NormArgs& a, int64_t ld1, int64_t ld2) {
  const int64_t x = a.dim | ld1 | ld2;  // the pointers are 16-byte aligned, checked at the entry
  return x % full_vector(a) == 0 ? full_vector(a) : a.bf16 && x % 2 == 0 ? 2 : 1;
}
// Vectors a thread may hold: 1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 32.  (Powers of two alone left up to
// half empty: 20,011 rows of 1,153 floats 45 us, so 34 us; backward 72 us and 56 us.)
constexpr int next_nv(int nv) {
  return nv < 6 ? nv + 1 : nv < 8 ? 8 : nv < 12 ? nv + 2 : nv < 16 ? 16 : 32;
}
int nv_at_least(int64_t x) {
  int nv = 1;
  while (nv < x) nv = next_nv(nv);
  return nv;
}
// At most 16 values a thread (32 in the largest group, forward).
Shape shape_of(const NormArgs& a, int V, bool forward) {
  Shape s = {V, 0, 0, 1};
  const int64_t nv = a.dim / s.V;
  const int most = 16 / s.V, last = forward ? 2 * most : most;
  // 8 lanes up to 64 values: a warp would leave three quarters of its lanes without
  s.G = nv <= 8 * (most < 4 ? 1 : 2) && a.dim <= 64 ? 8
        : nv <= 32 * most                          ? 32
        : nv <= 128 * most                         ? 128
        : nv <= 256 * most                         ? 256
        : nv <= 512 * last                         ? 512
                                                   : 0;
  if (s.G == 0) return s;
  s.NV = nv_at_least((nv + s.G - 1) / s.G);
  s.R = rows_at_once(s.G, s.NV, s.V, forward, !a.bf16);
  return s;
}

// Blocks of the kernels (and the rows of the backward kernel's partial sums).
int blocks_of(const NormArgs& a, const Shape& s, bool forward) {
  const int64_t rb = block_of(s.G) / s.G * s.R;
  const int64_t need = (a.rows + rb - 1) / rb;
  const int64_t most =
      148 * (forward ? (s.G == 512 ? 2 : s.G == 128 ? 8 : 4) : backward_resident(s.G));
  return (int)(need < most ? (need < 1 ? 1 : need) : most);
}
int wide_blocks(const NormArgs& a) { return (int)(a.rows < 256 ? (a.rows < 1 ? 1 : a.rows) : 256); }

// The wide kernels' type and vector, as go's arguments.
template <typename F>
void wide_by_type(const NormArgs& a, int V, const F& go) {
  using B = __nv_bfloat16;
  if (a.bf16 && V == 8)
    go(B(), std::integral_constant<int, 8>());
  else if (a.bf16)
    go(B(), std::integral_constant<int, 1>());
  else if (V == 4)
    go(0.f, std::integral_constant<int, 4>());
  else
    go(0.f, std::integral_constant<int, 1>());
}

struct Forward {
  const void* X;
  int64_t ldx;
  const float *w, *b;
  void* Y;
  float* stats;
  int blocks;
};
template <typename T, int V, int G, int NV>
cudaError_t launch_forward(const NormArgs& a, const Forward& f, cudaStream_t st) {
  norm_kernel<T, V, G, NV, rows_at_once(G, NV, V, true, sizeof(T) == 4)><<<f.blocks, block_of(G), 0, st>>>(
      static_cast<const T*>(f.X), f.ldx, a.rows, (int)a.dim, a.eps, f.w, f.b,
      static_cast<T*>(f.Y), f.stats);
  return cudaGetLastError();
}
template <typename T, int V, int G, int MOST, int NV = 1>
cudaError_t forward_by_nv(int nv, const NormArgs& a, const Forward& f, cudaStream_t st) {
  if constexpr (NV < MOST)
    if (nv > NV) return forward_by_nv<T, V, G, MOST, next_nv(NV)>(nv, a, f, st);
  return launch_forward<T, V, G, NV>(a, f, st);
}
template <typename T, int V>
cudaError_t forward_by_g(const Shape& s, const NormArgs& a, const Forward& f, cudaStream_t st) {
  return s.G == 8     ? forward_by_nv<T, V, 8, V == 8 ? 1 : 2>(s.NV, a, f, st)
         : s.G == 32  ? forward_by_nv<T, V, 32, 16 / V>(s.NV, a, f, st)
         : s.G == 128 ? forward_by_nv<T, V, 128, 16 / V>(s.NV, a, f, st)
         : s.G == 256 ? forward_by_nv<T, V, 256, 16 / V>(s.NV, a, f, st)
                      : forward_by_nv<T, V, 512, 32 / V>(s.NV, a, f, st);
}

struct Backward {
  const void* X;
  int64_t ldx;
  const void* dY;
  int64_t lddy;
  const float *w, *stats;
  void* dX;
  float* part;
  int blocks;
};
template <typename T, int V, int G, int NV>
cudaError_t launch_backward(const NormArgs& a, const Backward& b, cudaStream_t st) {
  constexpr int R = rows_at_once(G, NV, V, false, sizeof(T) == 4);
  const auto go = [&](auto kernel, int smem) {
    kernel<<<b.blocks, block_of(G), smem, st>>>(static_cast<const T*>(b.X), b.ldx,
                                                static_cast<const T*>(b.dY), b.lddy, a.rows,
                                                (int)a.dim, b.w, b.stats, static_cast<T*>(b.dX),
                                                b.part);
    return cudaGetLastError();
  };
  if (b.part != nullptr)
    return go(norm_backward_kernel<T, V, G, NV, R, true>, G <= 32 ? (int)a.dim * 4 : 0);
  return go(norm_backward_kernel<T, V, G, NV, R, false>, 0);
}
template <typename T, int V, int G, int MOST, int NV = 1>
cudaError_t backward_by_nv(int nv, const NormArgs& a, const Backward& b, cudaStream_t st) {
  if constexpr (NV < MOST)
    if (nv > NV) return backward_by_nv<T, V, G, MOST, next_nv(NV)>(nv, a, b, st);
  return launch_backward<T, V, G, NV>(a, b, st);
}
template <typename T, int V>
cudaError_t backward_by_g(const Shape& s, const NormArgs& a, const Backward& b, cudaStream_t st) {
  return s.G == 8     ? backward_by_nv<T, V, 8, V == 8 ? 1 : 2>(s.NV, a, b, st)
         : s.G == 32  ? backward_by_nv<T, V, 32, 16 / V>(s.NV, a, b, st)
         : s.G == 128 ? backward_by_nv<T, V, 128, 16 / V>(s.NV, a, b, st)
         : s.G == 256 ? backward_by_nv<T, V, 256, 16 / V>(s.NV, a, b, st)
                      : backward_by_nv<T, V, 512, 16 / V>(s.NV, a, b, st);
}

}  // namespace

size_t norm_workspace_bytes(const NormArgs& a) {
  // the largest of the plans that strides may ask for
  size_t most = (size_t)wide_blocks(a);
  for (int V : {1, 2, full_vector(a)}) {
    if (a.dim % V != 0) continue;
    const Shape s = shape_of(a, V, false);
    if (s.G != 0 && (size_t)blocks_of(a, s, false) > most) most = (size_t)blocks_of(a, s, false);
  }
  return most * 2 * (size_t)a.dim * 4;
}

cudaError_t norm_forward(const NormArgs& a, const void* X, int64_t ldx, const float* w,
                         const float* b, void* Y, float* stats, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const Shape s = shape_of(a, vector_of(a, ldx, a.dim), true);
  TraceScope ts("layer_norm", st);
  if (s.G == 0) {
    const auto go = [&](auto t, auto v) {
      using T = decltype(t);
      norm_wide_kernel<T, decltype(v)::value><<<(unsigned)a.rows, 512, 0, st>>>(
          static_cast<const T*>(X), ldx, (int)a.dim, a.eps, w, b, static_cast<T*>(Y), stats);
    };
    wide_by_type(a, s.V, go);
    return cudaGetLastError();
  }
  const Forward f = {X, ldx, w, b, Y, stats, blocks_of(a, s, true)};
  if (a.bf16)
    return s.V == 8   ? forward_by_g<__nv_bfloat16, 8>(s, a, f, st)
           : s.V == 2 ? forward_by_g<__nv_bfloat16, 2>(s, a, f, st)
                      : forward_by_g<__nv_bfloat16, 1>(s, a, f, st);
  return s.V == 4 ? forward_by_g<float, 4>(s, a, f, st) : forward_by_g<float, 1>(s, a, f, st);
}

cudaError_t norm_backward(const NormArgs& a, const void* X, int64_t ldx, const void* dY,
                          int64_t lddy, const float* w, const float* stats, void* dX, float* dw,
                          float* db, void* ws, cudaStream_t st) {
  const bool cols = dw != nullptr || db != nullptr;
  if (a.rows == 0) {
    cudaError_t e = cudaSuccess;
    if (dw != nullptr) e = cudaMemsetAsync(dw, 0, (size_t)a.dim * 4, st);
    if (e == cudaSuccess && db != nullptr) e = cudaMemsetAsync(db, 0, (size_t)a.dim * 4, st);
    return e;
  }
  const Shape s = shape_of(a, vector_of(a, ldx, lddy), false);
  float* part = cols ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = cudaSuccess;
  int blocks;
  if (s.G == 0) {
    blocks = wide_blocks(a);
    const int64_t per = (a.rows + blocks - 1) / blocks;
    TraceScope ts("layer_norm_backward", st);
    const auto go = [&](auto t, auto v) {
      using T = decltype(t);
      constexpr int V = decltype(v)::value;
      const T *x = static_cast<const T*>(X), *dy = static_cast<const T*>(dY);
      if (cols)
        norm_cols_wide_kernel<T, V>
            <<<dim3((unsigned)((a.dim + 256 * V - 1) / (256 * V)), (unsigned)blocks), 256, 0, st>>>(
                x, ldx, dy, lddy, a.rows, per, (int)a.dim, stats, part);
      if (dX != nullptr)
        norm_backward_wide_kernel<T, V><<<(unsigned)a.rows, 512, 0, st>>>(
            x, ldx, dy, lddy, (int)a.dim, w, stats, static_cast<T*>(dX));
    };
    wide_by_type(a, s.V, go);
    e = cudaGetLastError();
  } else {
    blocks = blocks_of(a, s, false);
    TraceScope ts("layer_norm_backward", st);
    const Backward b = {X, ldx, dY, lddy, w, stats, dX, part, blocks};
    if (a.bf16)
      e = s.V == 8   ? backward_by_g<__nv_bfloat16, 8>(s, a, b, st)
          : s.V == 2 ? backward_by_g<__nv_bfloat16, 2>(s, a, b, st)
                     : backward_by_g<__nv_bfloat16, 1>(s, a, b, st);
    else
      e = s.V == 4 ? backward_by_g<float, 4>(s, a, b, st) : backward_by_g<float, 1>(s, a, b, st);
  }
  if (e != cudaSuccess || !cols) return e;
  TraceScope ts("layer_norm_columns", st);
  norm_columns_kernel<<<dim3((unsigned)((a.dim + 31) / 32), 2), 1024, 0, st>>>(part, blocks,
                                                                              (int)a.dim, dw, db);
  return cudaGetLastError();
}

}  // namespace ttt
