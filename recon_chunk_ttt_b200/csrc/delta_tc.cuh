// Shared pieces of the tensor-core kernels of the gated delta rule
// (kernels_delta_tc.cu, kernels_delta_grad.cu): sequences and chunks, operand
// splitting, warp-level matrix fragments.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "ops_internal.h"
#include "tc_util.cuh"

namespace ttt {
namespace {

constexpr int kC = 64;  // tokens of a chunk
constexpr float kNoBeta = 0x1p-64f;  // what stands for a beta of 0 in the gradient's chains

// The tokens of sequence i, and its first chunk slot: start / kC + i leaves
// room for the chunks of every sequence before it (ceil(len / kC) <= end / kC -
// start / kC + 1) and needs no scan.  Offsets that decrease or leave 0..n are
// cut, so that every slot and row stays inside its array.
struct SeqRange {
  int64_t t0, t1, slot;
  bool bad;
};
__device__ __forceinline__ SeqRange seq_range(const int64_t* offsets, int64_t n, int64_t i) {
  if (offsets == nullptr) return {0, n, 0, false};
  const int64_t a = offsets[i], b = offsets[i + 1];
  SeqRange s;
  s.bad = a < 0 || b < a || b > n;
  s.t0 = a < 0 ? 0 : (a > n ? n : a);
  s.t1 = b < s.t0 ? s.t0 : (b > n ? n : b);
  s.slot = s.t0 / kC + i;
  return s;
}

// The tokens of a chunk slot (len = 0: the slot holds none): the last sequence
// whose first slot is not behind it, found by halving.
struct ChunkRange {
  int64_t t0;
  int len;
  int64_t sequence;  // tokens of the sequence it is of
};
__device__ __forceinline__ ChunkRange chunk_range(const int64_t* offsets, int64_t n, int64_t seqs,
                                                  int64_t slot) {
  int64_t lo = 0, hi = seqs;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (seq_range(offsets, n, mid).slot <= slot)
      lo = mid;
    else
      hi = mid;
  }
  const SeqRange s = seq_range(offsets, n, lo);
  ChunkRange c;
  c.t0 = s.t0 + (slot - s.slot) * kC;
  c.sequence = s.t1 - s.t0;
  c.len = slot < s.slot || c.t0 >= s.t1 ? 0 : s.t1 - c.t0 < kC ? (int)(s.t1 - c.t0) : kC;
  return c;
}

// ---------------------------------------------------------------- fragments
// Byte offset of (row, col) in a tile of 64-value (128-byte) columns blocks of
// `rows` rows each, 16-byte units swizzled by the row: what a TMA load with the
// 128-byte swizzle lays down, and free of bank conflicts for ldmatrix.
__device__ __forceinline__ uint32_t sw(int rows, int row, int col) {
  return (uint32_t)((col >> 6) * rows * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) +
                    (col & 7) * 2);
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 operands, fp32 sums.  c: rows lane/4
// and +8, columns 2 (lane%4) + {0, 1}; a pair of c tiles is laid out like an a
// operand, which lets a product's result be the next one's operand in place.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + mid + lo in bf16: hi and mid are x's upper bits cut off (exact
// remainders), lo the rest rounded: 24 bits, as good as fp32.  Two values, packed.
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
  hi = __byte_perm(xb, yb, 0x7632);
  const float x1 = x - __uint_as_float(xb & 0xffff0000u);
  const float y1 = y - __uint_as_float(yb & 0xffff0000u);
  const uint32_t xc = __float_as_uint(x1), yc = __float_as_uint(y1);
  mid = __byte_perm(xc, yc, 0x7632);
  lo = pack_bf16x2(x1 - __uint_as_float(xc & 0xffff0000u), y1 - __uint_as_float(yc & 0xffff0000u));
}
// The a operand made of two neighbouring c tiles, split.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4],
                                        uint32_t (&hi)[4], uint32_t (&mid)[4], uint32_t (&lo)[4]) {
  split3(c0[0], c0[1], hi[0], mid[0], lo[0]);
  split3(c0[2], c0[3], hi[1], mid[1], lo[1]);
  split3(c1[0], c1[1], hi[2], mid[2], lo[2]);
  split3(c1[2], c1[3], hi[3], mid[3], lo[3]);
}

// An A operand kept in shared memory, 16 bytes a lane.
__device__ __forceinline__ void load_a(const uint4* p, uint32_t (&r)[4]) {
  const uint4 v = *p;
  r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
}
// Mask of a packed pair of tokens t, t + 1 of which those before `valid` count.
__device__ __forceinline__ uint32_t keep_pair(int t, int valid) {
  return t + 1 < valid ? 0xffffffffu : t < valid ? 0xffffu : 0u;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- workspace
// What the chunk kernel leaves for each (slot, head): T as three bf16 parts,
// P (one part for the forward pass, three for the gradient), and the gates
// gamma[64], rest[64], beta[64], each token's.  T and P are lower triangular:
// their 16-column strips hold the rows from the diagonal block down, 32 bytes
// a row, the two 16-byte units exchanged in every second group of four rows
// (free of bank conflicts for ldmatrix, and what a TMA load with the 32-byte
// swizzle lays down).  They are stored as they lie in shared memory, so one
// bulk copy brings the whole block.
constexpr int kTri = 32 * (64 + 48 + 32 + 16);
constexpr int kGates = 1024;
__host__ __device__ constexpr int chunk_bytes(int p_parts) { return (3 + p_parts) * kTri + kGates; }
// (row, 8-value unit) of a tile of 16 columns, 32 bytes a row
__device__ __forceinline__ uint32_t sw32(int row, int unit) {
  return (uint32_t)(row * 32 + ((unit ^ ((row >> 2) & 1)) << 4));
}
// Where row 0 of a triangle's strip k would lie (it begins with row 16 k).
__device__ __forceinline__ uint32_t tri_strip(int k) {
  return (uint32_t)(32 * (64 * k - 8 * k * (k - 1)) - 512 * k);
}
// (row, col) of a triangle, col / 16 <= row / 16
__device__ __forceinline__ uint32_t tri(int row, int col) {
  const int k = col >> 4;
  return (uint32_t)(32 * (64 * k - 8 * k * (k - 1))) + sw32(row - 16 * k, (col >> 3) & 1) +
         (col & 7) * 2;
}

// Running sums G of a chunk's log decays, in fp64 so that differences of far sums stay exact;
// kept as two floats each.  One warp; tokens from `len` on add nothing.
__device__ __forceinline__ void sum_decays(const float* g, int64_t t0, int len, int H, int h,
                                           int lane, float2* G) {
  double x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * lane + i;
    const float v = j < len ? g[(t0 + j) * H + h] : 0.f;
    x[i] = v < -1e4f ? -1e4 : (double)v;  // e^-1e4 is 0 like e^-inf, but its sums are numbers
  }
  double s = x[0] + x[1];
  for (int m = 1; m < 32; m *= 2) {
    const double o = __shfl_up_sync(0xffffffffu, s, m);
    if (lane >= m) s += o;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double v = i == 0 ? s - x[1] : s;
    G[2 * lane + i] = make_float2((float)v, (float)(v - (double)(float)v));
  }
}
// e^(a - b)
__device__ __forceinline__ float decay(float2 a, float2 b) { return expf((a.x - b.x) + (a.y - b.y)); }
__device__ __forceinline__ float decay(float2 a) { return expf(a.x + a.y); }

// Every kAnchor-th chunk the state is kept in fp32: there the gradient of the decays,
// a running sum over tokens, starts anew.
constexpr int kAnchor = 8;

// Stores of accumulators for a later kernel, as bf16 in blocks of 8 x 8 values (8
// rows of 16 bytes: what ldmatrix reads, and a whole line for a warp to write).
// The state [D rows][DK columns from c0]: blocks [column / 16][row / 8][column / 8 % 2].
template <int D, int DK>
__device__ __forceinline__ void keep_state(__nv_bfloat16* to, const float (&s)[DK / 8][4], int r0,
                                           int c0, int lane) {
  uint32_t* w = reinterpret_cast<uint32_t*>(to);
#pragma unroll
  for (int j = 0; j < DK / 8; ++j) {
    const int c = c0 / 8 + j;
    const int block = (c / 2 * (D / 8) + r0 / 8) * 2 + c % 2;
    w[block * 32 + lane] = pack_bf16x2(s[j][0], s[j][1]);
    w[(block + 2) * 32 + lane] = pack_bf16x2(s[j][2], s[j][3]);
  }
}
// The state in fp32, as the registers lie.
template <int N>
__device__ __forceinline__ void keep_anchor(float* to, const float (&s)[N][4], int first,
                                            int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    reinterpret_cast<float4*>(to)[(first + j) * 32 + lane] =
        make_float4(s[j][0], s[j][1], s[j][2], s[j][3]);
}
// Sums over 16 rows of an accumulator times the tile's bf16 values (w0: rows 0-7,
// w1: rows 8-15), of the lane's two tokens; in every lane of the column.
__device__ __forceinline__ float2 rows_sum(float2 x) {
#pragma unroll
  for (int m = 4; m < 32; m *= 2) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
  }
  return x;
}
__device__ __forceinline__ float2 dot_pair(const float (&y)[4], uint32_t w0, uint32_t w1) {
  return rows_sum(make_float2(
      fmaf(y[0], __uint_as_float(w0 << 16), y[2] * __uint_as_float(w1 << 16)),
      fmaf(y[1], __uint_as_float(w0 & 0xffff0000u), y[3] * __uint_as_float(w1 & 0xffff0000u))));
}
__device__ __forceinline__ void put_dots(float* to, float2 x, int t, int valid, int lane) {
  if (lane < 4) {
    if (t + 2 * lane < valid) to[2 * lane] = x.x;
    if (t + 2 * lane + 1 < valid) to[2 * lane + 1] = x.y;
  }
}

inline int64_t chunk_slots(const DeltaArgs& a) { return a.n / kC + a.seqs; }
// In front of the blocks: the sequences' ranking by length, for up to kRanked of
// them (more fill the GPU in any order).
constexpr int kRanked = 512;
constexpr int kOrderBytes = kRanked * 4;
inline size_t blocks_bytes(const DeltaArgs& a, int p_parts) {
  return kOrderBytes + (size_t)chunk_slots(a) * a.H * chunk_bytes(p_parts);
}
inline int32_t* order_of(const DeltaArgs& a, const uint8_t* blocks) {
  if (a.n == 0 || a.seqs < 2 || a.seqs > kRanked) return nullptr;
  return reinterpret_cast<int32_t*>(const_cast<uint8_t*>(blocks) - kOrderBytes);
}

// Token rows as boxes of 64 tokens: all columns of a head, as [d / 64][64][64];
// or 16 columns, as [64][16].
inline bool head_map(CUtensorMap* m, const void* base, int64_t n, int64_t ld, int cols, int d) {
  const uint64_t dims[3] = {64, (uint64_t)n, (uint64_t)cols / 64};
  const uint64_t str[2] = {(uint64_t)ld * 2, 128};
  const uint32_t box[3] = {64, kC, (uint32_t)d / 64};
  return make_map(m, base, 3, dims, str, box);
}
inline bool strip_map(CUtensorMap* m, const void* base, int64_t n, int64_t ld, int cols) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)n};
  const uint64_t str[1] = {(uint64_t)ld * 2};
  const uint32_t box[2] = {16, kC};
  return make_map(m, base, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_32B);
}

}  // namespace

// What the forward pass leaves for the gradient, by chunk slot and head.
struct DeltaKept {
  __nv_bfloat16* S0;  // the state before the chunk
  float* U;           // in fp32, as registers lie: [d / 16][64 / 8][lane] of 4
  float* anchors;     // the state before every kAnchor-th chunk of a sequence
  float* last;        // the last states, or nullptr
  float* dots;        // [d / 16][H][n]: dO . O over 16 columns
};

// Inverses, P and gates of every chunk into `blocks` (kernels_delta_tc.cu).
cudaError_t delta_prepare(const DeltaArgs& a, bool gradient, uint8_t* blocks, cudaStream_t st);

}  // namespace ttt
