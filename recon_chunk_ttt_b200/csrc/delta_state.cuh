// The forward chain of the gated delta rule on the tensor cores (the formulas are in
// kernels_delta_tc.cu): for the forward pass, and run once more for the gradient.
#pragma once

#include <type_traits>

#include "delta_tc.cuh"

namespace ttt {
namespace {

// ----------------------------------------------------------------------------
// The chain over a sequence's chunks: one block's part.
//
// It works on the transposes: a group of KS warps owns 16 rows of S in registers, D / KS
// columns each, as accumulators, whose layout is that of an A operand; rows of S never
// meet, so blocks do not either.  A step: every warp forms its columns' share of S K^T and
// S Q^T; the shares are added through shared memory, each warp takes its share of the
// tokens through r = beta (v - ..), u = r T^T and o, and gets the others' u for its columns
// of S: three meetings, by mbarrier, within a group.  (tcgen05 takes 64 or 128 rows: too
// few blocks for the GPU, and every intermediate would go from tensor memory through
// registers to shared memory and back, three times a step, on the path that nothing
// overlaps.)  K, Q, V tiles come by TMA and T, P, gates by one bulk copy, ST chunks deep.
//
// The state is fp32 in and out, so operands that are not bf16 by nature (S, T, r, u) enter
// as three bf16 parts, of whose products those above 2^-24 are taken: S K^T and U^T K three
// each (K is exact), T six.  O is rounded to bf16 in the end: two parts of S and U, one of
// P (2^-9, a bf16 operand's rounding, next to O's own); for the gradient, whose decays take
// dO . O in fp32, all three.
// The tensor cores cut an accumulator's last bits off with every product they
// add to it (measured: 1 + 0.75 ulp stays 1), so small parts are summed apart
// from large ones, and the state takes one fp32 addition a chunk.
// ----------------------------------------------------------------------------
template <int D, int KS, int RG, int ST, bool GRAD>
struct SK {
  static constexpr int WARPS = KS * RG;
  static constexpr int KQ = kC * D * 2;               // one of K, Q
  static constexpr int BLOCK = chunk_bytes(GRAD ? 3 : 1);
  static constexpr int V = kC * 32;                   // 16 columns of V (or dO)
  static constexpr int STAGE = KQ + (GRAD ? 2 : 1) * RG * V + BLOCK;
  // exchange of a group: partial r, partial o (each warp's for the others'
  // tiles), r in parts, u in parts
  static constexpr int U_PARTS = GRAD ? 6 : 5;
  static constexpr int X_PART = 8 * (KS - 1) * 32 * 16, X_R = 8 * 3 * 32 * 8,
                       X_U = 8 * U_PARTS * 32 * 8;
  static constexpr int X = 2 * X_PART + X_R + X_U;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int OFF_Q = ST * STAGE;             // Q is free again early in a step: one stage
  static constexpr int OFF_X = OFF_Q + KQ;
  static constexpr int OFF_BAR = OFF_X + RG * X;
  static constexpr int SMEM = OFF_BAR + 192 + 1024;
  static_assert((KS == 2 || KS == 4) && RG <= 2, "tiles and barriers of a group");
  static_assert(STAGE % 1024 == 0, "tiles are aligned to the swizzle");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct StateArgs {
  int64_t n;
  const int64_t* offsets;
  int H, Hk;
  float scale;
  const uint8_t* blocks;
  const int32_t* order;  // sequences from the longest, or nullptr: as they come
  const float* S_in;
  float* S_out;
  __nv_bfloat16* O;
  int64_t brief;   // sequences of at most so many tokens are left alone
  DeltaKept kept;  // for the gradient
  int* err;
};

// Block x of (rows, head, sequence); GRAD: the chain is run for the gradient, which finds
// what it needs in a.kept.
template <int D, int KS, int RG, int ST, bool GRAD>
__device__ __forceinline__ void delta_state_chain(const CUtensorMap& mQ, const CUtensorMap& mK,
                                                  const CUtensorMap& mV, const CUtensorMap& mG,
                                                  const StateArgs& a, uint8_t* smem_raw, int bx,
                                                  int h, int64_t rank) {
  using L = SK<D, KS, RG, ST, GRAD>;
  constexpr int DK = D / KS, NT = 8 / KS;  // a warp's columns of S; its token tiles of r, u, o
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + 2;
  uint64_t* qfull = empty + 2;
  uint64_t* qempty = qfull + 1;
  uint64_t* met = qempty + 1;  // 3 for each group: partial sums, r, u are written
  volatile int* abort_flag = reinterpret_cast<volatile int*>(met + 3 * RG);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = h / (a.H / a.Hk);
  const int64_t seq = a.order != nullptr ? a.order[rank] : rank;
  const SeqRange sr = seq_range(a.offsets, a.n, seq);
  const int64_t len = sr.t1 - sr.t0;
  if (!GRAD && len <= a.brief) return;
  const int64_t nc = (len + kC - 1) / kC;
  if (threadIdx.x == 0) {
    if (sr.bad) atomicExch(a.err, (int)kErrOffsets);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], L::WARPS);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, L::WARPS);
    for (int i = 0; i < 3 * RG; ++i) mbar_init(&met[i], KS);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == L::WARPS) {  // ------------------------------------------------ loads
    if (lane == 0) {
      int64_t issued = 0, q_issued = 0;
      for (int64_t c = 0; c < nc; ++c) {
        const int s = (int)(c % ST);
        if (!mbar_wait(&empty[s], (uint32_t)(c / ST & 1) ^ 1, abort_flag, a.err, kErrWaitEmpty))
          break;
        uint8_t* st = smem + s * L::STAGE;
        const int t = (int)(sr.t0 + c * kC);
        mbar_arrive_expect_tx(&full[s], L::STAGE);
        tma_load_3d(st, &mK, &full[s], 0, t, hk * (D / 64));
        for (int g = 0; g < RG; ++g) {
          const int x = h * D + (bx * RG + g) * 16;
          tma_load_2d(st + L::KQ + g * L::V, &mV, &full[s], x, t);
          if (GRAD) tma_load_2d(st + L::KQ + (RG + g) * L::V, &mG, &full[s], x, t);
        }
        bulk_load(st + L::STAGE - L::BLOCK,
                  a.blocks + ((sr.slot + c) * a.H + h) * (int64_t)L::BLOCK, L::BLOCK, &full[s]);
        ++issued;
        if (!mbar_wait(qempty, (uint32_t)(c & 1) ^ 1, abort_flag, a.err, kErrWaitEmpty)) break;
        mbar_arrive_expect_tx(qfull, L::KQ);
        tma_load_3d(smem + L::OFF_Q, &mQ, qfull, 0, t, hk * (D / 64));
        ++q_issued;
      }
      drain_ring(full, ST, issued, a.err);
      drain_ring(qfull, 1, q_issued, a.err);
    }
    return;
  }

  // ---------------------------------------------------------------- 16 rows
  const int grp = warp / KS, kw = warp % KS;
  const int r0 = (bx * RG + grp) * 16, c0 = kw * DK;
  const int row = lane / 4, col = 2 * (lane % 4);
  uint8_t* x_part = smem + L::OFF_X + grp * L::X;
  uint8_t* x_r = x_part + 2 * L::X_PART;
  uint8_t* x_u = x_r + L::X_R;
  // A warp's token tiles (8 tokens): of each 2 KS the one of its number from the
  // front and from the back, so that all warps have the same share of the
  // triangles; the warp a tile belongs to; this lane's ldmatrix row in a pair.
  const auto tile = [&](int j) { return j / 2 * 2 * KS + (j % 2 == 0 ? kw : 2 * KS - 1 - kw); };
  const auto owner = [](int t) { return t % (2 * KS) < KS ? t % (2 * KS) : 2 * KS - 1 - t % (2 * KS); };
  const auto pair_row = [&](int p) { return tile(2 * p + lane / 16) * 8 + lane % 8; };
  met += 3 * grp;
  // all lanes' writes before it are seen by the warps that wait
  const auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&met[i]);
  };
  const auto wait = [&](int i, int64_t c) {
    return __all_sync(0xffffffffu,
                      mbar_wait(&met[i], (uint32_t)(c & 1), abort_flag, a.err, kErrWaitOperand));
  };
  float s[DK / 8][4];
  const float* Si =
      a.S_in == nullptr ? nullptr : a.S_in + ((seq * a.H + h) * D + r0) * (int64_t)D + c0;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j) {
    float2 x = make_float2(0.f, 0.f), y = x;
    if (Si != nullptr) {
      x = *reinterpret_cast<const float2*>(Si + row * D + j * 8 + col);
      y = *reinterpret_cast<const float2*>(Si + (row + 8) * D + j * 8 + col);
    }
    s[j][0] = x.x, s[j][1] = x.y, s[j][2] = y.x, s[j][3] = y.y;
  }
  // ldmatrix rows and columns of this lane: operands stored [n][k] and [k][n]
  const int nk_r = (lane / 16) * 8 + lane % 8, nk_c = lane / 8 % 2;
  const int kn_r = lane % 16, kn_c = (lane / 16) * 8;

  for (int64_t c = 0; c < nc; ++c) {
    const int st = (int)(c % ST);
    if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (uint32_t)(c / ST & 1), abort_flag, a.err,
                                           kErrWaitFull)))
      break;
    uint8_t* base = smem + st * L::STAGE;
    uint8_t* vp = base + L::KQ + grp * L::V;
    const uint32_t sK = smem_u32(base), sQ = smem_u32(smem + L::OFF_Q), sV = smem_u32(vp),
                   sT = sK + L::STAGE - L::BLOCK, sP = sT + 3 * kTri;
    const float* gates = reinterpret_cast<const float*>(base + L::STAGE - kGates);
    const int64_t at = (sr.slot + c) * a.H + h;  // this chunk's place among the kept arrays
    const int valid = len - c * kC < kC ? (int)(len - c * kC) : kC;

    if (GRAD) {
      keep_state<D, DK>(a.kept.S0 + at * D * D, s, r0, c0, lane);
      if (c % kAnchor == 0)
        keep_anchor(a.kept.anchors + ((sr.t0 / (kC * kAnchor) + seq + c / kAnchor) * a.H + h) *
                                         (int64_t)D * D, s, ((r0 / 16) * KS + kw) * (DK / 8), lane);
    }

    // r = S K^T (three parts of S), o = S Q^T (two; for the gradient three), both [16 rows x
    // 64 tokens], over this warp's columns of S.  The shares of r are sent off before o's turn.
    uint32_t sh[DK / 16][4], sm[DK / 16][4], sl[GRAD ? DK / 16 : 1][4];
    float rt[NT][4], ot[NT][4];  // this warp's tiles of the group's sums
    {
      float r[8][4] = {}, rs[8][4] = {};  // of the first part of S, of the small ones
      uint32_t b[2][4];
      ldsm4(sK + sw(kC, nk_r, c0 + nk_c * 8), b[0]);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k) {
        uint32_t(&lo)[4] = sl[GRAD ? k : 0];
        split_a(s[2 * k], s[2 * k + 1], sh[k], sm[k], lo);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int f = k * 4 + p + 1;
          uint32_t(&x)[4] = b[p % 2];
          if (f < DK / 4)
            ldsm4(sK + sw(kC, f % 4 * 16 + nk_r, c0 + f / 4 * 16 + nk_c * 8), b[f % 2]);
          mma(rs[2 * p], sm[k], x[0], x[1]);
          mma(rs[2 * p + 1], sm[k], x[2], x[3]);
          mma(r[2 * p], sh[k], x[0], x[1]);
          mma(r[2 * p + 1], sh[k], x[2], x[3]);
          mma(rs[2 * p], lo, x[0], x[1]);
          mma(rs[2 * p + 1], lo, x[2], x[3]);
        }
      }
      float4* xp = reinterpret_cast<float4*>(x_part);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int y = 0; y < 4; ++y) r[t][y] += rs[t][y];
        if (owner(t) != kw)
          xp[(t * (KS - 1) + (kw < owner(t) ? kw : kw - 1)) * 32 + lane] =
              make_float4(r[t][0], r[t][1], r[t][2], r[t][3]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int w = 0; w < KS; ++w)  // registers have no index: pick by this warp's number
          if (w == kw)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              rt[j][y] = r[j / 2 * 2 * KS + (j % 2 == 0 ? w : 2 * KS - 1 - w)][y];
      arrive(0);
    }
    {
      float o[8][4] = {};
      uint32_t b[2][4];
      if (!__all_sync(0xffffffffu,
                      mbar_wait(qfull, (uint32_t)(c & 1), abort_flag, a.err, kErrWaitFull)))
        break;
#pragma unroll
      for (int pass = GRAD ? 0 : 1; pass < 2; ++pass) {  // small parts first
        ldsm4(sQ + sw(kC, nk_r, c0 + nk_c * 8), b[0]);
#pragma unroll
        for (int e = 0; e < DK / 4; ++e) {  // 4 pairs of tiles for each 16 columns
          const int k = e / 4, p = e % 4, f = e + 1;
          if (f < DK / 4)
            ldsm4(sQ + sw(kC, f % 4 * 16 + nk_r, c0 + f / 4 * 16 + nk_c * 8), b[f % 2]);
          uint32_t(&x)[4] = b[e % 2];
          if (pass == 0) {
            mma(o[2 * p], sl[GRAD ? k : 0], x[0], x[1]);
            mma(o[2 * p + 1], sl[GRAD ? k : 0], x[2], x[3]);
          } else {
            mma(o[2 * p], sh[k], x[0], x[1]);
            mma(o[2 * p + 1], sh[k], x[2], x[3]);
          }
          if (pass == (GRAD ? 0 : 1)) {
            mma(o[2 * p], sm[k], x[0], x[1]);
            mma(o[2 * p + 1], sm[k], x[2], x[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty);
      float4* xp = reinterpret_cast<float4*>(x_part + L::X_PART);
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (owner(t) != kw)
          xp[(t * (KS - 1) + (kw < owner(t) ? kw : kw - 1)) * 32 + lane] =
              make_float4(o[t][0], o[t][1], o[t][2], o[t][3]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int w = 0; w < KS; ++w)
          if (w == kw)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              ot[j][y] = o[j / 2 * 2 * KS + (j % 2 == 0 ? w : 2 * KS - 1 - w)][y];
    }
    const auto add_parts = [&](float(&x)[NT][4], const uint8_t* from) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int w = 0; w < KS - 1; ++w) {
          const float4 v =
              reinterpret_cast<const float4*>(from)[(tile(j) * (KS - 1) + w) * 32 + lane];
          x[j][0] += v.x, x[j][1] += v.y, x[j][2] += v.z, x[j][3] += v.w;
        }
    };
    if (!wait(0, c)) break;
    add_parts(rt, x_part);
    // r = beta (v - gamma r)
#pragma unroll
    for (int p = 0; p < NT / 2; ++p) {
      uint32_t v[4];  // (tokens, rows 0-7), (tokens, rows 8-15) of a tile, then of the next
      ldsm4_t(sV + sw32(pair_row(p), nk_c), v);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = tile(2 * p + x) * 8 + col;
        const float2 ga = *reinterpret_cast<const float2*>(gates + t);
        const float2 be = *reinterpret_cast<const float2*>(gates + 2 * kC + t);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t w = v[2 * x + y / 2];
          const float vv = __uint_as_float(y % 2 ? w & 0xffff0000u : w << 16);
          const float gg = y % 2 ? ga.y : ga.x, bb = y % 2 ? be.y : be.x;
          rt[2 * p + x][y] = t + y % 2 < valid ? bb * (vv - gg * rt[2 * p + x][y]) : 0.f;
        }
      }
    }
    // u = r T^T: tokens i take tokens j <= i
    float ut[NT][4] = {};
    {
      // the parts of r as A operands [tokens / 16][part][lane]: a tile is half of one
      uint2* xr = reinterpret_cast<uint2*>(x_r);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t hi[2], mid[2], lo[2];
        split3(rt[j][0], rt[j][1], hi[0], mid[0], lo[0]);
        split3(rt[j][2], rt[j][3], hi[1], mid[1], lo[1]);
        const int t = tile(j);
        uint2* d = xr + (t / 2 * 3 * 32 + lane) * 2 + t % 2;
        d[0] = make_uint2(hi[0], hi[1]);
        d[64] = make_uint2(mid[0], mid[1]);
        d[128] = make_uint2(lo[0], lo[1]);
      }
      arrive(1);
      if (!wait(1, c)) break;
      // o's parts were written before r's; read before arrive(2), behind which the next
      // step's may come
      add_parts(ot, x_part + L::X_PART);
      float us[2][NT][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k > tile(NT - 1) / 2) break;
        uint32_t hi[4], mid[4], lo[4];
        const uint4* d = reinterpret_cast<const uint4*>(xr) + k * 3 * 32 + lane;
        load_a(d, hi);
        load_a(d + 32, mid);
        load_a(d + 64, lo);
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
          if (k > tile(2 * p + 1) / 2) continue;
          uint32_t b[3][4];
          // strip k of T holds rows from 16 k on; a pair's first tile may lie above
          const int tr = pair_row(p) < 16 * k ? 16 * k : pair_row(p);
#pragma unroll
          for (int x = 0; x < 3; ++x) ldsm4(sT + x * kTri + tri(tr, k * 16 + nk_c * 8), b[x]);
          if (k <= tile(2 * p) / 2) {
            mma(ut[2 * p], hi, b[0][0], b[0][1]);
            mma(us[0][2 * p], mid, b[0][0], b[0][1]);
            mma(us[1][2 * p], hi, b[1][0], b[1][1]);
            mma(us[0][2 * p], lo, b[0][0], b[0][1]);
            mma(us[1][2 * p], mid, b[1][0], b[1][1]);
            mma(us[0][2 * p], hi, b[2][0], b[2][1]);
          }
          mma(ut[2 * p + 1], hi, b[0][2], b[0][3]);
          mma(us[0][2 * p + 1], mid, b[0][2], b[0][3]);
          mma(us[1][2 * p + 1], hi, b[1][2], b[1][3]);
          mma(us[0][2 * p + 1], lo, b[0][2], b[0][3]);
          mma(us[1][2 * p + 1], mid, b[1][2], b[1][3]);
          mma(us[0][2 * p + 1], hi, b[2][2], b[2][3]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int y = 0; y < 4; ++y) ut[j][y] += us[0][j][y] + us[1][j][y];
    }
    // parts of u (for o) and of rest u (for S)
    uint4* xu = reinterpret_cast<uint4*>(x_u);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = tile(j);
      uint32_t hi[2], mid[2], lo[2];
      uint2* d = reinterpret_cast<uint2*>(xu) + (t / 2 * L::U_PARTS * 32 + lane) * 2 + t % 2;
      split3(ut[j][0], ut[j][1], hi[0], mid[0], lo[0]);
      split3(ut[j][2], ut[j][3], hi[1], mid[1], lo[1]);
      d[0] = make_uint2(hi[0], hi[1]);
      d[64] = make_uint2(mid[0], mid[1]);
      if (GRAD) {
        d[320] = make_uint2(lo[0], lo[1]);
        reinterpret_cast<float4*>(a.kept.U)[((at * (D / 16) + r0 / 16) * 8 + t) * 32 + lane] =
            make_float4(ut[j][0], ut[j][1], ut[j][2], ut[j][3]);
      }
      const float2 re = *reinterpret_cast<const float2*>(gates + kC + t * 8 + col);
      split3(ut[j][0] * re.x, ut[j][1] * re.y, hi[0], mid[0], lo[0]);
      split3(ut[j][2] * re.x, ut[j][3] * re.y, hi[1], mid[1], lo[1]);
      d[128] = make_uint2(hi[0], hi[1]);
      d[192] = make_uint2(mid[0], mid[1]);
      d[256] = make_uint2(lo[0], lo[1]);
    }
    arrive(2);
    // o = scale gamma o + u P^T
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float2 ga = *reinterpret_cast<const float2*>(gates + tile(j) * 8 + col);
#pragma unroll
      for (int y = 0; y < 4; ++y) ot[j][y] *= a.scale * (y % 2 ? ga.y : ga.x);
    }
    if (!wait(2, c)) break;
    float os[GRAD ? NT : 1][4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k > tile(NT - 1) / 2) break;
      uint32_t hi[4], mid[4], lo[4];
      load_a(xu + k * L::U_PARTS * 32 + lane, hi);
      load_a(xu + k * L::U_PARTS * 32 + 32 + lane, mid);
      if (GRAD) load_a(xu + k * L::U_PARTS * 32 + 160 + lane, lo);
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        if (k > tile(2 * p + 1) / 2) continue;
        uint32_t b[4];
        const int tr = pair_row(p) < 16 * k ? 16 * k : pair_row(p);
        const uint32_t from = sP + tri(tr, k * 16 + nk_c * 8);
        ldsm4(from, b);
        const bool first = k <= tile(2 * p) / 2;
        float(&s0)[4] = GRAD ? os[GRAD ? 2 * p : 0] : ot[2 * p];
        float(&s1)[4] = GRAD ? os[GRAD ? 2 * p + 1 : 0] : ot[2 * p + 1];
        mma(ot[2 * p + 1], hi, b[2], b[3]);
        if (first) mma(ot[2 * p], hi, b[0], b[1]);
        mma(s1, mid, b[2], b[3]);
        if (first) mma(s0, mid, b[0], b[1]);
        if (GRAD) {
          mma(s1, lo, b[2], b[3]);
          if (first) mma(s0, lo, b[0], b[1]);
          ldsm4(from + kTri, b);
          mma(s1, hi, b[2], b[3]);
          if (first) mma(s0, hi, b[0], b[1]);
          mma(s1, mid, b[2], b[3]);
          if (first) mma(s0, mid, b[0], b[1]);
          ldsm4(from + 2 * kTri, b);
          mma(s1, hi, b[2], b[3]);
          if (first) mma(s0, hi, b[0], b[1]);
        }
      }
    }
    if (GRAD) {
      // this group's share of dO . O, for the gradient of the decays
      const uint32_t sG = sV + RG * L::V;
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        uint32_t w[4];
        ldsm4_t(sG + sw32(pair_row(p), nk_c), w);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = 2 * p + x;
          float y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = ot[j][q] + os[GRAD ? j : 0][q];
          put_dots(a.kept.dots + ((r0 / 16) * (int64_t)a.H + h) * a.n + sr.t0 + c * kC + tile(j) * 8,
                   dot_pair(y, w[2 * x], w[2 * x + 1]), tile(j) * 8, valid, lane);
        }
      }
    } else {
      // O over this group's V (each warp over the tokens it has read), then out
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        const uint32_t w[4] = {pack_bf16x2(ot[2 * p][0], ot[2 * p][1]),
                               pack_bf16x2(ot[2 * p][2], ot[2 * p][3]),
                               pack_bf16x2(ot[2 * p + 1][0], ot[2 * p + 1][1]),
                               pack_bf16x2(ot[2 * p + 1][2], ot[2 * p + 1][3])};
        stsm4_t(sV + sw32(pair_row(p), nk_c), w);
      }
      __syncwarp();
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        const int t = tile(2 * p + lane / 16) * 8 + lane / 2 % 8;
        const uint4 w = *reinterpret_cast<const uint4*>(vp + sw32(t, lane % 2));
        if (t < valid)
          *reinterpret_cast<uint4*>(a.O + (sr.t0 + c * kC + t) * (int64_t)a.H * D + h * D + r0 +
                                    (lane % 2) * 8) = w;
      }
    }
    // S = gamma_64 S + (rest u) K
    {
      uint32_t hi[4][4], mid[4][4], lo[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        load_a(xu + k * L::U_PARTS * 32 + 64 + lane, hi[k]);
        load_a(xu + k * L::U_PARTS * 32 + 96 + lane, mid[k]);
        load_a(xu + k * L::U_PARTS * 32 + 128 + lane, lo[k]);
      }
      const float gl = gates[kC - 1];
      // Rows of K behind the sequence may hold anything: they count as zero here, where
      // tokens are summed (elsewhere they only reach their own columns).
      const auto update = [&](auto tail) {
        uint32_t b[2][4];
        ldsm4_t(sK + sw(kC, kn_r, c0 + kn_c), b[0]);
        float d0[4] = {}, d1[4] = {}, e0[4] = {}, e1[4] = {};
#pragma unroll
        for (int e = 0; e < DK / 4; ++e) {  // 4 steps of 16 tokens for each 16 columns
          const int j = e / 4, k = e % 4, f = e + 1;
          uint32_t(&x)[4] = b[e % 2];
          if (f < DK / 4)
            ldsm4_t(sK + sw(kC, f % 4 * 16 + kn_r, c0 + f / 4 * 16 + kn_c), b[f % 2]);
          if (decltype(tail)::value) {
            const uint32_t k0 = keep_pair(k * 16 + col, valid),
                           k1 = keep_pair(k * 16 + 8 + col, valid);
            x[0] &= k0, x[1] &= k1, x[2] &= k0, x[3] &= k1;
          }
          mma(e0, mid[k], x[0], x[1]);
          mma(e1, mid[k], x[2], x[3]);
          mma(d0, hi[k], x[0], x[1]);
          mma(d1, hi[k], x[2], x[3]);
          mma(e0, lo[k], x[0], x[1]);
          mma(e1, lo[k], x[2], x[3]);
          if (k == 3)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              s[2 * j][y] = fmaf(gl, s[2 * j][y], d0[y] + e0[y]);
              s[2 * j + 1][y] = fmaf(gl, s[2 * j + 1][y], d1[y] + e1[y]);
              d0[y] = d1[y] = e0[y] = e1[y] = 0.f;
            }
        }
      };
      if (valid == kC)
        update(std::false_type());
      else
        update(std::true_type());
    }
    fence_proxy_async_smem();  // O's stores into the stage come before the next loads
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }

  if (GRAD && a.kept.last != nullptr)
    keep_anchor(a.kept.last + (seq * a.H + h) * (int64_t)D * D, s, ((r0 / 16) * KS + kw) * (DK / 8),
                lane);
  if (a.S_out != nullptr) {
    float* So = a.S_out + ((seq * a.H + h) * D + r0) * (int64_t)D + c0;
#pragma unroll
    for (int j = 0; j < DK / 8; ++j) {
      *reinterpret_cast<float2*>(So + row * D + j * 8 + col) = make_float2(s[j][0], s[j][1]);
      *reinterpret_cast<float2*>(So + (row + 8) * D + j * 8 + col) = make_float2(s[j][2], s[j][3]);
    }
  }
}

}  // namespace
}  // namespace ttt
