// Gradient of the gated delta rule in chunks of 64 tokens (the notation of
// kernels_delta_tc.cu; E is the gradient of the state behind a chunk, dO that
// of the outputs).  With u_t = beta_t w_t:
//   dU = P^T dO + rest (K E^T),   X = T^T dU,   dV = beta X,   dbeta = X . w
//   E <- gamma_64 E + (scale gamma dO)^T Q - (gamma dV)^T K
//   dQ = scale gamma (dO S) + A K,              A = lower part of scale Gamma (dO U^T)
//   dK = A^T Q + (M + M^T) K + rest (U E) - gamma (dV S),
//        M = strictly lower part of -Gamma (dV U^T)
// The decays' gradient needs none of these products: scaling S and its gradient
// against each other shows that <E_t, S_t>, the gradient of token t+1's decay,
// changes from token to token by dO_t . O_t - dV_t . V_t alone, so it is a running sum
// from the end, started anew from a product of the two states every 512 tokens.  Of a token
// that fades the state below e^-6 the sum would keep few digits: its gradient is formed from
// the terms that cross it, and the sum starts anew there too.
//
// Three kernels: the inverses of all chunks; delta_chains_kernel, the forward chain once more
// (which keeps the state before each chunk in bf16, as it only enters dQ, dK and those terms, and
// U and dO . O in fp32) and beside it the chain of E from the last chunk to the first (which keeps
// E likewise, and X and dV . V); delta_tokens_grad_kernel, dQ, dK and dbeta of all chunks at
// once, and the decays' gradients.  Where heads share a key head a fourth adds their shares.  The
// chains carry fp32 in three bf16 parts (the gates' gradients and dS are fp32 results), the
// rest is bf16 products summed in fp32.
//
// Bound as the forward pass is by the chain (one frame of 1,374 tokens, 4 heads of 256: 95 us
// of 137), and where there are enough chains to fill the GPU by how many of them an SM holds
// (16,384 tokens in 7 sequences, 16 heads of 128: 1.07 ms of 1.57; two a SM, the tensor
// cores busy for 39% of the time).

#include "delta_state.cuh"

namespace ttt {
namespace {

// ----------------------------------------------------------------------------
// The chain of E: as in delta_state_chain, KS warps share 16 rows of E.
// ----------------------------------------------------------------------------
template <int D, int KS, int RG, int ST>
struct RK {
  static constexpr int WARPS = KS * RG;
  static constexpr int KQ = kC * D * 2;
  static constexpr int BLOCK = chunk_bytes(3);
  static constexpr int V = kC * 32;
  static constexpr int STAGE = 2 * KQ + 2 * RG * V + BLOCK;
  // exchange of a group: partial K E^T, dU in parts, gamma dV in parts
  static constexpr int X_PART = 8 * (KS - 1) * 32 * 16, X_U = 8 * 3 * 32 * 8;
  static constexpr int X = X_PART + 2 * X_U;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int OFF_X = ST * STAGE;
  static constexpr int OFF_BAR = OFF_X + RG * X;
  static constexpr int SMEM = OFF_BAR + 192 + 1024;
  static_assert((KS == 2 || KS == 4) && RG <= 2, "tiles and barriers of a group");
  static_assert(STAGE % 1024 == 0, "tiles are aligned to the swizzle");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct ReverseArgs {
  int64_t n;
  const int64_t* offsets;
  int H, Hk;
  float scale;
  const uint8_t* blocks;
  const int32_t* order;
  const float* dS_out;
  float* dS_in;
  __nv_bfloat16* dV;
  __nv_bfloat16* E;    // the gradient behind each chunk, blocked as S0
  float* X;            // in fp32, as U
  float* anchors;      // E before every kAnchor-th chunk, as the states' anchors
  float* last;         // E behind the last tokens, or nullptr
  float* dots;         // [d / 16][H][n]: dV . V over 16 columns
  int* err;
};

template <int D, int KS, int RG, int ST>
__device__ __forceinline__ void delta_reverse_chain(const CUtensorMap& mQ, const CUtensorMap& mK,
                                                    const CUtensorMap& mV, const CUtensorMap& mG,
                                                    const ReverseArgs& a, uint8_t* smem_raw,
                                                    int bx, int h, int64_t rank) {
  using L = RK<D, KS, RG, ST>;
  constexpr int DK = D / KS, NT = 8 / KS;
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + 2;
  uint64_t* met = empty + 2;  // 3 for each group: partial sums, dU, dV are written
  volatile int* abort_flag = reinterpret_cast<volatile int*>(met + 3 * RG);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = h / (a.H / a.Hk);
  const int64_t seq = a.order != nullptr ? a.order[rank] : rank;
  const SeqRange sr = seq_range(a.offsets, a.n, seq);
  const int64_t len = sr.t1 - sr.t0;
  const int64_t nc = (len + kC - 1) / kC;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], L::WARPS);
    }
    for (int i = 0; i < 3 * RG; ++i) mbar_init(&met[i], KS);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == L::WARPS) {  // ------------------------------------------------ loads
    if (lane == 0) {
      int64_t issued = 0;
      for (int64_t i = 0; i < nc; ++i) {
        const int s = (int)(i % ST);
        if (!mbar_wait(&empty[s], (uint32_t)(i / ST & 1) ^ 1, abort_flag, a.err, kErrWaitEmpty))
          break;
        uint8_t* st = smem + s * L::STAGE;
        const int64_t c = nc - 1 - i;
        const int t = (int)(sr.t0 + c * kC);
        mbar_arrive_expect_tx(&full[s], L::STAGE);
        tma_load_3d(st, &mK, &full[s], 0, t, hk * (D / 64));
        tma_load_3d(st + L::KQ, &mQ, &full[s], 0, t, hk * (D / 64));
        for (int g = 0; g < RG; ++g) {
          const int x = h * D + (bx * RG + g) * 16;
          tma_load_2d(st + 2 * L::KQ + g * L::V, &mV, &full[s], x, t);
          tma_load_2d(st + 2 * L::KQ + (RG + g) * L::V, &mG, &full[s], x, t);
        }
        bulk_load(st + L::STAGE - L::BLOCK,
                  a.blocks + ((sr.slot + c) * a.H + h) * (int64_t)L::BLOCK, L::BLOCK, &full[s]);
        ++issued;
      }
      drain_ring(full, ST, issued, a.err);
    }
    return;
  }

  const int grp = warp / KS, kw = warp % KS;
  const int r0 = (bx * RG + grp) * 16, c0 = kw * DK;
  const int row = lane / 4, col = 2 * (lane % 4);
  uint8_t* x_part = smem + L::OFF_X + grp * L::X;
  uint8_t* x_u = x_part + L::X_PART;
  uint8_t* x_v = x_u + L::X_U;
  // token tiles of this warp, as in delta_state_kernel
  const auto tile = [&](int j) { return j / 2 * 2 * KS + (j % 2 == 0 ? kw : 2 * KS - 1 - kw); };
  const auto owner = [](int t) { return t % (2 * KS) < KS ? t % (2 * KS) : 2 * KS - 1 - t % (2 * KS); };
  const auto pair_row = [&](int p) { return tile(2 * p + lane / 16) * 8 + lane % 8; };
  met += 3 * grp;
  const auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&met[i]);
  };
  const auto wait = [&](int i, int64_t n) {
    return __all_sync(0xffffffffu,
                      mbar_wait(&met[i], (uint32_t)(n & 1), abort_flag, a.err, kErrWaitOperand));
  };
  float s[DK / 8][4];  // E
  const int64_t state = ((seq * a.H + h) * D + r0) * (int64_t)D + c0;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j) {
    float2 x = make_float2(0.f, 0.f), y = x;
    if (a.dS_out != nullptr) {
      x = *reinterpret_cast<const float2*>(a.dS_out + state + row * D + j * 8 + col);
      y = *reinterpret_cast<const float2*>(a.dS_out + state + (row + 8) * D + j * 8 + col);
    }
    s[j][0] = x.x, s[j][1] = x.y, s[j][2] = y.x, s[j][3] = y.y;
  }
  if (a.last != nullptr)  // dS_in may lie over dS_out
    keep_anchor(a.last + (seq * a.H + h) * (int64_t)D * D, s, (r0 / 16 * KS + kw) * (DK / 8), lane);
  const int nk_r = (lane / 16) * 8 + lane % 8, nk_c = lane / 8 % 2;
  const int kn_r = lane % 16, kn_c = (lane / 16) * 8;

  for (int64_t i = 0; i < nc; ++i) {
    const int64_t c = nc - 1 - i;
    const int st = (int)(i % ST);
    if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (uint32_t)(i / ST & 1), abort_flag, a.err,
                                           kErrWaitFull)))
      break;
    uint8_t* base = smem + st * L::STAGE;
    uint8_t* vp = base + 2 * L::KQ + grp * L::V;
    const uint32_t sK = smem_u32(base), sQ = sK + L::KQ, sV = smem_u32(vp), sG = sV + RG * L::V,
                   sT = sK + L::STAGE - L::BLOCK, sP = sT + 3 * kTri;
    const float* gates = reinterpret_cast<const float*>(base + L::STAGE - kGates);
    const int valid = len - c * kC < kC ? (int)(len - c * kC) : kC;
    const int64_t at = (sr.slot + c) * a.H + h;
    keep_state<D, DK>(a.E + at * D * D, s, r0, c0, lane);

    // K E^T over this warp's columns of E
    float du[NT][4];
    {
      float r[8][4] = {}, rs[8][4] = {};
      uint32_t b[2][4];
      ldsm4(sK + sw(kC, nk_r, c0 + nk_c * 8), b[0]);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k) {
        uint32_t hi[4], mid[4], lo[4];
        split_a(s[2 * k], s[2 * k + 1], hi, mid, lo);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int f = k * 4 + p + 1;
          uint32_t(&x)[4] = b[p % 2];
          if (f < DK / 4)
            ldsm4(sK + sw(kC, f % 4 * 16 + nk_r, c0 + f / 4 * 16 + nk_c * 8), b[f % 2]);
          mma(rs[2 * p], mid, x[0], x[1]);
          mma(rs[2 * p + 1], mid, x[2], x[3]);
          mma(r[2 * p], hi, x[0], x[1]);
          mma(r[2 * p + 1], hi, x[2], x[3]);
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
        for (int w = 0; w < KS; ++w)
          if (w == kw)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              du[j][y] = r[j / 2 * 2 * KS + (j % 2 == 0 ? w : 2 * KS - 1 - w)][y];
      arrive(0);
    }
    // dO^T of the group's rows as A operands (rows behind the sequence count as zero), and
    // P^T dO of this warp's tokens: tokens j take tokens i >= j
    uint32_t go[4][4];
    float pd[NT][4] = {};
    {
      float ps[NT][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ldsm4_t(sG + sw32(k * 16 + nk_r, nk_c), go[k]);
        const uint32_t k0 = keep_pair(k * 16 + col, valid), k1 = keep_pair(k * 16 + 8 + col, valid);
        go[k][0] &= k0, go[k][1] &= k0, go[k][2] &= k1, go[k][3] &= k1;
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
          if (k < tile(2 * p) / 2) continue;
          const bool second = k >= tile(2 * p + 1) / 2;
          // rows 16 k .. of the two tiles' strips; one that starts below is not used
          const int tj = lane / 16 == 0 || second ? tile(2 * p + lane / 16) : tile(2 * p);
          const uint32_t from = sP + tri(k * 16 + kn_r, tj * 8);
          uint32_t b[4];
#pragma unroll
          for (int x = 2; x >= 0; --x) {
            ldsm4_t(from + x * kTri, b);
            mma(x == 0 ? pd[2 * p] : ps[2 * p], go[k], b[0], b[1]);
            if (second) mma(x == 0 ? pd[2 * p + 1] : ps[2 * p + 1], go[k], b[2], b[3]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int y = 0; y < 4; ++y) pd[j][y] += ps[j][y];
    }
    if (!wait(0, i)) break;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int w = 0; w < KS - 1; ++w) {
        const float4 v =
            reinterpret_cast<const float4*>(x_part)[(tile(j) * (KS - 1) + w) * 32 + lane];
        du[j][0] += v.x, du[j][1] += v.y, du[j][2] += v.z, du[j][3] += v.w;
      }
      const int t = tile(j) * 8 + col;
      const float2 re = *reinterpret_cast<const float2*>(gates + kC + t);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        du[j][y] = t + y % 2 < valid ? fmaf(y % 2 ? re.y : re.x, du[j][y], pd[j][y]) : 0.f;
    }
    // the parts of an array's tiles as A operands [tokens / 16][part][lane]
    const auto put_parts = [&](uint8_t* to, const float(&x)[NT][4]) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t hi[2], mid[2], lo[2];
        split3(x[j][0], x[j][1], hi[0], mid[0], lo[0]);
        split3(x[j][2], x[j][3], hi[1], mid[1], lo[1]);
        const int t = tile(j);
        uint2* d = reinterpret_cast<uint2*>(to) + (t / 2 * 3 * 32 + lane) * 2 + t % 2;
        d[0] = make_uint2(hi[0], hi[1]);
        d[64] = make_uint2(mid[0], mid[1]);
        d[128] = make_uint2(lo[0], lo[1]);
      }
    };
    put_parts(x_u, du);
    arrive(1);
    if (!wait(1, i)) break;
    // X = T^T dU
    float xt[NT][4] = {};
    {
      float xs[2][NT][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < tile(0) / 2) continue;
        uint32_t hi[4], mid[4], lo[4];
        const uint4* d = reinterpret_cast<const uint4*>(x_u) + k * 3 * 32 + lane;
        load_a(d, hi);
        load_a(d + 32, mid);
        load_a(d + 64, lo);
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
          if (k < tile(2 * p) / 2) continue;
          const bool second = k >= tile(2 * p + 1) / 2;
          const int tj = lane / 16 == 0 || second ? tile(2 * p + lane / 16) : tile(2 * p);
          const uint32_t from = sT + tri(k * 16 + kn_r, tj * 8);
          uint32_t b[3][4];
#pragma unroll
          for (int x = 0; x < 3; ++x) ldsm4_t(from + x * kTri, b[x]);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (z == 1 && !second) continue;
            const int j = 2 * p + z;
            mma(xt[j], hi, b[0][2 * z], b[0][2 * z + 1]);
            mma(xs[0][j], mid, b[0][2 * z], b[0][2 * z + 1]);
            mma(xs[1][j], hi, b[1][2 * z], b[1][2 * z + 1]);
            mma(xs[0][j], lo, b[0][2 * z], b[0][2 * z + 1]);
            mma(xs[1][j], mid, b[1][2 * z], b[1][2 * z + 1]);
            mma(xs[0][j], hi, b[2][2 * z], b[2][2 * z + 1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int y = 0; y < 4; ++y) xt[j][y] += xs[0][j][y] + xs[1][j][y];
    }
    // dV = beta X; the gates' sums over these 16 columns
    float gd[NT][4];  // -gamma dV
    const int64_t dots = ((r0 / 16) * (int64_t)a.H + h) * a.n + sr.t0 + c * kC;
#pragma unroll
    for (int p = 0; p < NT / 2; ++p) {
      uint32_t v[4];
      ldsm4_t(sV + sw32(pair_row(p), nk_c), v);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int j = 2 * p + z, t = tile(j) * 8 + col;
        const float2 be = *reinterpret_cast<const float2*>(gates + 2 * kC + t);
        const float2 ga = *reinterpret_cast<const float2*>(gates + t);
        reinterpret_cast<float4*>(a.X)[((at * (D / 16) + r0 / 16) * 8 + tile(j)) * 32 + lane] =
            make_float4(xt[j][0], xt[j][1], xt[j][2], xt[j][3]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float b = y % 2 ? be.y : be.x;
          xt[j][y] *= b == kNoBeta ? 0.f : b;
          gd[j][y] = -(y % 2 ? ga.y : ga.x) * xt[j][y];
        }
        put_dots(a.dots + dots + tile(j) * 8, dot_pair(xt[j], v[2 * z], v[2 * z + 1]), tile(j) * 8,
                 valid, lane);
      }
    }
    put_parts(x_v, gd);
    arrive(2);
    // dV over this group's V (each warp over the tokens it has read), then out
#pragma unroll
    for (int p = 0; p < NT / 2; ++p) {
      const uint32_t w[4] = {pack_bf16x2(xt[2 * p][0], xt[2 * p][1]),
                             pack_bf16x2(xt[2 * p][2], xt[2 * p][3]),
                             pack_bf16x2(xt[2 * p + 1][0], xt[2 * p + 1][1]),
                             pack_bf16x2(xt[2 * p + 1][2], xt[2 * p + 1][3])};
      stsm4_t(sV + sw32(pair_row(p), nk_c), w);
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < NT / 2; ++p) {
      const int t = tile(2 * p + lane / 16) * 8 + lane / 2 % 8;
      const uint4 w = *reinterpret_cast<const uint4*>(vp + sw32(t, lane % 2));
      if (t < valid)
        *reinterpret_cast<uint4*>(a.dV + (sr.t0 + c * kC + t) * (int64_t)a.H * D + h * D + r0 +
                                  (lane % 2) * 8) = w;
    }
    // E = gamma_64 E + (scale gamma dO)^T Q - (gamma dV)^T K; rows of Q and K behind the
    // sequence may hold anything and count as zero
    const float gl = gates[kC - 1];
    const auto add = [&](uint32_t from, const uint32_t(&hi)[4][4], const uint32_t(&mid)[4][4],
                         const uint32_t(&lo)[4][4], float fade, auto tail) {
      uint32_t b[2][4];
      ldsm4_t(from + sw(kC, kn_r, c0 + kn_c), b[0]);
      float d0[4] = {}, d1[4] = {}, e0[4] = {}, e1[4] = {};
#pragma unroll
      for (int e = 0; e < DK / 4; ++e) {
        const int j = e / 4, k = e % 4, f = e + 1;
        uint32_t(&x)[4] = b[e % 2];
        if (f < DK / 4)
          ldsm4_t(from + sw(kC, f % 4 * 16 + kn_r, c0 + f / 4 * 16 + kn_c), b[f % 2]);
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
            s[2 * j][y] = fmaf(fade, s[2 * j][y], d0[y] + e0[y]);
            s[2 * j + 1][y] = fmaf(fade, s[2 * j + 1][y], d1[y] + e1[y]);
            d0[y] = d1[y] = e0[y] = e1[y] = 0.f;
          }
      }
    };
    const auto add_any = [&](uint32_t from, const uint32_t(&hi)[4][4], const uint32_t(&mid)[4][4],
                             const uint32_t(&lo)[4][4], float fade) {
      if (valid == kC)
        add(from, hi, mid, lo, fade, std::false_type());
      else
        add(from, hi, mid, lo, fade, std::true_type());
    };
    uint32_t hi[4][4], mid[4][4], lo[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // operand register x: tokens 16 k + 8 (x / 2) + col
        const float2 ga =
            *reinterpret_cast<const float2*>(gates + k * 16 + x / 2 * 8 + col);
        split3(__uint_as_float(go[k][x] << 16) * (a.scale * ga.x),
               __uint_as_float(go[k][x] & 0xffff0000u) * (a.scale * ga.y), hi[k][x], mid[k][x],
               lo[k][x]);
      }
    add_any(sQ, hi, mid, lo, gl);
    if (!wait(2, i)) break;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4* d = reinterpret_cast<const uint4*>(x_v) + k * 3 * 32 + lane;
      load_a(d, hi[k]);
      load_a(d + 32, mid[k]);
      load_a(d + 64, lo[k]);
    }
    add_any(sK, hi, mid, lo, 1.f);
    if (c % kAnchor == 0)  // E before the chunk: where the decays' running sum starts anew
      keep_anchor(a.anchors + ((sr.t0 / (kC * kAnchor) + seq + c / kAnchor) * a.H + h) *
                                  (int64_t)D * D, s, (r0 / 16 * KS + kw) * (DK / 8), lane);
    fence_proxy_async_smem();  // dV's stores into the stage come before the next loads
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }

  if (a.dS_in != nullptr) {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j) {
      *reinterpret_cast<float2*>(a.dS_in + state + row * D + j * 8 + col) =
          make_float2(s[j][0], s[j][1]);
      *reinterpret_cast<float2*>(a.dS_in + state + (row + 8) * D + j * 8 + col) =
          make_float2(s[j][2], s[j][3]);
    }
  }
}

// ----------------------------------------------------------------------------
// delta_chains_kernel: both chains of every sequence at once.  Neither needs the other:
// what joins them (dbeta and the decays' gradient) is formed behind them.  So few long
// sequences fill twice the SMs (1,374 tokens, 4 heads of 256: 99 us, one chain after the
// other 189 us), and where there are many, the short chains of one kind fill up beside the
// long ones of the other.  Blocks of a kind lie together in the grid: neighbouring SMs share
// what they fetch of the code (alternating kinds: 127 us).
// ----------------------------------------------------------------------------
template <int D, int ST>
constexpr int chains_smem() {
  return SK<D, 4, 1, ST, true>::SMEM > RK<D, 4, 1, ST>::SMEM ? SK<D, 4, 1, ST, true>::SMEM
                                                             : RK<D, 4, 1, ST>::SMEM;
}
template <int D, int ST>
__global__ void __launch_bounds__(RK<D, 4, 1, ST>::THREADS, ST == 1 ? 2 : 1)
    delta_chains_kernel(const __grid_constant__ CUtensorMap mQ,
                        const __grid_constant__ CUtensorMap mK,
                        const __grid_constant__ CUtensorMap mV,
                        const __grid_constant__ CUtensorMap mG,
                        const __grid_constant__ StateArgs f, const __grid_constant__ ReverseArgs r) {
  extern __shared__ uint8_t smem_raw[];
  const int h = blockIdx.y;
  if (h < f.H)
    delta_reverse_chain<D, 4, 1, ST>(mQ, mK, mV, mG, r, smem_raw, blockIdx.x, h, blockIdx.z);
  else
    delta_state_chain<D, 4, 1, ST, true>(mQ, mK, mV, mG, f, smem_raw, blockIdx.x, h - f.H,
                                         blockIdx.z);
}

constexpr int kGW = 8;  // warps of a block
constexpr int kStretch = kC * kAnchor;

// ----------------------------------------------------------------------------
// dlog_decay of the tokens of one chunk and head whose log decay is below kFade.
// dlog_decay_t = <E_t, S'_t> is e^g_t of what the states on its two sides make together, but
// the running sum's terms are not that small, and what their rounding leaves has e^g_t's digits
// less: at e^-6 as many as the states in bf16 have (8 heads of 256: 3e-3, at e^-8 1.5e-2),
// below that fewer, at last none.  So here it is the sum of all that crosses token t, each
// term with e^g_t in it:
//   from a token j of this chunk to a token i:  Z_ij = Gamma_ij (scale (dO_i . U_j)(q_i . k_j)
//                                                     - (dV_i . U_j)(k_i . k_j)),  j < t <= i
//   from the state before the chunk to i:  gamma_i (scale dO_i . S q_i - dV_i . S k_i)
//   from j to the state behind it:         rest_j (U_j . E k_j)
//   from the one to the other:             gamma_64 <E, S>
// U and dV go in as two bf16 parts (2^-17), S and E as they are kept (2^-9, rounded once).
// U, X, S and E lie as registers hold them and come straight from memory; movmatrix turns U's
// and dV's blocks.  The whole block works on one chunk, some 30 us at d = 256, and forms only what
// a token lies between (one frame of 1,374 tokens, 4 heads of 256: 137 us without such a token,
// 149 us with one in every 512 of every head, 360 us where one head has no others); a call of its
// own keeps its registers apart from those of dQ and dK.
// ----------------------------------------------------------------------------
constexpr float kFade = -6.f;
// such a token, but for those that leave nothing: their gradient is 0
__device__ __forceinline__ bool fades(float g) { return g < kFade && expf(g) != 0.f; }

// What the chains leave and the tokens, of all chunks.
struct ChunksArgs {
  int64_t n;
  const int64_t* offsets;
  int64_t seqs;
  int H, Hk;
  float scale;
  const __nv_bfloat16 *Q, *K, *dO;
  int64_t ldq, ldk;
  const float *g, *b;
  const __nv_bfloat16 *S0, *E;
  const float *U, *X;
  float* dg;
};

__device__ __forceinline__ uint32_t turned(uint32_t x) {  // an 8 x 8 block's transpose
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Two values as two bf16 parts, packed.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

struct FadeSmem {
  float2 G[kC];
  float beta[kC];
  uint32_t tokens[2];  // those to do, a bit each
  float Z[kC][kC + 1];
  float from_s[kGW][kC], to_e[kGW][kC], s_to_e[kGW];  // by warp
};
constexpr int kFadeTiles = 22 * 1024;  // behind it: K, Q, dO as [d / 64][64 tokens][64]
static_assert(sizeof(FadeSmem) <= kFadeTiles, "shared memory of the decays' gradients");

template <int D>
__device__ __noinline__ void fade_chunk(const ChunksArgs& a, uint8_t* smem, int64_t slot, int h) {
  FadeSmem& m = *reinterpret_cast<FadeSmem*>(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, hk = h / (a.H / a.Hk);
  const ChunkRange c = chunk_range(a.offsets, a.n, a.seqs, slot);
  if (c.len == 0) return;  // offsets that are no offsets
  const uint32_t sK = smem_u32(smem + kFadeTiles), sQ = sK + kC * D * 2, sG = sQ + kC * D * 2;
  for (int e = tid; e < kC * D / 8; e += 32 * kGW) {  // rows behind the sequence count as zero
    const int t = e / (D / 8), of = e % (D / 8) * 8;
    const bool ok = t < c.len;
    const int64_t at = c.t0 + (ok ? t : 0);
    cp16(sK + sw(kC, t, of), a.K + at * a.ldk + hk * D + of, ok);
    cp16(sQ + sw(kC, t, of), a.Q + at * a.ldq + hk * D + of, ok);
    cp16(sG + sw(kC, t, of), a.dO + (at * a.H + h) * D + of, ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (warp < 2) {
    const bool in = tid < c.len;
    const float x = in ? a.b[(c.t0 + tid) * a.H + h] : 0.f;
    m.beta[tid] = fabsf(x) <= kNoBeta ? 0.f : x;  // as in the chains
    const uint32_t bits = __ballot_sync(0xffffffffu, in && fades(a.g[(c.t0 + tid) * a.H + h]));
    if (lane == 0) m.tokens[warp] = bits;
  } else if (warp == 2) {
    sum_decays(a.g, c.t0, c.len, a.H, h, lane, m.G);
  }
  for (int t = lane; t < kC; t += 32) m.from_s[warp][t] = m.to_e[warp][t] = 0.f;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  const uint64_t tokens = (uint64_t)m.tokens[1] << 32 | m.tokens[0];
  const int first = __ffsll((int64_t)tokens) - 1, last = 63 - __clzll((int64_t)tokens);
  const int64_t at = slot * a.H + h;
  const int row = lane / 4, col = 2 * (lane % 4);
  const int nk_r = (lane / 16) * 8 + lane % 8, nk_c = (lane / 8 % 2) * 8;
  const int kn_r = lane % 16, kn_c = (lane / 16) * 8;
  const float4 *U = reinterpret_cast<const float4*>(a.U) + at * (D / 16) * 256 + lane,
               *X = reinterpret_cast<const float4*>(a.X) + at * (D / 16) * 256 + lane;

  // steps of 16 of d whose operands are on their way (128 registers a thread, or 256)
  constexpr int U_AHEAD = D == 256 ? 2 : 1, S_AHEAD = D == 256 ? 4 : 1, UNROLL = D == 256 ? 16 : 2;
  // Z of 16 tokens i and 16 tokens j <= i, ten such; those that a token lies between, shared out
  int turn = 0;
#pragma unroll 1
  for (int unit = 0; unit < 10; ++unit) {
    const int mb = unit < 1 ? 0 : unit < 3 ? 1 : unit < 6 ? 2 : 3, m0 = mb * 16,
              j0 = (unit - mb * (mb + 1) / 2) * 16;
    const uint64_t between = tokens >> j0 & (2ull << (m0 + 15 - j0)) - 1;  // j0 .. m0 + 15
    if (between == 0 || turn++ % kGW != warp) {
      if (between == 0 && warp == 0)  // it adds nothing to the sums below
        for (int e = lane; e < 256; e += 32) m.Z[m0 + e / 16][j0 + e % 16] = 0.f;
      continue;
    }
    float dp[2][4] = {}, dl[2][4] = {}, qk[2][4] = {}, kk[2][4] = {};
    float2 b[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) b[x] = *reinterpret_cast<const float2*>(m.beta + m0 + x * 8 + col);
    float4 xs[U_AHEAD][2], us[U_AHEAD][2];
    const auto fetch = [&](int d0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        xs[d0 / 16 % U_AHEAD][x] = X[(d0 / 2 + m0 / 8 + x) * 32];
        us[d0 / 16 % U_AHEAD][x] = U[(d0 / 2 + j0 / 8 + x) * 32];
      }
    };
#pragma unroll
    for (int i = 0; i < U_AHEAD; ++i) fetch(i * 16);
#pragma unroll UNROLL
    for (int d0 = 0; d0 < D; d0 += 16) {
      uint32_t ag[4], aq[4], ak[4], bk[4], vh[4], vl[4];
      ldsm4(sG + sw(kC, m0 + kn_r, d0 + kn_c), ag);
      ldsm4(sQ + sw(kC, m0 + kn_r, d0 + kn_c), aq);
      ldsm4(sK + sw(kC, m0 + kn_r, d0 + kn_c), ak);
      ldsm4(sK + sw(kC, j0 + nk_r, d0 + nk_c), bk);
      const float4 uv[2] = {us[d0 / 16 % U_AHEAD][0], us[d0 / 16 % U_AHEAD][1]};
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // dV = beta X of 8 tokens: rows d, columns tokens
        const float4 v = xs[d0 / 16 % U_AHEAD][x];
        split2(b[x].x * v.x, b[x].y * v.y, vh[x], vl[x]);
        split2(b[x].x * v.z, b[x].y * v.w, vh[x + 2], vl[x + 2]);
      }
      if (d0 + U_AHEAD * 16 < D) fetch(d0 + U_AHEAD * 16);
#pragma unroll
      for (int x = 0; x < 4; ++x) vh[x] = turned(vh[x]), vl[x] = turned(vl[x]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 u = uv[j];
        uint32_t uh[2], ul[2];
        split2(u.x, u.y, uh[0], ul[0]);
        split2(u.z, u.w, uh[1], ul[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) uh[x] = turned(uh[x]), ul[x] = turned(ul[x]);
        mma(dp[j], ag, ul[0], ul[1]);
        mma(dp[j], ag, uh[0], uh[1]);
        mma(dl[j], vl, uh[0], uh[1]);
        mma(dl[j], vh, ul[0], ul[1]);
        mma(dl[j], vh, uh[0], uh[1]);
        mma(qk[j], aq, bk[2 * j], bk[2 * j + 1]);
        mma(kk[j], ak, bk[2 * j], bk[2 * j + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int ti = m0 + row + y / 2 * 8, tj = j0 + j * 8 + col + y % 2;
        m.Z[ti][tj] = tj < ti && ti < c.len ? decay(m.G[ti], m.G[tj]) *
                                                  (a.scale * dp[j][y] * qk[j][y] - dl[j][y] * kk[j][y])
                                            : 0.f;
      }
  }

  // S q, S k and E k of 16 rows of S and E and 32 tokens: rows of S, columns tokens
  float both = 0.f;  // <E, S>
#pragma unroll 1
  for (int unit = warp; unit < D / 8; unit += kGW) {
    const int r = unit / 2, t0 = unit % 2 * 32;
    // what goes to tokens from the first on, and from those before the last
    const bool with_s = t0 + 32 > first, with_e = t0 < last;
    float sq[4][4] = {}, sk[4][4] = {}, ek[4][4] = {};
    // blocks [column / 16][row / 8][column / 8 % 2], as operands want them: row, then column
    const uint32_t *S = reinterpret_cast<const uint32_t*>(a.S0) + at * (D * D / 2) + r * 128 + lane,
                   *E = reinterpret_cast<const uint32_t*>(a.E) + at * (D * D / 2) + r * 128 + lane;
    uint32_t ss[S_AHEAD][4], es[S_AHEAD][4];
    const auto fetch = [&](int i) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int at = i * D * 8 + x % 2 * 64 + x / 2 * 32;
        ss[i % S_AHEAD][x] = S[at], es[i % S_AHEAD][x] = E[at];
      }
    };
#pragma unroll
    for (int i = 0; i < S_AHEAD; ++i) fetch(i);
#pragma unroll UNROLL
    for (int i = 0; i < D / 16; ++i) {
      const int d0 = i * 16;
      uint32_t s[4], e[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] = ss[i % S_AHEAD][x], e[x] = es[i % S_AHEAD][x];
      if (i + S_AHEAD < D / 16) fetch(i + S_AHEAD);
      if (t0 == 0)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          both = fmaf(low(s[x]), low(e[x]), fmaf(high(s[x]), high(e[x]), both));
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t bq[4], bk[4];
        ldsm4(sK + sw(kC, t0 + p * 16 + nk_r, d0 + nk_c), bk);
        if (with_s) {
          ldsm4(sQ + sw(kC, t0 + p * 16 + nk_r, d0 + nk_c), bq);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma(sq[2 * p + j], s, bq[2 * j], bq[2 * j + 1]);
            mma(sk[2 * p + j], s, bk[2 * j], bk[2 * j + 1]);
          }
        }
        if (with_e)
#pragma unroll
          for (int j = 0; j < 2; ++j) mma(ek[2 * p + j], e, bk[2 * j], bk[2 * j + 1]);
      }
    }
    float4 us[4], xs[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      us[q] = U[(r * 8 + t0 / 8 + q) * 32], xs[q] = X[(r * 8 + t0 / 8 + q) * 32];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t go[4];  // dO: (rows 0-7, 8-15) of 8 tokens, then of the next
      ldsm4_t(sG + sw(kC, t0 + p * 16 + nk_r, r * 16 + nk_c), go);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = 2 * p + j, t = t0 + q * 8 + col;
        const float4 u = us[q], x = xs[q];
        const float2 b = *reinterpret_cast<const float2*>(m.beta + t);
        const float dv[4] = {b.x * x.x, b.y * x.y, b.x * x.z, b.y * x.w};
        float f[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t w = go[2 * j + y / 2];
          f[y] = a.scale * (y % 2 ? high(w) : low(w)) * sq[q][y] - dv[y] * sk[q][y];
        }
        const float2 from = rows_sum(make_float2(f[0] + f[2], f[1] + f[3])),
                     to = rows_sum(make_float2(fmaf(u.x, ek[q][0], u.z * ek[q][2]),
                                               fmaf(u.y, ek[q][1], u.w * ek[q][3])));
        if (lane < 4) {
          m.from_s[warp][t] += from.x, m.from_s[warp][t + 1] += from.y;
          m.to_e[warp][t] += to.x, m.to_e[warp][t + 1] += to.y;
        }
      }
    }
  }
  for (int x = 16; x > 0; x /= 2) both += __shfl_xor_sync(0xffffffffu, both, x);
  if (lane == 0) m.s_to_e[warp] = both;
  __syncthreads();
  // the warps' sums in order, each with its decay; rows of Z to sums of what is before a column
  if (tid < kC) {
    float f = 0.f, g = 0.f;
    for (int w = 0; w < kGW; ++w) f += m.from_s[w][tid], g += m.to_e[w][tid];
    m.from_s[0][tid] = decay(m.G[tid]) * f;
    m.to_e[0][tid] = decay(m.G[kC - 1], m.G[tid]) * g;
  } else if (tid < 2 * kC) {
    const int i = tid - kC;
    float x = 0.f;
#pragma unroll 4
    for (int j = 0; j <= i; ++j) {
      const float z = m.Z[i][j];
      m.Z[i][j] = x;
      x += z;
    }
  }
  __syncthreads();
  if (tid < kC && (tokens >> tid & 1) != 0) {  // what crosses each token
    float x = 0.f;
    for (int w = 0; w < kGW; ++w) x += m.s_to_e[w];
    x *= decay(m.G[kC - 1]);
#pragma unroll 4
    for (int i = 0; i < kC; ++i) x += i < tid ? m.to_e[0][i] : m.from_s[0][i] + m.Z[i][tid];
    a.dg[(c.t0 + tid) * a.H + h] = x;
  }
}

// ----------------------------------------------------------------------------
// dlog_decay of 512 tokens of a sequence and head (from one anchor to the next): <E, S>
// at the stretch's end and the running sum from there, which starts anew with every token below
// kFade.  A few blocks' work, done beside dQ and dK.
// ----------------------------------------------------------------------------
struct GateArgs {
  int groups;
  const float *dots_o, *dots_v;
  const float *S, *E;            // anchors
  const float *S_last, *E_last;  // behind the last tokens, or both nullptr: zeros
};

template <int D>
__device__ __forceinline__ void gate_stretch(const GateArgs& a, const ChunksArgs& c, uint8_t* smem,
                                             int64_t slot, int h, int tid) {
  const int64_t* offsets = c.offsets;
  const int64_t n = c.n, seqs = c.seqs;
  const int H = c.H;
  // the sequence of this stretch
  int64_t lo = 0, hi = seqs;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (seq_range(offsets, n, mid).t0 / kStretch + mid <= slot)
      lo = mid;
    else
      hi = mid;
  }
  const SeqRange sr = seq_range(offsets, n, lo);
  const int64_t b0 = sr.t0 + (slot - (sr.t0 / kStretch + lo)) * kStretch;
  if (b0 < sr.t0 || b0 >= sr.t1) return;
  const int64_t b1 = b0 + kStretch < sr.t1 ? b0 + kStretch : sr.t1;
  // <E, S> at the end, the next anchor's or the last states': this thread's share
  const int64_t size = (int64_t)a.groups * a.groups * 256;
  const bool next = b1 < sr.t1;
  const float* es = next ? a.E + ((slot + 1) * H + h) * size
                         : a.E_last != nullptr ? a.E_last + (lo * H + h) * size : nullptr;
  const float* ss = next ? a.S + ((slot + 1) * H + h) * size : a.S_last + (lo * H + h) * size;
  float x = 0.f;
  if (es != nullptr)
#pragma unroll 4
    for (int64_t i = tid * 4; i < size; i += 32 * kGW * 4) {
      const float4 e = *reinterpret_cast<const float4*>(es + i);
      const float4 y = *reinterpret_cast<const float4*>(ss + i);
      x = fmaf(e.x, y.x, fmaf(e.y, y.y, fmaf(e.z, y.z, fmaf(e.w, y.w, x))));
    }
  const auto decay_of = [&](int64_t t) { return t < b1 ? c.g[t * H + h] : 0.f; };
  if (__syncthreads_or(fades(decay_of(b0 + tid)) || fades(decay_of(b0 + tid + 32 * kGW))))
    for (int64_t t = b0; t < b1; t += kC) {
      if (!__syncthreads_or(tid < kC && fades(decay_of(t + tid)))) continue;
      fade_chunk<D>(c, smem, sr.slot + (t - sr.t0) / kC, h);
      __syncthreads();  // its results are there, its arrays are free
    }
  // x of a token: its own value where it has been formed, else v + x of the next.  Over several
  // tokens: s, and whether it ends there (`own`) or x of the token behind them is to be added.
  constexpr int PER = kStretch / (32 * kGW);
  float v[PER], s = 0.f;
  bool done[PER], own = false;
#pragma unroll
  for (int q = PER - 1; q >= 0; --q) {
    const int64_t t = b0 + tid * PER + q;
    const float g = decay_of(t);
    done[q] = g < kFade;
    v[q] = 0.f;
    if (done[q]) {
      if (fades(g)) v[q] = c.dg[t * H + h];
    } else if (t < b1) {
      float o = 0.f, w = 0.f;
#pragma unroll 4
      for (int r = 0; r < a.groups; ++r) {
        const int64_t at = (r * (int64_t)H + h) * n + t;
        o += a.dots_o[at];
        w += a.dots_v[at];
      }
      v[q] = o - w;
    }
    s = done[q] ? v[q] : s + v[q];
    own |= done[q];
  }
  __shared__ float warp_s[kGW], warp_x[kGW];
  __shared__ bool warp_own[kGW];
  const int lane = tid % 32, warp = tid / 32;
  for (int m = 1; m < 32; m *= 2) {
    const float y = __shfl_down_sync(0xffffffffu, s, m);
    const bool z = __shfl_down_sync(0xffffffffu, own, m);
    if (lane + m < 32) {
      s = own ? s : s + y;
      own |= z;
    }
  }
  for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  if (lane == 0) warp_s[warp] = s, warp_own[warp] = own, warp_x[warp] = x;
  __syncthreads();
  x = 0.f;
  for (int w = 0; w < kGW; ++w) x += warp_x[w];
  for (int w = kGW - 1; w > warp; --w) x = warp_own[w] ? warp_s[w] : warp_s[w] + x;
  // the threads behind this one in its warp
  s = __shfl_down_sync(0xffffffffu, s, 1);
  own = __shfl_down_sync(0xffffffffu, own, 1);
  if (lane < 31) x = own ? s : s + x;
#pragma unroll
  for (int q = PER - 1; q >= 0; --q) {
    const int64_t t = b0 + tid * PER + q;
    x = done[q] ? v[q] : v[q] + x;
    if (t < b1) c.dg[t * H + h] = x;
  }
}

// ----------------------------------------------------------------------------
// delta_tokens_grad_kernel: dQ, dK and dbeta of one chunk and head.  8 warps: 4 blocks of 16
// tokens; of the two warps of a block one takes the products with S (dQ, and for dK dV S and
// A^T Q, which it hands over), the other those with E and M (dK).  They hold dO and dV, or U,
// of their tokens in registers; S, E, Q, K pass in strips of 16 columns, as many ahead as
// shared memory holds.  Two blocks share an SM (d = 256: one).
//
// U and A enter in two parts: with one each, dK is off by 3.0e-3 and dQ by 2.7e-3 of which
// 1.7e-3 are the results' own rounding; so 2.4e-3 and 2.1e-3.  Two parts of S, E, dV as well
// would leave 1.9e-3 for twice the traffic.
// 4,320 chunks and heads of d = 128: 358 us, 1.04 GB (161 us); half of the rest is a block's
// start, U, X and dO on their way and A and M formed, with one other block to fill it.
// ----------------------------------------------------------------------------
template <int D>
struct GK {
  static constexpr int TOK = kC * D * 2;        // one of dO, U (two parts), dV
  static constexpr int ST = D * 16 * 2;         // 16 columns of S or E
  static constexpr int QS = kC * 32;            // 16 columns of Q or K
  static constexpr int STRIP = 2 * ST + 2 * QS;
  static constexpr int NS = D / 16;
  // strips in flight: two from the start, then as many more as dO, U, dV leave room for
  // once they are in registers, filled from the back
  static constexpr int RING = 2 + (4 * TOK / STRIP < NS - 2 ? 4 * TOK / STRIP : NS - 2);
  static constexpr int OFF_S = 4 * TOK - (RING - 2) * STRIP;
  static constexpr int OFF_A = 4 * TOK + 2 * STRIP;     // A in two parts, M: triangles
  static constexpr int OFF_X = OFF_A + 3 * kTri;        // what is handed over, two deep
  static constexpr int X = 4 * 2 * 32 * 16;
  static constexpr int OFF_BAR = OFF_X + 2 * X;
  static constexpr int SMEM = OFF_BAR + (1 + 2 * RING) * 8 + 8 + 1024;
  static constexpr uint8_t* place(uint8_t* smem, int s) {  // of strip s
    return smem + OFF_S + (s % RING + RING - 2) % RING * STRIP;
  }
  static_assert(SMEM <= (D == 256 ? 227 : 113) * 1024, "shared memory");
  static_assert(kFadeTiles + 3 * kC * D * 2 + 1024 <= SMEM, "shared memory of the decays' gradients");
};

struct TokensGradArgs : ChunksArgs {
  float* db;
  __nv_bfloat16 *dQ, *dK;  // heads of their own
  float *pq, *pk;          // shared heads: each head's share, [n][H * d]
  int64_t stretches;       // the first blocks take the decays' gradients
  GateArgs gates;
  int* err;
};

template <int D>
__global__ void __launch_bounds__(32 * kGW, D == 256 ? 1 : 2)
    delta_tokens_grad_kernel(const __grid_constant__ CUtensorMap mQ,
                             const __grid_constant__ CUtensorMap mK,
                             const __grid_constant__ CUtensorMap mG,
                             const __grid_constant__ TokensGradArgs a) {
  using L = GK<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ float2 G[kC];
  uint8_t *pG = smem, *pU = smem + L::TOK, *pV = smem + 3 * L::TOK,
          *pA = smem + L::OFF_A, *pM = pA + 2 * kTri;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);  // tokens
  uint64_t *full = bar + 1, *empty = full + L::RING;               // strips
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + L::RING);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t slot = (int64_t)blockIdx.x - a.stretches;
  const int h = blockIdx.y, hk = h / (a.H / a.Hk);
  if (slot < 0) {
    gate_stretch<D>(a.gates, a, smem, blockIdx.x, h, tid);
    return;
  }
  const ChunkRange c = chunk_range(a.offsets, a.n, a.seqs, slot);
  if (c.len == 0) return;
  const int64_t at = slot * a.H + h;
  const auto load_strip = [&](int s) {
    uint8_t* to = L::place(smem, s);
    uint64_t* b = &full[s % L::RING];
    mbar_arrive_expect_tx(b, L::STRIP);
    bulk_load(to, a.S0 + at * D * D + s * (D * 16), L::ST, b);
    bulk_load(to + L::ST, a.E + at * D * D + s * (D * 16), L::ST, b);
    tma_load_2d(to + 2 * L::ST, &mQ, b, hk * D + s * 16, (int)c.t0);
    tma_load_2d(to + 2 * L::ST + L::QS, &mK, b, hk * D + s * 16, (int)c.t0);
  };
  if (tid == 0) {
    mbar_init(bar, 1);
    for (int i = 0; i < L::RING; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kGW);
    }
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(&bar[0], L::TOK);
    tma_load_3d(pG, &mG, &bar[0], 0, (int)c.t0, h * (D / 64));
    load_strip(0);
    load_strip(1);
  }
  if (warp == 1) sum_decays(a.g, c.t0, c.len, a.H, h, lane, G);
  // From U and X: U in two parts and dV = beta X, both [d][64 tokens] in blocks of 8 x 8 (8 rows
  // of 16 bytes: what ldmatrix reads), and dbeta = X . U / beta.  A warp takes 8 tokens.
  {
    const int64_t first = (at * (D / 16) * 8 + warp) * 32 + lane;
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = warp * 8 + lane % 4 * 2 + i;
      b[i] = j < c.len ? a.b[(c.t0 + j) * a.H + h] : 0.f;
      if (fabsf(b[i]) <= kNoBeta) b[i] = 0.f;  // as in the chains
    }
    float2 xw = make_float2(0.f, 0.f);
    constexpr int AHEAD = D / 16 < 8 ? D / 16 : 8;
    float4 xs[AHEAD], uu[AHEAD];
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      xs[r] = reinterpret_cast<const float4*>(a.X)[first + r * 256];
      uu[r] = reinterpret_cast<const float4*>(a.U)[first + r * 256];
    }
#pragma unroll
    for (int r = 0; r < D / 16; ++r) {
      const float4 x = xs[r % AHEAD], u = uu[r % AHEAD];
      if (r + AHEAD < D / 16) {
        xs[r % AHEAD] = reinterpret_cast<const float4*>(a.X)[first + (r + AHEAD) * 256];
        uu[r % AHEAD] = reinterpret_cast<const float4*>(a.U)[first + (r + AHEAD) * 256];
      }
      xw.x = fmaf(x.x, u.x, fmaf(x.z, u.z, xw.x));
      xw.y = fmaf(x.y, u.y, fmaf(x.w, u.w, xw.y));
      const float us[4] = {u.x, u.y, u.z, u.w}, dv[4] = {b[0] * x.x, b[1] * x.y, b[0] * x.z, b[1] * x.w};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t word = (r * 16 + y * 8 + warp) * 32 + lane;
        const uint32_t hi = pack_bf16x2(us[2 * y], us[2 * y + 1]);
        reinterpret_cast<uint32_t*>(pU)[word] = hi;
        reinterpret_cast<uint32_t*>(pU + L::TOK)[word] =
            pack_bf16x2(us[2 * y] - __uint_as_float(hi << 16),
                        us[2 * y + 1] - __uint_as_float(hi & 0xffff0000u));
        reinterpret_cast<uint32_t*>(pV)[word] = pack_bf16x2(dv[2 * y], dv[2 * y + 1]);
      }
    }
    xw = rows_sum(xw);
    if (lane < 4)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (warp * 8 + 2 * lane + i < c.len)
          a.db[(c.t0 + warp * 8 + 2 * lane + i) * a.H + h] =
              (i == 0 ? xw.x : xw.y) / (b[i] == 0.f ? kNoBeta : b[i]);
  }
  __syncthreads();
  bool ok = mbar_wait(&bar[0], 0, abort_flag, a.err, kErrWaitFull);
  const uint32_t sG = smem_u32(pG), sU = smem_u32(pU), sV = smem_u32(pV), sA = smem_u32(pA),
                 sM = smem_u32(pM);
  const int mb = warp / 2, m0 = mb * 16, half = warp % 2;
  const int row = lane / 4, col = 2 * (lane % 4);
  const int nk_r = (lane / 16) * 8 + lane % 8, nk_c = (lane / 8 % 2) * 8;
  const int kn_r = lane % 16, kn_c = (lane / 16) * 8;
  // this lane's row address in a transposed array of 8 x 8 blocks [d / 8][token / 8]: for
  // (16 d from k, 16 tokens from t) as A (tokens are rows) and as B (tokens are columns)
  const auto blk_a = [&](int k, int t) {
    return (uint32_t)(((k / 8 + lane / 16) * 8 + t / 8 + lane / 8 % 2) * 128 + lane % 8 * 16);
  };
  const auto blk_b = [&](int k, int t) {
    return (uint32_t)(((k / 8 + lane / 8 % 2) * 8 + t / 8 + lane / 16) * 128 + lane % 8 * 16);
  };

  // dO U^T (both parts of U) and dV U^T: 16 tokens i x 32 tokens j
  {
    float dp[4][4] = {}, dl[4][4] = {};
#pragma unroll 4
    for (int k = 0; k < D; k += 16) {
      uint32_t ag[4], av[4], b[4];
      ldsm4(sG + sw(kC, m0 + kn_r, k + kn_c), ag);
      ldsm4_t(sV + blk_a(k, m0), av);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t o = sU + blk_b(k, half * 32 + p * 16);
        ldsm4_t(o + L::TOK, b);
        mma(dp[2 * p], ag, b[0], b[1]);
        mma(dp[2 * p + 1], ag, b[2], b[3]);
        ldsm4_t(o, b);
        mma(dp[2 * p], ag, b[0], b[1]);
        mma(dp[2 * p + 1], ag, b[2], b[3]);
        mma(dl[2 * p], av, b[0], b[1]);
        mma(dl[2 * p + 1], av, b[2], b[3]);
      }
    }
    // A (rows behind the sequence are zero: dO there may be anything) and M
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = m0 + row + 8 * y, j = half * 32 + q * 8 + col;
        if (j / 16 > mb) continue;
        float x[2], m[2], left[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float e = j + z <= i ? decay(G[i], G[j + z]) : 0.f;
          x[z] = j + z <= i && i < c.len ? a.scale * e * dp[q][2 * y + z] : 0.f;
          left[z] = x[z] - __bfloat162float(__float2bfloat16_rn(x[z]));
          m[z] = j + z < i ? -e * dl[q][2 * y + z] : 0.f;
        }
        *reinterpret_cast<uint32_t*>(pA + tri(i, j)) = pack_bf16x2(x[0], x[1]);
        *reinterpret_cast<uint32_t*>(pA + kTri + tri(i, j)) = pack_bf16x2(left[0], left[1]);
        *reinterpret_cast<uint32_t*>(pM + tri(i, j)) = pack_bf16x2(m[0], m[1]);
      }
  }
  __syncthreads();

  float gi[2], re[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int i = m0 + row + 8 * y;
    gi[y] = decay(G[i]);
    re[y] = decay(G[kC - 1], G[i]);
  }
  const bool with_e = half == 1;
  // this warp's rows of U in two parts, or of dO and dV: they stay in registers
  uint32_t ax[D / 16][4], ay[D / 16][4];
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    if (with_e) {
      ldsm4_t(sU + blk_a(e * 16, m0), ax[e]);
      ldsm4_t(sU + L::TOK + blk_a(e * 16, m0), ay[e]);
    } else {
      ldsm4(sG + sw(kC, m0 + kn_r, e * 16 + kn_c), ax[e]);
      ldsm4_t(sV + blk_a(e * 16, m0), ay[e]);
    }
  }
  float* shares = with_e ? a.pk : a.pq;
  __nv_bfloat16* grads = with_e ? a.dK : a.dQ;
  const int64_t out_ld = (int64_t)(shares != nullptr ? a.H : a.Hk) * D,
                out = (c.t0 + m0 + row) * out_ld + h * D + col;
  // this lane's addresses in Q's and K's strips; in the triangles, its row of these 16 tokens
  // (strip kb begins at tri_strip(kb)) and of the tokens from 0 on in their columns
  const uint32_t strip_row = sw32(kn_r, lane / 16);
  const uint32_t tri_row = sw32(m0 + kn_r, lane / 16),
                 tri_col = tri_strip(mb) + sw32(nk_r, lane / 8 % 2);
  // dO, U, dV have been read: strips may lie over them.  U and dV were this block's own
  // stores, which the copies have to come behind.
  fence_proxy_async_smem();
  __syncthreads();
  int issued = L::RING;
  if (tid == 0)
    for (int s = 2; s < L::RING; ++s) load_strip(s);
  for (int s = 0; s < L::NS; ++s) {  // 16 columns of dQ, dK at a time
    ok = mbar_wait(&full[s % L::RING], (uint32_t)(s / L::RING & 1), abort_flag, a.err,
                   kErrWaitFull) && ok;
    const uint32_t sS = smem_u32(L::place(smem, s)), sE = sS + L::ST, sQ = sS + 2 * L::ST,
                   sK = sQ + L::QS;
    float4* hand = reinterpret_cast<float4*>(smem + L::OFF_X + s % 2 * L::X) + mb * 64 + lane;
    // acc: scale gamma dO S, or rest U E;  ve: dV S, or rest U E of U's second part
    float acc[2][4] = {}, ve[2][4] = {};
    {
      // 16 rows x 16 columns of a strip [row / 8][2 column blocks]: stored [k][n]
      const uint32_t from = (with_e ? sE : sS) +
                            (uint32_t)((lane / 8 % 2 * 2 + lane / 16) * 128 + lane % 8 * 16);
      uint32_t b[2][4];
      ldsm4_t(from, b[0]);
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const int f = e % 2;
        if (e + 1 < D / 16) ldsm4_t(from + (uint32_t)((e + 1) * 512), b[1 - f]);
        mma(acc[0], ax[e], b[f][0], b[f][1]);
        mma(acc[1], ax[e], b[f][2], b[f][3]);
        mma(ve[0], ay[e], b[f][0], b[f][1]);
        mma(ve[1], ay[e], b[f][2], b[f][3]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (with_e)
          acc[x][y] = re[y / 2] * (acc[x][y] + ve[x][y]);
        else
          acc[x][y] *= a.scale * gi[y / 2], ve[x][y] *= -gi[y / 2];
      }
    }
    // + A K and A^T Q (for dK), or + (M + M^T) K
    const auto triangles = [&](auto tail) {
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        uint32_t x[4], bk[4], bq[4];
        ldsm4_t(sK + strip_row + kb * 512, bk);
        const uint32_t k0 = decltype(tail)::value ? keep_pair(kb * 16 + col, c.len) : 0xffffffffu,
                       k1 = decltype(tail)::value ? keep_pair(kb * 16 + 8 + col, c.len) : 0xffffffffu;
        if (decltype(tail)::value) bk[0] &= k0, bk[1] &= k1, bk[2] &= k0, bk[3] &= k1;
        if (!with_e) {
          if (kb <= mb)
#pragma unroll
            for (int part = 1; part >= 0; --part) {
              ldsm4(sA + part * kTri + tri_row + tri_strip(kb), x);
              mma(acc[0], x, bk[0], bk[1]);
              mma(acc[1], x, bk[2], bk[3]);
            }
          if (kb >= mb) {  // transposes: their rows are the columns
            ldsm4_t(sQ + strip_row + kb * 512, bq);
            if (decltype(tail)::value) bq[0] &= k0, bq[1] &= k1, bq[2] &= k0, bq[3] &= k1;
#pragma unroll
            for (int part = 1; part >= 0; --part) {
              ldsm4_t(sA + part * kTri + tri_col + kb * 512, x);
              mma(ve[0], x, bq[0], bq[1]);
              mma(ve[1], x, bq[2], bq[3]);
            }
          }
        } else {
          if (kb <= mb) {
            ldsm4(sM + tri_row + tri_strip(kb), x);
            mma(acc[0], x, bk[0], bk[1]);
            mma(acc[1], x, bk[2], bk[3]);
          }
          if (kb >= mb) {
            ldsm4_t(sM + tri_col + kb * 512, x);
            mma(acc[0], x, bk[0], bk[1]);
            mma(acc[1], x, bk[2], bk[3]);
          }
        }
      }
    };
    if (c.len == kC)
      triangles(std::false_type());
    else  // rows of Q and K behind the sequence may hold anything and count as zero
      triangles(std::true_type());
    if (!with_e)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        hand[x * 32] = make_float4(ve[x][0], ve[x][1], ve[x][2], ve[x][3]);
    // the two warps of 16 tokens meet; in the buffer before, what this one hands over has
    // been read when they meet again
    asm volatile("bar.sync %0, 64;" ::"r"(1 + mb) : "memory");
    if (L::RING < L::NS) {
      if (lane == 0) mbar_arrive(&empty[s % L::RING]);
      // the place of the strip before is free as soon as the slowest warp is through with it
      if (tid == 0 && ok && *abort_flag == 0 && s > 0 && s - 1 + L::RING < L::NS) {
        if (mbar_wait(&empty[(s - 1) % L::RING], (uint32_t)((s - 1) / L::RING & 1), abort_flag,
                      a.err, kErrWaitEmpty)) {
          load_strip(s - 1 + L::RING);
          issued = s + L::RING;
        }
      }
      __syncwarp();
    }
    if (with_e)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float4 v = hand[x * 32];
        acc[x][0] += v.x, acc[x][1] += v.y, acc[x][2] += v.z, acc[x][3] += v.w;
      }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (m0 + row + 8 * y >= c.len) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int64_t to = out + y * 8 * out_ld + s * 16 + x * 8;
        if (shares != nullptr)
          *reinterpret_cast<float2*>(shares + to) = make_float2(acc[x][2 * y], acc[x][2 * y + 1]);
        else
          *reinterpret_cast<uint32_t*>(grads + to) = pack_bf16x2(acc[x][2 * y], acc[x][2 * y + 1]);
      }
    }
  }
  if (!ok && tid == 0) {  // a wait gave up: the copies must land before the block is gone
    volatile int never = 0;
    mbar_wait(&bar[0], 0, &never, a.err, kErrWaitFinal);
    for (int s = issued - L::RING; s < issued; ++s)
      mbar_wait(&full[s % L::RING], (uint32_t)(s / L::RING & 1), &never, a.err, kErrWaitFinal);
  }
}

// ----------------------------------------------------------------------------
struct Plan {  // byte offsets in the workspace, and the whole
  size_t blocks, S0, E, U, X, anchors, anchors_e, last, last_e, dots_o, dots_v, pq, pk, total;
};
int64_t stretches(const DeltaArgs& a) { return a.n / kStretch + a.seqs; }
Plan plan_of(const DeltaArgs& a) {
  const size_t D = a.d, DD = D * D, ch = (size_t)chunk_slots(a) * a.H,
               an = (size_t)stretches(a) * a.H, sq = (size_t)a.seqs * a.H;
  Plan p;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes, 1024);
    return at;
  };
  p.blocks = take(blocks_bytes(a, 3)) + kOrderBytes;
  p.S0 = take(ch * DD * 2);
  p.E = take(ch * DD * 2);
  p.U = take(ch * kC * D * 4);
  p.X = take(ch * kC * D * 4);
  p.anchors = take(an * DD * 4);
  p.anchors_e = take(an * DD * 4);
  p.last = take(sq * DD * 4);
  p.last_e = take(sq * DD * 4);
  p.dots_o = take(D / 16 * a.H * (size_t)a.n * 4);
  p.dots_v = take(D / 16 * a.H * (size_t)a.n * 4);
  const size_t share = a.H == a.Hk ? 0 : (size_t)a.n * a.H * D * 4;
  p.pq = take(share);
  p.pk = take(share);
  p.total = o;
  return p;
}

struct Call {
  const float* dS_out;
  const void* dO;
  void *dQ, *dK, *dV;
  float *dg, *db, *dS_in;
};

template <int D, int ST>
cudaError_t launch_chains(const DeltaArgs& a, const Call& x, const StateArgs& f,
                          const ReverseArgs& r, cudaStream_t st) {
  CUtensorMap mQ = {}, mK = {}, mV = {}, mG = {};
  if (a.n > 0 && (!head_map(&mQ, a.Q, a.n, a.ldq, a.Hk * D, D) ||
                  !head_map(&mK, a.K, a.n, a.ldk, a.Hk * D, D) ||
                  !strip_map(&mV, a.V, a.n, a.ldv, a.H * D) ||
                  !strip_map(&mG, x.dO, a.n, (int64_t)a.H * D, a.H * D)))
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_attr(delta_chains_kernel<D, ST>, chains_smem<D, ST>());
  if (e != cudaSuccess) return e;
  TraceScope ts("delta_chains", st);
  delta_chains_kernel<D, ST><<<dim3(D / 16, 2 * (unsigned)a.H, (unsigned)a.seqs),
                               RK<D, 4, 1, ST>::THREADS, chains_smem<D, ST>(), st>>>(mQ, mK, mV, mG,
                                                                                     f, r);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tokens(const DeltaArgs& a, const Call& x, char* w, const Plan& p,
                          const GateArgs& gates, cudaStream_t st) {
  using L = GK<D>;
  CUtensorMap mQ, mK, mG;
  if (!strip_map(&mQ, a.Q, a.n, a.ldq, a.Hk * D) || !strip_map(&mK, a.K, a.n, a.ldk, a.Hk * D) ||
      !head_map(&mG, x.dO, a.n, (int64_t)a.H * D, a.H * D, D))
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_attr(delta_tokens_grad_kernel<D>, L::SMEM);
  if (e != cudaSuccess) return e;
  const bool own = a.H == a.Hk;
  const ChunksArgs chunks = {a.n, a.offsets, a.seqs, a.H, a.Hk, a.scale,
                             static_cast<const __nv_bfloat16*>(a.Q),
                             static_cast<const __nv_bfloat16*>(a.K),
                             static_cast<const __nv_bfloat16*>(x.dO), a.ldq, a.ldk, a.g, a.b,
                             reinterpret_cast<const __nv_bfloat16*>(w + p.S0),
                             reinterpret_cast<const __nv_bfloat16*>(w + p.E),
                             reinterpret_cast<const float*>(w + p.U),
                             reinterpret_cast<const float*>(w + p.X), x.dg};
  const TokensGradArgs k = {chunks, x.db, static_cast<__nv_bfloat16*>(x.dQ),
                            static_cast<__nv_bfloat16*>(x.dK),
                            own ? nullptr : reinterpret_cast<float*>(w + p.pq),
                            own ? nullptr : reinterpret_cast<float*>(w + p.pk), stretches(a), gates,
                            device_error_ptr()};
  TraceScope ts("delta_tokens_grad", st);
  delta_tokens_grad_kernel<D><<<dim3((unsigned)(chunk_slots(a) + stretches(a)), (unsigned)a.H), 32 * kGW, L::SMEM,
                                st>>>(mQ, mK, mG, k);
  return cudaGetLastError();
}

}  // namespace

size_t delta_grad_bytes(const DeltaArgs& a) { return plan_of(a).total; }

cudaError_t delta_grad(const DeltaArgs& a, const float* S_in, const void* dO, const float* dS_out,
                       void* dQ, void* dK, void* dV, float* dg, float* db, float* dS_in, void* ws,
                       cudaStream_t st) {
  if (device_error_ptr() == nullptr) return cudaErrorInvalidDevice;
  const Plan p = plan_of(a);
  char* w = static_cast<char*>(ws);
  uint8_t* blocks = reinterpret_cast<uint8_t*>(w + p.blocks);
  const auto floats = [&](size_t at) { return reinterpret_cast<float*>(w + at); };
  const auto halves = [&](size_t at) { return reinterpret_cast<__nv_bfloat16*>(w + at); };
  const Call x = {dS_out, dO, dQ, dK, dV, dg, db, dS_in};
  cudaError_t e = delta_prepare(a, true, blocks, st);
  if (e != cudaSuccess) return e;
  float* last = dS_out != nullptr ? floats(p.last) : nullptr;
  float* last_e = dS_out != nullptr ? floats(p.last_e) : nullptr;
  const DeltaKept kept = {halves(p.S0), floats(p.U), floats(p.anchors),
                          last, floats(p.dots_o)};
  const StateArgs f = {a.n, a.offsets, a.H, a.Hk, a.scale, blocks, order_of(a, blocks), S_in, nullptr,
                       nullptr, -1, kept, device_error_ptr()};
  const ReverseArgs r = {a.n, a.offsets, a.H, a.Hk, a.scale, blocks, order_of(a, blocks), dS_out,
                         dS_in, static_cast<__nv_bfloat16*>(dV), halves(p.E),
                         floats(p.X), floats(p.anchors_e), last_e,
                         floats(p.dots_v), device_error_ptr()};
  // Two stages of copies and all registers, or two blocks an SM: the first where every chain
  // has an SM (1,374 tokens, 4 heads of 128: 70 us against 84), the second from there on (16
  // heads: 111 us against 131; 16,384 tokens in 7 sequences: 1,061 against 1,284).  A block
  // of d = 256 fills an SM.
  const bool few = 2 * a.seqs * a.H * (a.d / 16) <= num_sms();
  e = a.d == 64    ? few ? launch_chains<64, 2>(a, x, f, r, st) : launch_chains<64, 1>(a, x, f, r, st)
      : a.d == 128 ? few ? launch_chains<128, 2>(a, x, f, r, st) : launch_chains<128, 1>(a, x, f, r, st)
                   : launch_chains<256, 2>(a, x, f, r, st);
  if (e != cudaSuccess || a.n == 0) return e;
  const GateArgs gates = {a.d / 16, floats(p.dots_o), floats(p.dots_v), floats(p.anchors),
                          floats(p.anchors_e), last, last_e};
  e = a.d == 64    ? launch_tokens<64>(a, x, w, p, gates, st)
      : a.d == 128 ? launch_tokens<128>(a, x, w, p, gates, st)
                   : launch_tokens<256>(a, x, w, p, gates, st);
  if (e != cudaSuccess || a.H == a.Hk) return e;
  return delta_share(a, reinterpret_cast<const float*>(w + p.pq),
                     reinterpret_cast<const float*>(w + p.pk), dQ, dK, st);
}

}  // namespace ttt
