// The gradients of the gated delta rule that need no further walk.  For 64
// tokens of a head, with S the state that enters them, dS the gradient of the
// state that leaves them, e_t and d_t from the walks (u = beta e, dv = beta d),
// cs the cumulative sum of g over the 64, Gam_ts = exp(cs_t - cs_s):
//
//   P_ts = scale Gam_ts beta_s dy_t.e_s (s <= t),  Z_ts = -Gam_ts beta_t beta_s d_t.e_s (s < t)
//   dq = P K + scale exp(cs) dY S
//   dk = P^T Q + (Z + Z^T) K - beta exp(cs) D S + exp(cs_C - cs) beta E dS
//   dbeta_t = d_t.e_t
//   dg_t = sum_{s < t <= r} W_rs + sum_{r >= t} A_r + sum_{s < t} B_s + exp(cs_C) <dS, S>   (for each head)
//     W_rs = P_rs q_r.k_s + Z_rs k_r.k_s,  B_s = exp(cs_C - cs_s) beta_s e_s.(dS k_s)
//     A_r = scale exp(cs_r) dy_r.(S q_r) - beta_r exp(cs_r) d_r.(S k_r)
//
// dg_t is the sum of all that passes token t, each term with its decay in it, so it
// is held to its own size however small that is.  (dg_t = dg_{t+1} + dq_t.q_t -
// dv_t.v_t costs less, but leaves the rounding of terms that do not pass t: at
// exp(g) = 1e-6 a thousandth of dg, and noise where it is zero.)  A and B are the
// products of what the state's products add to dq and dk with q and k; the sums of
// W are taken in the registers that hold P and Z, 16 x 16 tokens a warp, and put
// together by one thread a token.  All operands that are results are split in two
// terms, and what is returned is rounded once.  (One term for dk's in bf16, errors
// of 2^-12 before its own rounding: 354 us where it now takes 424, of which dg as it
// is now some 20.)
//
// One CTA takes 64 tokens of a group, a slice of the columns n, and some of the
// group's heads, whose dq and dk it adds in registers in a fixed order; sixteen
// warps: four times 16 rows, four quarters of the columns.  (Eight warps with
// twice the columns each took 1.24 times as long: between its barriers a warp's
// instructions depend on one another, and two warps a scheduler do not fill it.)
//
// b4 L2048 H32 G8 P64 N128: 424 us, 507 MB from HBM (1.2 TB/s).  Bound by latency
// between its barriers: the tiles of a head take 220 KB, so one CTA an SM, whose
// sixteen warps issue in 40 % of the clocks and keep the matrix pipe busy for 28 %;
// what waits is barriers (2.2 clocks an instruction: the sums of W are some of the
// warps' only), fixed latencies (1.9) and shared memory (1.3).  Half the columns in each of two CTAs an SM took 899 us
// against 461 at that step, since P and Z are then formed twice.
#pragma once

#include "ssd_delta_blocks.h"
#include "ssd_delta_prep.cuh"

namespace ssd {
namespace delta {

constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kPS = 64;  // headdim columns staged at once

struct GradArgs {
  int64_t L, H, G, P, N, hpg;
  int per_row;        // checkpoints of a row, without a list
  int splits, heads;  // CTAs that share a group's heads, heads of each
  int nslices;        // slices of the columns n
  int pg;
  float scale;
  const char* tokens;  // TokenTiles of both 32-token chunks
  const char* head;    // RevTiles: factors and decays
  const void* dy;
  const float* e;
  const float* d;
  const float* s;       // [slot][head][P][N] states that enter
  const float* ds;      // gradients of the states that leave
  const float *max_y, *max_e, *max_d, *max_s, *max_ds;
  const Slot* slots;    // packed, or null
  void* dq;
  void* dk;
  float* part;          // [split][2][tokens][G][N], with several splits
  int64_t part_size;    // tokens G N
  float* dg;            // [nslice][tokens][H]: with one slice, the gradient itself
  int64_t dg_size;      // tokens H
  float* dbeta;
  int64_t slots_n;
  int64_t pv, pe;       // row pitches of dy, and of e and d: multiples of four
  int pair;             // dq and dk can be written by twos
};

// Sizes of the shared tiles of k_delta_grads, in bytes.
template <typename T, int NT>
struct GradTiles {
  static constexpr int kTerms = sizeof(T) == 2 ? 1 : 2;  // of k, q and dY; what is a result has two
  static constexpr int kNS = sizeof(T) == 4 || NT == 64 ? 64 : 128;  // columns n of a CTA
  static constexpr int kTok = 64 * kNS * 2, kSmall = 64 * 64 * 2;
  static constexpr int kK = 0, kQ = kK + kTerms * kTok;
  static constexpr int kS = kQ + kTerms * kTok;        // hi, lo
  static constexpr int kDS = kS + 2 * kTok;            // hi, lo, as all that follow but Y
  static constexpr int kE = kDS + 2 * kTok;
  static constexpr int kD = kE + 2 * kSmall;
  static constexpr int kY = kD + 2 * kSmall;           // terms
  // P and Z of a head, once its pieces' E, D and dY are used up: in their place
  static constexpr int kW1 = kE;                       // P with k's scales
  static constexpr int kW2 = kW1 + 2 * kSmall;         // P with q's scales
  static constexpr int kZa = kW2 + 2 * kSmall;         // Z with k's scales by row
  static constexpr int kZb = kZa + 2 * kSmall;         // Z with k's scales by column
  static constexpr int kEnd = kZb + 2 * kSmall;
  static_assert(kY + kTerms * kSmall <= kEnd, "the operands of a piece");
  // q k^T and k k^T of the group's tokens: eight values each of every thread of
  // the ten warps whose block lies on or below the diagonal
  static constexpr int kGram = kEnd;
  // E, D and dY of the next piece as they are in memory
  static constexpr int kRawE = kGram + 10 * 32 * 64, kRawD = kRawE + 64 * 64 * 4;
  static constexpr int kRawY = kRawD + 64 * 64 * 4;
  static constexpr int kRawEnd = kRawY + 64 * 64 * (int)sizeof(T);
  // fp32 pieces are read when they are needed
  static constexpr bool kAhead = sizeof(T) == 2;
  static constexpr int kBytes = kAhead ? kRawEnd : kRawE;
};

// A operand: rows row0.., columns col0.. of a row-major tile W wide; or, TRANS,
// the transpose of a tile stored by rows of k.
template <int W, bool TRANS>
__device__ __forceinline__ void a_frag(uint32_t tile, int row0, int col0, int lane, uint32_t (&r)[4]) {
  if constexpr (!TRANS) ldsm4(tile + tile_off<W>(row0 + (lane & 15), col0 + (lane >> 4) * 8), r);
  else ldsm4t(tile + tile_off<W>(col0 + ((lane >> 4) & 1) * 8 + (lane & 7), row0 + ((lane >> 3) & 1) * 8), r);
}

// acc (16 x 8 TN) += A (rows m0.., k steps k0..k1) B, B stored by rows of k
// (columns n0..): TA, TB terms, lo times lo left out.  ATRANS: A is stored by
// rows of k too.
template <int TN, int AW, bool ATRANS, int TA, int BW, int TB>
__device__ __forceinline__ void product(float (&acc)[TN][4], uint32_t a, int as, int m0, uint32_t b, int bs, int n0, int k0,
                                        int k1, int lane) {
  const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, nc = (lane >> 4) * 8;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    uint32_t A[TA][4];
#pragma unroll
    for (int t = 0; t < TA; ++t) a_frag<AW, ATRANS>(a + t * as, m0, 16 * k, lane, A[t]);
#pragma unroll
    for (int t = 0; t < TB; ++t)
      {
        uint32_t B[TN / 2][4];
#pragma unroll
        for (int x = 0; x < TN / 2; ++x) ldsm4t(b + t * bs + tile_off<BW>(16 * k + tr, n0 + 16 * x + nc), B[x]);
#pragma unroll
        for (int x = 0; x < TN; ++x) mma(acc[x], A[0], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
        if (TA == 2 && t == 0) {
#pragma unroll
          for (int x = 0; x < TN; ++x) mma(acc[x], A[TA - 1], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
        }
      }
  }
}

template <int TN>
__device__ __forceinline__ void clear(float (&x)[TN][4]) {
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
}
// to += x times a factor for each of the two rows
template <int TN>
__device__ __forceinline__ void add_rows(float (&to)[TN][4], const float (&x)[TN][4], float f0, float f1) {
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    to[i][0] = fmaf(x[i][0], f0, to[i][0]), to[i][1] = fmaf(x[i][1], f0, to[i][1]);
    to[i][2] = fmaf(x[i][2], f1, to[i][2]), to[i][3] = fmaf(x[i][3], f1, to[i][3]);
  }
}
// The same with a second factor for all, where the product of both may be too
// small for a number.
template <int TN>
__device__ __forceinline__ void add_rows(float (&to)[TN][4], const float (&x)[TN][4], float f0, float f1, float f) {
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    to[i][0] = fmaf(x[i][0] * f0, f, to[i][0]), to[i][1] = fmaf(x[i][1] * f0, f, to[i][1]);
    to[i][2] = fmaf(x[i][2] * f1, f, to[i][2]), to[i][3] = fmaf(x[i][3] * f1, f, to[i][3]);
  }
}
// the rows' products with those of a tile of tokens (columns n0.., TERMS terms, unscaled)
template <int TN, int W, int TERMS>
__device__ __forceinline__ float2 dot_rows(const float (&x)[TN][4], const char* tile, int term_bytes, int r0, int n0, int lane) {
  float d[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t o = tile_off<W>(r0 + 8 * hh, n0 + 8 * i + 2 * (lane & 3));
      float2 q = unpack2(*reinterpret_cast<const uint32_t*>(tile + o));
      if constexpr (TERMS == 2) {
        const float2 l = unpack2(*reinterpret_cast<const uint32_t*>(tile + term_bytes + o));
        q.x += l.x, q.y += l.y;
      }
      d[hh] = fmaf(q.x, x[i][2 * hh], fmaf(q.y, x[i][2 * hh + 1], d[hh]));
    }
  return make_float2(d[0], d[1]);
}

// four scaled values as fp16 terms at byte offset o of a tile
template <int TERMS>
__device__ __forceinline__ void put4(char* tile, int term_bytes, uint32_t o, const float (&x)[4], float sc) {
  uint32_t h0, l0, h1, l1;
  split2(mul2(x[0], x[1], sc), h0, l0);
  split2(mul2(x[2], x[3], sc), h1, l1);
  *reinterpret_cast<uint2*>(tile + o) = make_uint2(h0, h1);
  if constexpr (TERMS == 2) *reinterpret_cast<uint2*>(tile + term_bytes + o) = make_uint2(l0, l1);
}

// four elements of a row, zeros where there are none
template <typename T>
__device__ __forceinline__ void get4(const T* p, int left, bool vec, float (&x)[4]) {
  if (left >= 4 && vec) {
    if constexpr (sizeof(T) == 2) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      const float2 a = bf16x2(u.x), b = bf16x2(u.y);
      x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    } else {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p));
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < left ? to_f(p[e]) : 0.f;
  }
}

// The slot of a call without a list.
__device__ __forceinline__ Slot row_slot(const GradArgs& a, int64_t slot) {
  const int64_t row = slot / a.per_row, i = slot % a.per_row;
  Slot s;
  s.tok = (int)(row * a.L + i * kCheck), s.n = a.L - i * kCheck < kCheck ? (int)(a.L - i * kCheck) : kCheck;
  s.chunk = (int)(row * ((a.L + kC - 1) / kC) + 2 * i);
  return s;
}

// Copy four elements, zeros where there are none: on their way if they lie on
// a boundary of four (`vec`), at once otherwise.
template <typename T>
__device__ __forceinline__ void copy4(char* to, const T* base, int64_t o, int left, bool vec) {
  if (vec) {
    const T* p = left > 0 ? base + o : base;
    if constexpr (sizeof(T) == 4) cp_async16(sm100::smem_u32(to), p, left > 0);
    else cp_async8(sm100::smem_u32(to), p, left > 0);
  } else {
    T* d = reinterpret_cast<T*>(to);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = e < left ? base[o + e] : from_f<T>(0.f);
  }
}
// four elements of shared memory
__device__ __forceinline__ void get4(const float* p, float (&x)[4]) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = bf16x2(u.x), b = bf16x2(u.y);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

template <typename T, int NT>
__global__ void __launch_bounds__(kGradThreads, 1) k_delta_grads(const GradArgs a) {
  using G = GradTiles<T, NT>;
  using X = TokenTiles<T, NT>;
  constexpr int NS = G::kNS, TM = G::kTerms, TN = NS / 32;  // accumulator tiles of a warp: a quarter of the columns
  extern __shared__ __align__(128) char sm[];
  // of the 64 tokens: exp(cs), exp(cs_C - cs), 1 / exp(cs) within their 32-token
  // chunk, and beta, as they were copied; exp(cs) and exp(cs_C - cs) over all 64
  __shared__ __align__(16) float intol[kCheck], outl[kCheck], inv[kCheck], bet[kCheck], into[kCheck], outof[kCheck];
  __shared__ __align__(8) float ik[kCheck], iq[kCheck];  // 1 / scale of the tokens' k and q, the same for all heads
  __shared__ __align__(16) float most[5][8];  // largest magnitudes: chunk (2), 16 columns of headdim (4)
  __shared__ float whole[2];  // of the chunks that exist
  __shared__ int plain[2];
  __shared__ float scale[5], iscale[5];       // of Y, E, D, S, dS
  __shared__ float dde[kCheck];               // d.e
  __shared__ float past[4][kCheck], next[4][kCheck];  // A and B of each quarter of the columns
  __shared__ float rows_w[10][16], cols_w[10][16];    // of the blocks of W: sums over the columns before a token of
                                                      // the rows from it on; over all rows of the columns before it
  __shared__ float wmax[3][kGradWarps], wpi[kGradWarps];
  const uint32_t smu = sm100::smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mt = warp & 3, quarter = warp >> 2;
  int64_t u = blockIdx.x;
  const int split = (int)(u % a.splits);
  u /= a.splits;
  const int ns = (int)(u % a.nslices);
  u /= a.nslices;
  const int64_t grp = u % a.G, slot = u / a.G;
  const Slot sl = a.slots ? a.slots[slot] : row_slot(a, slot);
  if (sl.n == 0) return;
  const int nch = sl.n > kC ? 2 : 1, n0 = ns * NS;
  const int64_t h0 = grp * a.hpg + (int64_t)split * a.heads;
  const int64_t h1 = grp * a.hpg + ((int64_t)(split + 1) * a.heads < a.hpg ? (int64_t)(split + 1) * a.heads : a.hpg);
  const auto image = [&](int c, int64_t h) { return a.head + ((int64_t)(sl.chunk + c) * a.H + h) * RevTiles::kStride; };
  const auto decays = [&](int c, int64_t h) { return reinterpret_cast<const Decays*>(image(c, h) + RevTiles::kBytes); };
  const auto factors = [&](int c, int64_t h) { return reinterpret_cast<const Factors*>(image(c, h) + RevTiles::kF); };
  // the group's k and q: this slice of both chunks' images
#pragma unroll
  for (int w = 0; w < 2; ++w)
    for (int i = threadIdx.x; i < TM * 64 * (NS / 8); i += kGradThreads) {
      const int t = i / (64 * (NS / 8)), r = i / (NS / 8) % 64, c = i % (NS / 8);
      const char* src = a.tokens + ((int64_t)(sl.chunk + (r >> 5)) * a.G + grp) * X::kBytes + (w * TM + t) * X::kTile +
                        (r & 31) * (NT * 2) + n0 * 2 + c * 16;
      const uint32_t dst = (w ? G::kQ : G::kK) + t * G::kTok + r * (NS * 2) + c * 16;
      *reinterpret_cast<uint4*>(sm + dst) =
          r < kC * nch ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    }
  if (threadIdx.x < kCheck) {
    const int t = threadIdx.x;
    ik[t] = t < kC * nch ? decays(t >> 5, h0)->ik[t & 31] : 1.f;
    iq[t] = t < kC * nch ? decays(t >> 5, h0)->iq[t & 31] : 1.f;
  }
  __syncthreads();
  const int sb = quarter;  // this warp's block of P, Z and W: columns 16 sb.., if not above the diagonal
  const int r0 = 16 * mt + (lane >> 2);  // this thread's rows: r0, r0 + 8
  const int blk = mt * (mt + 1) / 2 + sb;
  if (sb <= mt) {  // q k^T and k k^T
    float x[2][4], z[2][4];
    clear(x);
    clear(z);
    const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
#pragma unroll 2
    for (int k = 0; k < NS / 16; ++k) {
      uint32_t Q[TM][4], K[TM][4], B[TM][4];
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        a_frag<NS, false>(smu + G::kQ + t * G::kTok, 16 * mt, 16 * k, lane, Q[t]);
        a_frag<NS, false>(smu + G::kK + t * G::kTok, 16 * mt, 16 * k, lane, K[t]);
        ldsm4(smu + G::kK + t * G::kTok + tile_off<NS>(16 * sb + br, 16 * k + bc), B[t]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mma(x[i], Q[0], B[0][2 * i], B[0][2 * i + 1]);
        mma(z[i], K[0], B[0][2 * i], B[0][2 * i + 1]);
        if constexpr (TM == 2) {
          mma(x[i], Q[0], B[TM - 1][2 * i], B[TM - 1][2 * i + 1]);
          mma(z[i], K[0], B[TM - 1][2 * i], B[TM - 1][2 * i + 1]);
          mma(x[i], Q[TM - 1], B[0][2 * i], B[0][2 * i + 1]);
          mma(z[i], K[TM - 1], B[0][2 * i], B[0][2 * i + 1]);
        }
      }
    }
    float4* const to = reinterpret_cast<float4*>(sm + G::kGram) + blk * 128 + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 ks = *reinterpret_cast<const float2*>(ik + 16 * sb + 8 * i + 2 * (lane & 3));
      to[64 * i] = make_float4(x[i][0] * iq[r0] * ks.x, x[i][1] * iq[r0] * ks.y, x[i][2] * iq[r0 + 8] * ks.x,
                               x[i][3] * iq[r0 + 8] * ks.y);
      to[64 * i + 32] = make_float4(z[i][0] * ik[r0] * ks.x, z[i][1] * ik[r0] * ks.y, z[i][2] * ik[r0 + 8] * ks.x,
                                    z[i][3] * ik[r0 + 8] * ks.y);
    }
  }
  float dq[TN][4], dk[TN][4];
  clear(dq);
  clear(dk);

  // A piece is 64 columns of headdim of one head.  What the next piece needs is
  // copied while this one is worked on: decays and largest magnitudes, E, D and
  // dY, and, where this piece's operands have been used up, the states.
  const bool n4 = a.N % 4 == 0;
  const auto copy_small = [&](int64_t h, int p0) {
    if (h >= h1) return;
    const int t = threadIdx.x;
    if (t < kCheck) {
      if (p0 == 0 && t < kC * nch) {
        const Decays* d = decays(t >> 5, h);
        cp_async4(sm100::smem_u32(intol + t), d->into + (t & 31));
        cp_async4(sm100::smem_u32(outl + t), d->outof + (t & 31));
        cp_async4(sm100::smem_u32(inv + t), d->inv + (t & 31));
        cp_async4(sm100::smem_u32(bet + t), factors(t >> 5, h)->beta + (t & 31));
        if ((t & 31) == 0) {
          cp_async4(sm100::smem_u32(whole + (t >> 5)), &factors(t >> 5, h)->whole);
          cp_async4(sm100::smem_u32(plain + (t >> 5)), &d->plain);
        }
      }
    } else if (t < kCheck + 40) {
      const int w = (t - kCheck) >> 3, c = ((t - kCheck) >> 2) & 1, i = p0 / 16 + (t & 3);
      const float* src = w == 0 ? a.max_y : w == 1 ? a.max_e : w == 2 ? a.max_d : w == 3 ? a.max_s : a.max_ds;
      const int64_t row = w < 3 ? (int64_t)(sl.chunk + c) * a.H + h : slot * a.H + h;
      float* const to = &most[w][(t - kCheck) & 7];
      if (i < a.pg && (c == 0 || (w < 3 && nch == 2))) cp_async4(sm100::smem_u32(to), src + row * a.pg + i);
      else *to = 0.f;
    }
  };
  const auto copy_rows = [&](int64_t h, int p0) {
    if (h >= h1) return;
    if constexpr (G::kAhead) {
#pragma unroll
      for (int x = 0; x < 64 * 16 / kGradThreads; ++x) {
        const int t = (threadIdx.x >> 4) + (kGradThreads / 16) * x, p = (threadIdx.x & 15) * 4;
        const int left = t < sl.n ? (int)(a.P - p0 - p) : 0;
        const int64_t th = ((int64_t)sl.tok + t) * a.H + h, oe = th * a.pe + p0 + p, ov = th * a.pv + p0 + p;
        copy4(sm + G::kRawE + (t * 64 + p) * 4, a.e, oe, left, true);
        copy4(sm + G::kRawD + (t * 64 + p) * 4, a.d, oe, left, true);
        copy4(sm + G::kRawY + (t * 64 + p) * (int)sizeof(T), static_cast<const T*>(a.dy), ov, left, true);
      }
    }
  };
  constexpr int kSt = kPS * (NS / 4) / kGradThreads;  // fours of a state tile a thread holds
  const auto state_at = [&](int i, int p0, int& p, int& n) {
    const int at = threadIdx.x + i * kGradThreads;
    p = at / (NS / 4), n = (at % (NS / 4)) * 4;
    return p0 + p < a.P ? (int)(a.N - n0 - n) : 0;  // columns that exist
  };
  const auto copy_states = [&](int64_t h, int p0) {
    if (h >= h1) return;
    if constexpr (G::kAhead) {
#pragma unroll
      for (int i = 0; i < kSt; ++i) {
        int p, n;
        const int left = state_at(i, p0, p, n);
        const int64_t o = ((slot * a.H + h) * a.P + p0 + p) * a.N + n0 + n;
        const int to = (threadIdx.x + i * kGradThreads) * 16;
        copy4(sm + G::kS + to, a.s, o, left, n4);
        copy4(sm + G::kDS + to, a.ds, o, left, n4);
      }
    }
  };
  copy_small(h0, 0);
  copy_rows(h0, 0);
  copy_states(h0, 0);
  cp_async_commit();
  for (int64_t h = h0; h < h1; ++h) {
    float P[2][4], Z[2][4];
    clear(P);
    clear(Z);
    float pi = 0.f;
    float2 ra = make_float2(0.f, 0.f), rb = ra;  // A and B of this thread's rows
    for (int p0 = 0; p0 < a.P; p0 += kPS) {
      const int64_t hn = p0 + kPS < a.P ? h : h + 1;  // the next piece
      const int pn = p0 + kPS < a.P ? p0 + kPS : 0;
      cp_async_wait<0>();
      __syncthreads();  // this piece's copies are there, the last one's operands are used up
      if (threadIdx.x < kCheck) {
        const int t = threadIdx.x;
        if (p0 == 0) {
          if (t >= kC * nch) intol[t] = outl[t] = inv[t] = 1.f, bet[t] = 0.f;
          into[t] = intol[t] * (t >= kC && nch == 2 ? whole[0] : 1.f);
          outof[t] = outl[t] * (t < kC && nch == 2 ? whole[1] : 1.f);
          dde[t] = 0.f;
        }
      } else if (threadIdx.x < kCheck + 5) {
        const int w = threadIdx.x - kCheck;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, most[w][i]);
        scale[w] = pow2_scale(m, iscale[w]);
      }
      {  // the states to operands, and <dS, S>
        float xs[kSt][4], xd[kSt][4];
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
          int p, n;
          const int left = state_at(i, p0, p, n);
          if constexpr (G::kAhead) {
            get4(reinterpret_cast<const float*>(sm + G::kS) + (threadIdx.x + i * kGradThreads) * 4, xs[i]);
            get4(reinterpret_cast<const float*>(sm + G::kDS) + (threadIdx.x + i * kGradThreads) * 4, xd[i]);
          } else {
            const int64_t o = ((slot * a.H + h) * a.P + p0 + p) * a.N + n0 + n;
            get4(a.s + o, left, n4, xs[i]);
            get4(a.ds + o, left, n4, xd[i]);
          }
        }
        __syncthreads();  // the copied tiles are read; factors and scales are there
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
          int p, n;
          state_at(i, p0, p, n);
          const uint32_t to = tile_off<NS>(p, n);
          put4<2>(sm + G::kS, G::kTok, to, xs[i], scale[3]);
          put4<2>(sm + G::kDS, G::kTok, to, xd[i], scale[4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) pi = fmaf(xd[i][e], xs[i][e], pi);
        }
      }
#pragma unroll
      for (int x = 0; x < 64 * 16 / kGradThreads; ++x) {  // E, D and dY to operands; d.e
        const int t = (threadIdx.x >> 4) + (kGradThreads / 16) * x, p = (threadIdx.x & 15) * 4;
        float e4[4], d4[4], y4[4];
        if constexpr (G::kAhead) {
          get4(reinterpret_cast<const float*>(sm + G::kRawE) + t * 64 + p, e4);
          get4(reinterpret_cast<const float*>(sm + G::kRawD) + t * 64 + p, d4);
          get4(reinterpret_cast<const T*>(sm + G::kRawY) + t * 64 + p, y4);
        } else {
          const int left = t < sl.n ? (int)(a.P - p0 - p) : 0;
          const int64_t th = ((int64_t)sl.tok + t) * a.H + h, oe = th * a.pe + p0 + p, ov = th * a.pv + p0 + p;
          get4(a.e + oe, left, true, e4);
          get4(a.d + oe, left, true, d4);
          get4(static_cast<const T*>(a.dy) + ov, left, true, y4);
        }
        float de = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) de = fmaf(d4[i], e4[i], de);
#pragma unroll
        for (int i = 8; i > 0; i >>= 1) de += __shfl_xor_sync(0xffffffffu, de, i);
        if ((lane & 15) == 0) dde[t] += de;  // one thread of its own for each t
        const uint32_t to = tile_off<64>(t, p);
        put4<2>(sm + G::kE, G::kSmall, to, e4, scale[1]);
        put4<2>(sm + G::kD, G::kSmall, to, d4, scale[2]);
        put4<TM>(sm + G::kY, G::kSmall, to, y4, scale[0]);
      }
      __syncthreads();
      copy_rows(hn, pn);
      const float iy = iscale[0], ie = iscale[1], id = iscale[2], is = iscale[3], ids = iscale[4];
      // dY E^T and D E^T, blocks of 16 tokens on and below the diagonal
      if (sb <= mt) {
        float x[2][4], z[2][4];
        clear(x);
        clear(z);
        const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int k = 0; k < kPS / 16; ++k) {
          uint32_t Y[TM][4], D[2][4], E[2][4];
#pragma unroll
          for (int t = 0; t < TM; ++t) a_frag<64, false>(smu + G::kY + t * G::kSmall, 16 * mt, 16 * k, lane, Y[t]);
#pragma unroll
          for (int t = 0; t < 2; ++t) a_frag<64, false>(smu + G::kD + t * G::kSmall, 16 * mt, 16 * k, lane, D[t]);
#pragma unroll
          for (int t = 0; t < 2; ++t) ldsm4(smu + G::kE + t * G::kSmall + tile_off<64>(16 * sb + br, 16 * k + bc), E[t]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma(x[i], Y[0], E[0][2 * i], E[0][2 * i + 1]);
            mma(z[i], D[0], E[0][2 * i], E[0][2 * i + 1]);
            mma(x[i], Y[0], E[1][2 * i], E[1][2 * i + 1]);
            mma(z[i], D[0], E[1][2 * i], E[1][2 * i + 1]);
            if constexpr (TM == 2) mma(x[i], Y[TM - 1], E[0][2 * i], E[0][2 * i + 1]);
            mma(z[i], D[1], E[0][2 * i], E[0][2 * i + 1]);
          }
        }
        add_rows(P, x, iy, iy, ie);
        add_rows(Z, z, id, id, ie);
      }
      float tmp[TN][4];
      const int nb = quarter * (NS / 4);
      const float in0 = into[r0], in1 = into[r0 + 8], be0 = bet[r0], be1 = bet[r0 + 8];
      clear(tmp);
      product<TN, 64, false, TM, NS, 2>(tmp, smu + G::kY, G::kSmall, 16 * mt, smu + G::kS, G::kTok, nb, 0, kPS / 16, lane);
      // a row's product with its q or k is what it gives to A or B, as it is added
      const auto add = [&](float (&to)[TN][4], float f0, float f1, float f, float2& sum, int tile, const float* inv_scale) {
        const float2 d = dot_rows<TN, NS, TM>(tmp, sm + tile, G::kTok, r0, nb, lane);
        sum.x = fmaf(d.x * inv_scale[r0] * f0, f, sum.x), sum.y = fmaf(d.y * inv_scale[r0 + 8] * f1, f, sum.y);
        add_rows(to, tmp, f0, f1, f);
      };
      add(dq, a.scale * in0 * iy, a.scale * in1 * iy, is, ra, G::kQ, iq);
      clear(tmp);
      product<TN, 64, false, 2, NS, 2>(tmp, smu + G::kD, G::kSmall, 16 * mt, smu + G::kS, G::kTok, nb, 0, kPS / 16, lane);
      add(dk, -be0 * in0 * id, -be1 * in1 * id, is, ra, G::kK, ik);
      clear(tmp);
      product<TN, 64, false, 2, NS, 2>(tmp, smu + G::kE, G::kSmall, 16 * mt, smu + G::kDS, G::kTok, nb, 0, kPS / 16, lane);
      add(dk, be0 * outof[r0] * ie, be1 * outof[r0 + 8] * ie, ids, rb, G::kK, ik);
      if (hn == h) {  // another piece of this head
        __syncthreads();
        copy_small(hn, pn);
        copy_states(hn, pn);
        cp_async_commit();
      }
    }
    // P and Z with their decays; the scale of the token's k or q goes with the
    // one that is summed over.  A block's rows are in one chunk, its columns too.
    float m1 = 0.f, m2 = 0.f, m3 = 0.f;
    // Blocks of a second chunk that does not exist stay zero, as their rows of
    // the operands are: it has no decays to read.
    if (block_exists(mt, sb, nch)) {
      const bool cross = (mt >> 1) != (sb >> 1), simple = cross || plain[mt >> 1];
      const float* cf = cross ? outl : inv;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int t = r0 + 8 * hh;
        const float rf = intol[t], bt = -bet[t];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int s = 16 * sb + 8 * i + 2 * (lane & 3) + e;
            float w = rf * cf[s];
            if (!simple && s <= t) w = pow2_of(decays(mt >> 1, h)->cs[t & 31] - decays(mt >> 1, h)->cs[s & 31]);
            w = s <= t ? w * bet[s] : 0.f;
            float& p = P[i][2 * hh + e];
            float& z = Z[i][2 * hh + e];
            p *= a.scale * w;
            z = s < t ? z * (bt * w) : 0.f;
            m1 = fmaxf(m1, fabsf(p * ik[s])), m2 = fmaxf(m2, fabsf(p * iq[t]));
            m3 = fmaxf(m3, fmaxf(fabsf(z * ik[t]), fabsf(z * ik[s])));
          }
      }
    }
    if (sb <= mt) {  // W, and the sums of it that dg takes
      const float4* const from = reinterpret_cast<const float4*>(sm + G::kGram) + blk * 128 + lane;
      float w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 x = from[64 * i], z = from[64 * i + 32];
        const float qk[4] = {x.x, x.y, x.z, x.w}, kk[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = r0 + 8 * (e >> 1), s = 16 * sb + 8 * i + 2 * (lane & 3) + (e & 1);
          w[i][e] = s < t ? fmaf(P[i][e], qk[e], Z[i][e] * kk[e]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // over the rows from each one on
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, w[i][e], o), v = __shfl_down_sync(0xffffffffu, w[i][2 + e], o);
            if (lane + o < 32) w[i][e] += u, w[i][2 + e] += v;
          }
          w[i][e] += __shfl_sync(0xffffffffu, w[i][2 + e], lane & 3);
        }
      }
      float before = 0.f;  // all rows: the columns before each one
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float up = w[i][0] + w[i][1];
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          const float u = __shfl_up_sync(0xffffffffu, up, o);
          if ((lane & 3) >= o) up += u;
        }
        const float u = __shfl_up_sync(0xffffffffu, up, 1), x = before + ((lane & 3) ? u : 0.f);
        if (lane < 4) cols_w[blk][8 * i + 2 * lane] = x, cols_w[blk][8 * i + 2 * lane + 1] = x + w[i][0];
        before += __shfl_sync(0xffffffffu, up, 3);
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (16 * sb + 8 * i + 2 * (lane & 3) + e < r0 + 8 * hh) x += w[i][2 * hh + e];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if ((lane & 3) == 0) rows_w[blk][(lane >> 2) + 8 * hh] = x;
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ra.x += __shfl_xor_sync(0xffffffffu, ra.x, o), ra.y += __shfl_xor_sync(0xffffffffu, ra.y, o);
      rb.x += __shfl_xor_sync(0xffffffffu, rb.x, o), rb.y += __shfl_xor_sync(0xffffffffu, rb.y, o);
    }
    if ((lane & 3) == 0) {
      past[quarter][r0] = ra.x, past[quarter][r0 + 8] = ra.y;
      next[quarter][r0] = rb.x, next[quarter][r0 + 8] = rb.y;
    }
    {
      m1 = absmax_bits(__float_as_uint(m1)), m2 = absmax_bits(__float_as_uint(m2)), m3 = absmax_bits(__float_as_uint(m3));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) pi += __shfl_xor_sync(0xffffffffu, pi, o);
      if (lane == 0) wmax[0][warp] = m1, wmax[1][warp] = m2, wmax[2][warp] = m3, wpi[warp] = pi;
    }
    __syncthreads();  // and the states' operands are used up
    copy_states(h + 1, 0);
    float i1, i2, i3;
    {
      m1 = lane < kGradWarps ? wmax[0][lane] : 0.f, m2 = lane < kGradWarps ? wmax[1][lane] : 0.f;
      m3 = lane < kGradWarps ? wmax[2][lane] : 0.f;
      const float s1 = pow2_scale(absmax_bits(__float_as_uint(m1)), i1), s2 = pow2_scale(absmax_bits(__float_as_uint(m2)), i2),
                  s3 = pow2_scale(absmax_bits(__float_as_uint(m3)), i3);
      if (sb <= mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float kt = ik[r0 + 8 * hh], qt = iq[r0 + 8 * hh];
            const float2 ks = *reinterpret_cast<const float2*>(ik + 16 * sb + 8 * i + 2 * (lane & 3));
            const float2 p = make_float2(P[i][2 * hh], P[i][2 * hh + 1]), z = make_float2(Z[i][2 * hh], Z[i][2 * hh + 1]);
            const uint32_t o = tile_off<64>(r0 + 8 * hh, 16 * sb + 8 * i + 2 * (lane & 3));
            const auto put = [&](int at, float2 x) {
              uint32_t hi, lo;
              split2(x, hi, lo);
              *reinterpret_cast<uint32_t*>(sm + at + o) = hi;
              *reinterpret_cast<uint32_t*>(sm + at + G::kSmall + o) = lo;
            };
            put(G::kW1, mul2(p.x * ks.x, p.y * ks.y, s1));
            put(G::kW2, mul2(p.x * qt, p.y * qt, s2));
            put(G::kZa, mul2(z.x * kt, z.y * kt, s3));
            put(G::kZb, mul2(z.x * ks.x, z.y * ks.y, s3));
          }
      }
    }
    __syncthreads();
    {
      float tmp[TN][4];
      const int nb = quarter * (NS / 4);
      clear(tmp);
      product<TN, 64, false, 2, NS, TM>(tmp, smu + G::kW1, G::kSmall, 16 * mt, smu + G::kK, G::kTok, nb, 0, mt + 1, lane);
      add_rows(dq, tmp, i1, i1);
      clear(tmp);
      product<TN, 64, true, 2, NS, TM>(tmp, smu + G::kW2, G::kSmall, 16 * mt, smu + G::kQ, G::kTok, nb, mt, 4, lane);
      add_rows(dk, tmp, i2, i2);
      clear(tmp);
      product<TN, 64, true, 2, NS, TM>(tmp, smu + G::kZa, G::kSmall, 16 * mt, smu + G::kK, G::kTok, nb, mt, 4, lane);
      product<TN, 64, false, 2, NS, TM>(tmp, smu + G::kZb, G::kSmall, 16 * mt, smu + G::kK, G::kTok, nb, 0, mt + 1, lane);
      add_rows(dk, tmp, i3, i3);
    }
    __syncthreads();
    if (threadIdx.x < kCheck) {  // dg and dbeta: two warps of 32 tokens each
      const int t = threadIdx.x, o = t ^ 32;
      const auto four = [](const float (&x)[4][kCheck], int i) { return (x[0][i] + x[1][i]) + (x[2][i] + x[3][i]); };
      float from = four(past, t), upto = four(next, t), other = warp ? four(next, o) : four(past, o), all = 0.f;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const float u = __shfl_down_sync(0xffffffffu, from, i), v = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane + i < 32) from += u;
        if (lane >= i) upto += v;
        other += __shfl_xor_sync(0xffffffffu, other, i);
      }
      upto = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 0) upto = 0.f;
      if (warp) upto += other;
      else from += other;
#pragma unroll
      for (int i = 0; i < kGradWarps; ++i) all += wpi[i];
      const int m = t >> 4, r = t & 15;
      float w = 0.f;
      for (int i = 0; i <= m; ++i) w += rows_w[m * (m + 1) / 2 + i][r];
      for (int n = m + 1; n < 4; ++n) {
        for (int i = 0; i < m; ++i) w += rows_w[n * (n + 1) / 2 + i][0];
        w += cols_w[n * (n + 1) / 2 + m][r];
      }
      if (t < sl.n) {
        const int64_t at = ((int64_t)sl.tok + t) * a.H + h;
        a.dg[(int64_t)ns * a.dg_size + at] = (all * (nch == 2 ? whole[0] * whole[1] : whole[0]) + from) + (upto + w);
        if (ns == 0) a.dbeta[at] = dde[t];
      }
    }
    if (h + 1 < h1) {
      __syncthreads();  // the factors are used up
      copy_small(h + 1, 0);
    }
    cp_async_commit();
  }
  // dq and dk: rows of the group, or this split's part of them
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int t = r0 + 8 * hh, n = n0 + quarter * (NS / 4) + 8 * i + 2 * (lane & 3);
        if (t >= sl.n || n >= a.N) continue;
        const float x = (w ? dk : dq)[i][2 * hh], y = (w ? dk : dq)[i][2 * hh + 1];
        const int64_t o = (((int64_t)sl.tok + t) * a.G + grp) * a.N + n;
        if (a.splits > 1) {
          float* d = a.part + (int64_t)(2 * split + w) * a.part_size + o;
          d[0] = x;
          if (n + 1 < a.N) d[1] = y;
        } else {
          T* d = static_cast<T*>(w ? a.dk : a.dq) + o;
          if (n + 1 < a.N && a.pair) {
            if constexpr (sizeof(T) == 2) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
              *reinterpret_cast<__nv_bfloat162*>(d) = b;
            } else {
              *reinterpret_cast<float2*>(d) = make_float2(x, y);
            }
          } else {
            d[0] = from_f<T>(x);
            if (n + 1 < a.N) d[1] = from_f<T>(y);
          }
        }
      }
}

// dg from the parts of the slices of the columns n, in order.
__global__ void __launch_bounds__(256) k_delta_dg(const float* __restrict__ part, int slices, int64_t n, float* dg) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float x = 0.f;
  for (int s = 0; s < slices; ++s) x += part[s * n + i];
  dg[i] = x;
}

// dq and dk from the splits' parts, in order.
template <typename T>
__global__ void __launch_bounds__(256) k_delta_sum(const float* __restrict__ part, int splits, int64_t n, T* dq, T* dk) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float q = 0.f, k = 0.f;
  for (int s = 0; s < splits; ++s) q += part[2 * s * n + i], k += part[(2 * s + 1) * n + i];
  dq[i] = from_f<T>(q), dk[i] = from_f<T>(k);
}

template <typename T, int NT>
cudaError_t launch_grads_nt(const GradArgs& a, cudaStream_t stream) {
  constexpr int smem = GradTiles<T, NT>::kBytes;
  static_assert(smem <= 220 * 1024, "shared memory");
  static std::atomic<uint64_t> seen{0};
  return launch_kernel(k_delta_grads<T, NT>, seen, (unsigned)(a.slots_n * a.G * a.nslices * a.splits), kGradThreads, smem, smem,
                       false, stream, a);
}

template <typename T>
int grad_slices(int64_t N) {
  return N <= 64 ? 1 : N <= 128 ? 128 / GradTiles<T, 128>::kNS : 256 / GradTiles<T, 256>::kNS;
}

template <typename T>
cudaError_t launch_grads(const GradArgs& a, float* dg, cudaStream_t stream) {
  cudaError_t e = a.N <= 64    ? launch_grads_nt<T, 64>(a, stream)
                  : a.N <= 128 ? launch_grads_nt<T, 128>(a, stream)
                               : launch_grads_nt<T, 256>(a, stream);
  if (e != cudaSuccess) return e;
  if (a.nslices > 1) {
    k_delta_dg<<<(unsigned)((a.dg_size + 255) / 256), 256, 0, stream>>>(a.dg, a.nslices, a.dg_size, dg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.splits > 1) {
    k_delta_sum<T><<<(unsigned)((a.part_size + 255) / 256), 256, 0, stream>>>(a.part, a.splits, a.part_size,
                                                                             static_cast<T*>(a.dq), static_cast<T*>(a.dk));
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace delta
}  // namespace ssd
