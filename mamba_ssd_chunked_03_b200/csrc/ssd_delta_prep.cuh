// What a chunk of the gated delta rule needs besides the state, prepared for
// all chunks at once.
//
// Within a chunk of C = 32 tokens, with cs_t the cumulative sum of g,
// Gam_ts = exp(cs_t - cs_s) for s <= t and S the state that enters:
//
//   forward walk   E = (I + A)^-1 (V - exp(cs) K S^T),  A_ts = Gam_ts beta_s k_t.k_s  (s < t)
//                  U = beta E:  y = scale exp(cs) Q S^T + M U,  M_ts = scale Gam_ts q_t.k_s  (s <= t)
//                  S' = exp(cs_C) S + sum_s exp(cs_C - cs_s) u_s k_s^T
//   reverse walk   D = (I + A)^-T (M^T dY + exp(cs_C - cs) K dS^T),  A_ts = Gam_ts beta_t k_t.k_s
//                  dS' = exp(cs_C) dS + sum_t (scale exp(cs_t) dy_t q_t^T - beta_t exp(cs_t) d_t k_t^T)
//
// (E is v minus what the state already answers to k; D is the gradient of u.)
// The inverse, M and the factors need no state; only the products with S have
// to run one chunk after the other.  k_delta_prep makes them for every chunk
// and head, and the walks read them as they stand: tile images (fp16 terms,
// rows permuted for ldmatrix) and factors.  Preparing them inside the walk, by
// warps beside the state's, was measured first: at 7300 clocks a chunk, nearly
// all of it dependent instructions of one warp, it set the walk's pace (the
// state's own chain takes 4300).
//
// One CTA takes a chunk and a group of q and k: the tiles, k k^T and q k^T
// once (tensor cores), then a head a warp: the decays by a scan in 64 bits,
// A, its inverse by substitution with a row in each lane (496 steps of one
// FMA, the column of A broadcast from shared memory), M.  Bound by issue and
// the latency of shared memory in the substitution (issue slots 41 % busy, six
// CTAs an SM): b8 L2048 H80 N128, 40960 heads of chunks (368 MB
// written), 160 us, 2.3 TB/s.
#pragma once

#include "ssd_delta.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace delta {

constexpr int kPrepThreads = 128;
constexpr int kGP = 36;  // row pitch of the fp32 32 x 32 tiles

// Per-token factors of a chunk (the powers of two of the operand tiles' rows are in them).
struct alignas(16) Factors {
  float kc[kC];   // forward: exp(cs) / k scale;  reverse: exp(cs_C - cs) / k scale
  float qc[kC];   // scale exp(cs) / q scale
  float uc[kC];   // forward: exp(cs_C - cs) beta / k scale;  reverse: -beta exp(cs) / k scale
  float tau[kC];  // 1 / scale of the rows of the inverse (forward: times 1 / norm)
  float mu[kC];   // 1 / scale of the rows of M
  float beta[kC];
  float whole;     // exp(cs_C)
  float norm;      // forward: a power of two that no row sum of the inverse's magnitudes exceeds
  float ucm, qcm;  // largest magnitudes of uc and qc
};

// What the gradients need of a chunk's decays besides (kept beside the reverse
// walk's tiles).
struct alignas(16) Decays {
  double cs[kC];               // cumulative log2 decay
  float into[kC], outof[kC];   // exp(cs), exp(cs_C - cs)
  float inv[kC];               // 1 / exp(cs), if `plain`
  float ik[kC], iq[kC];        // 1 / scale of the rows of k and q
  int plain;                   // exp(cs_t - cs_s) is into_t inv_s
  int pad[3];
};

// Sizes of the images, in bytes.
constexpr int kSq = kC * kC * 2;  // a 32 x 32 fp16 tile
template <typename T, int NT>
struct TokenTiles {  // a chunk's k, then q, terms of each: one set for a group
  static constexpr int kTerms = sizeof(T) == 2 ? 1 : 2;
  static constexpr int kTile = kC * NT * 2;
  static constexpr int kBytes = 2 * kTerms * kTile;
};
// A head's: the inverse (hi, lo), M (terms), Factors; DECAYS: and, not copied by the walk, Decays.
template <int MTERMS, bool DECAYS = false>
struct HeadTiles {
  static constexpr int kM = 2 * kSq, kF = kM + MTERMS * kSq, kBytes = kF + (int)sizeof(Factors);
  static constexpr int kStride = kBytes + (DECAYS ? (int)sizeof(Decays) : 0);
};
using RevTiles = HeadTiles<2, true>;
static_assert(HeadTiles<2>::kBytes % 16 == 0, "16-byte copies");

struct PrepArgs {
  int64_t L, H, G, N, hpg;
  int per_row;       // chunks of a row, without a list
  int splits;        // CTAs that share the heads of a group
  int heads;         // heads of each of them
  float scale;
  const void* q;
  const void* k;
  const float* g;
  const float* beta;
  const Chunk* chunks;  // or null
  char* tokens;         // [chunk][group] TokenTiles
  char* fwd;            // [chunk][head] HeadTiles of the forward walk, or null
  char* rev;            // [chunk][head] HeadTiles of the reverse walk, or null
  int vec;              // rows of q and k start on 16-byte boundaries
};

__device__ __forceinline__ float absmax_bits(uint32_t m) { return __uint_as_float(__reduce_max_sync(0xffffffffu, m)); }

// A thread's 16 bytes of a row of q or k (columns c..), zeros behind N.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* s, int c, int64_t N, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const uint4*>(s));
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 2) {
      const unsigned short* u = reinterpret_cast<const unsigned short*>(s);
      w[e] = (c + 2 * e < N ? (uint32_t)u[2 * e] : 0u) | (c + 2 * e + 1 < N ? (uint32_t)u[2 * e + 1] << 16 : 0u);
    } else {
      w[e] = c + e < N ? __float_as_uint(s[e]) : 0u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The inverse's row of this lane (t[s], unit lower triangular) as hi + lo; 1 / its scale.
__device__ __forceinline__ float store_row(const float (&t)[kC], int lane, char* hi_tile, char* lo_tile) {
  float m = 0.f;
#pragma unroll
  for (int s = 0; s < kC; ++s) m = fmaxf(m, fabsf(t[s]));
  float inv;
  const float sc = pow2_scale(m, inv);
#pragma unroll
  for (int c = 0; c < kC; c += 8) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(mul2(t[c + 2 * e], t[c + 2 * e + 1], sc), hi[e], lo[e]);
    const uint32_t o = tile_off<32>(lane, c);
    *reinterpret_cast<uint4*>(hi_tile + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(lo_tile + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return inv;
}

// FWD, REV: which walk's tiles are made.
template <typename T, int NT, bool FWD, bool REV>
__global__ void __launch_bounds__(kPrepThreads, NT * sizeof(T) <= 256 ? 6 : 3) k_delta_prep(const PrepArgs a) {
  using X = TokenTiles<T, NT>;
  constexpr bool kFwdM = !REV;  // the backward's forward walk makes no y
  using HF = HeadTiles<kFwdM ? 2 : 0>;
  using HR = RevTiles;
  constexpr int E = 16 / (int)sizeof(T), PC = NT / E, V = kC * NT / E / kPrepThreads;
  extern __shared__ __align__(128) char sm[];
  float* gk = reinterpret_cast<float*>(sm);  // k k^T, q k^T: true values
  float* gq = gk + kC * kGP;
  char* const tiles = sm + 2 * kC * kGP * 4;                // k and q; when their products are formed,
  float* at = reinterpret_cast<float*>(tiles);              // a warp's A, transposed
  __shared__ __align__(8) float iscale[2][kC];     // 1 / scale of the rows of k and q
  __shared__ uint32_t parts[2][kC][2];         // of a row that lies across two warps
  __shared__ __align__(16) float col[kPrepThreads / 32][2][kC];
  __shared__ double css[kPrepThreads / 32][kC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits;
  const int64_t cg = blockIdx.x / a.splits, grp = cg % a.G, ch = cg / a.G;
  Chunk c;
  if (a.chunks) {
    c = a.chunks[ch];
  } else {
    const int j = (int)(ch % a.per_row);
    c.tok = (int)(ch / a.per_row * a.L + (int64_t)j * kC);
    c.n = a.L - (int64_t)j * kC < kC ? (int)(a.L - (int64_t)j * kC) : kC;
  }
  if (c.n == 0) return;
  const uint32_t smu = sm100::smem_u32(tiles);
  // The tiles of k and q: fp16, each row scaled by its largest magnitude, so that
  // a token's bits do not depend on the tokens beside it.
  {
    const int row0 = threadIdx.x / PC, cc = (threadIdx.x % PC) * E;
    constexpr int kStep = kPrepThreads / PC;
    char* out = a.tokens + (ch * a.G + grp) * X::kBytes;
    uint4 raw[2][V];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const T* src = static_cast<const T*>(w ? a.q : a.k) + ((int64_t)c.tok * a.G + grp) * a.N + cc;
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const int row = row0 + x * kStep;
        raw[w][x] = row < c.n && cc < a.N ? load_piece<T>(src + (int64_t)row * a.G * a.N, cc, a.N, a.vec)
                                          : make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t most[2][V];  // a row's largest magnitude: the bits of magnitudes order as they do
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const uint32_t u[4] = {raw[w][x].x, raw[w][x].y, raw[w][x].z, raw[w][x].w};
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 2) m = __vmaxu2(m, u[e] & 0x7fff7fffu);
          else m = max(m, u[e] & 0x7fffffffu);
        }
        if constexpr (sizeof(T) == 2) m = max(m << 16, m & 0xffff0000u);
#pragma unroll
        for (int o = 1; o < PC && o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if constexpr (PC > 32) {
          if (lane == 0) parts[w][row0 + x * kStep][warp & 1] = m;
        }
        most[w][x] = m;
      }
    if constexpr (PC > 32) __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const int row = row0 + x * kStep;
        if constexpr (PC > 32) most[w][x] = max(parts[w][row][0], parts[w][row][1]);
        float inv;
        const float sc = pow2_unit(__uint_as_float(most[w][x]), inv);
        if (cc == 0) iscale[w][row] = inv;
        const uint32_t u[4] = {raw[w][x].x, raw[w][x].y, raw[w][x].z, raw[w][x].w};
        const uint32_t o = w * X::kTerms * X::kTile + tile_off<NT>(row, cc);
        if constexpr (sizeof(T) == 2) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = pack2(__fmul2_rn(bf16x2(u[e]), make_float2(sc, sc)));
          const uint4 p = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(tiles + o) = p;
          if (split == 0) *reinterpret_cast<uint4*>(out + o) = p;
        } else {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            split2(mul2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]), sc), hi[e], lo[e]);
          *reinterpret_cast<uint2*>(tiles + o) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(tiles + o + X::kTile) = make_uint2(lo[0], lo[1]);
          if (split == 0) {
            *reinterpret_cast<uint2*>(out + o) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(out + o + X::kTile) = make_uint2(lo[0], lo[1]);
          }
        }
      }
    __syncthreads();
  }
  {  // k k^T by warps 0, 1 and q k^T by warps 2, 3, 16 rows each; the columns above the diagonal are not used
    const bool isq = warp >= 2;
    const int mt = warp & 1;
    const uint32_t ab = smu + (isq ? X::kTerms * X::kTile : 0);
    float acc[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    const int ar = mt * 16 + (lane & 15), ac = (lane >> 4) * 8;
    const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
#pragma unroll 4
    for (int kk = 0; kk < NT; kk += 16) {
      uint32_t A[X::kTerms][4], B[X::kTerms][2][4];
#pragma unroll
      for (int t = 0; t < X::kTerms; ++t) {
        ldsm4(ab + t * X::kTile + tile_off<NT>(ar, kk + ac), A[t]);
#pragma unroll
        for (int np = 0; np < 2; ++np) ldsm4(smu + t * X::kTile + tile_off<NT>(np * 16 + br, kk + bc), B[t][np]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(acc[n], A[0], B[0][n >> 1][2 * (n & 1)], B[0][n >> 1][2 * (n & 1) + 1]);
      if constexpr (X::kTerms == 2) {
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(acc[n], A[0], B[1][n >> 1][2 * (n & 1)], B[1][n >> 1][2 * (n & 1) + 1]);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma(acc[n], A[1], B[0][n >> 1][2 * (n & 1)], B[0][n >> 1][2 * (n & 1) + 1]);
      }
    }
    const float w0[2] = {iscale[isq][mt * 16 + (lane >> 2)], iscale[isq][mt * 16 + (lane >> 2) + 8]};
    float* dst = (isq ? gq : gk) + (mt * 16 + (lane >> 2)) * kGP + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float2 w1 = *reinterpret_cast<const float2*>(iscale[0] + 8 * n + 2 * (lane & 3));
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        *reinterpret_cast<float2*>(dst + 8 * hh * kGP + 8 * n) =
            make_float2(acc[n][2 * hh] * w0[hh] * w1.x, acc[n][2 * hh + 1] * w0[hh] * w1.y);
    }
    __syncthreads();
  }
  at += warp * kC * kGP;
  const float inv_k = iscale[0][lane], inv_q = iscale[1][lane];
  float* vb = col[warp][0];  // forward: beta / exp(cs);  reverse: 1 / exp(cs)
  double* cs = css[warp];
  const int64_t h1 = grp * a.hpg + ((int64_t)(split + 1) * a.heads < a.hpg ? (int64_t)(split + 1) * a.heads : a.hpg);
  for (int64_t h = grp * a.hpg + (int64_t)split * a.heads + warp; h < h1; h += kPrepThreads / 32) {
    const int64_t go = ((int64_t)c.tok + lane) * a.H + h;
    const bool live = lane < c.n;
    const float bt = live ? a.beta[go] : 0.f;
    double sum = decay_log2(live ? a.g[go] : 0.f);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // in 64 bits: only differences are used
      const double up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31);
    // decays within 2^+-100: exp(cs_t - cs_s) is the product of two fp32 numbers
    const bool plain = __all_sync(0xffffffffu, fabs(sum) <= 100.0);
    const float into = pow2_of(sum), outof = pow2_of(end - sum), inv = plain ? pow2_of(-sum) : 0.f;
#pragma unroll
    for (int dir = 0; dir < 2; ++dir) {
      if (dir == 0 ? !FWD : !REV) continue;
      const bool rev = dir == 1;
      char* img = rev ? a.rev + (ch * a.H + h) * HR::kStride : a.fwd + (ch * a.H + h) * HF::kStride;
      Factors* f = reinterpret_cast<Factors*>(img + (rev ? HR::kF : HF::kF));
      __syncwarp();
      vb[lane] = rev ? inv : inv * bt;
      cs[lane] = sum;
      col[warp][1][lane] = bt;
      __syncwarp();
      // w_c = exp(cs_t - cs_c) (beta_c) x (row t of a product), c + lim <= t; t is this lane's row
      const auto row = [&](const float* gram, float rowf, int lim, auto&& put) {
#pragma unroll
        for (int c0 = 0; c0 < kC; c0 += 4) {
          const float4 gv = *reinterpret_cast<const float4*>(gram + lane * kGP + c0);
          const float g4[4] = {gv.x, gv.y, gv.z, gv.w};
          if (plain) {
            const float4 bv = *reinterpret_cast<const float4*>(vb + c0);
            const float b4[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) put(c0 + e, c0 + e + lim <= lane ? (rowf * into) * b4[e] * g4[e] : 0.f);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float w = 0.f;
              if (c0 + e + lim <= lane)
                w = rowf * pow2_of(sum - cs[c0 + e]) * (rev ? 1.f : col[warp][1][c0 + e]) * g4[e];
              put(c0 + e, w);
            }
          }
        }
      };
      row(gk, rev ? bt : 1.f, 1, [&](int cidx, float w) { at[cidx * kGP + lane] = w; });
      __syncwarp();
      float t[kC];  // this lane's row of the inverse: t (I + A) = e
#pragma unroll
      for (int s = kC - 1; s >= 0; --s) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = kC - 4; r + 3 > s; r -= 4) {
          const float4 av = *reinterpret_cast<const float4*>(at + s * kGP + r);
          if (r + 3 > s) p[3] = fmaf(t[r + 3], av.w, p[3]);
          if (r + 2 > s) p[2] = fmaf(t[r + 2], av.z, p[2]);
          if (r + 1 > s) p[1] = fmaf(t[r + 1], av.y, p[1]);
          if (r > s) p[0] = fmaf(t[r], av.x, p[0]);
        }
        t[s] = (s == lane ? 1.f : 0.f) - ((p[0] + p[1]) + (p[2] + p[3]));
      }
      float tau = store_row(t, lane, img, img + kSq);
      const float uc = (rev ? -into : outof) * bt * inv_k, qc = a.scale * into * inv_q;
      const float ucm = absmax_bits(__float_as_uint(fabsf(uc))), qcm = absmax_bits(__float_as_uint(fabsf(qc)));
      float norm = 1.f;
      if (!rev) {
        float l1 = 0.f;
#pragma unroll
        for (int s = 0; s < kC; ++s) l1 += fabsf(t[s]);
        const uint32_t e = __float_as_uint(absmax_bits(__float_as_uint(l1))) >> 23;  // at least 127: the diagonal is 1
        norm = __uint_as_float((e < 252 ? e + 1 : 253) << 23);
        tau *= __uint_as_float((e < 252 ? 253 - e : 1) << 23);
      }
      f->tau[lane] = tau;
      f->kc[lane] = (rev ? outof : into) * inv_k;
      f->uc[lane] = uc;
      f->beta[lane] = bt;
      if (lane == 31) f->whole = into, f->norm = norm, f->ucm = ucm, f->qcm = qcm;
      if (rev || kFwdM) {
        row(gq, a.scale, 0, [&](int cidx, float w) { t[cidx] = w; });
        char* mi = img + (rev ? HR::kM : HF::kM);
        f->mu[lane] = store_row(t, lane, mi, mi + kSq);
        f->qc[lane] = qc;
        if (rev) {
          Decays* d = reinterpret_cast<Decays*>(img + HR::kBytes);
          d->cs[lane] = sum, d->into[lane] = into, d->outof[lane] = outof, d->inv[lane] = inv;
          d->ik[lane] = inv_k, d->iq[lane] = inv_q;
          if (lane == 0) d->plain = plain;
        }
      }
    }
  }
}

template <typename T, int NT, bool FWD, bool REV>
cudaError_t launch_prep_nt(PrepArgs& a, int64_t chunks, cudaStream_t stream) {
  constexpr int kHeads = kPrepThreads / 32 * kC * kGP * 4, kTok = TokenTiles<T, NT>::kBytes;
  constexpr int smem = (kTok > kHeads ? kTok : kHeads) + 2 * kC * kGP * 4;
  static_assert(smem <= 227 * 1024, "shared memory");
  // Heads of a group in one CTA share its tiles and products; they are spread
  // until every SM has some 24 CTAs, five at a time, so that the last ones
  // leave little idle, a head a warp at the least.
  const int64_t units = chunks * a.G, most = (a.hpg + 3) / 4;
  int64_t splits = (24 * 148 + units - 1) / units;
  splits = splits < 1 ? 1 : splits > most ? most : splits;
  a.heads = (int)((a.hpg + splits - 1) / splits);
  a.splits = (int)((a.hpg + a.heads - 1) / a.heads);
  static std::atomic<uint64_t> seen{0};
  return launch_kernel(k_delta_prep<T, NT, FWD, REV>, seen, (unsigned)(units * a.splits), kPrepThreads, smem, smem, false, stream, a);
}

template <typename T, bool FWD, bool REV>
cudaError_t launch_prep(PrepArgs& a, int64_t chunks, cudaStream_t stream) {
  if (a.N <= 64) return launch_prep_nt<T, 64, FWD, REV>(a, chunks, stream);
  if (a.N <= 128) return launch_prep_nt<T, 128, FWD, REV>(a, chunks, stream);
  return launch_prep_nt<T, 256, FWD, REV>(a, chunks, stream);
}

inline int64_t padded_n(int64_t N) { return N <= 64 ? 64 : N <= 128 ? 128 : 256; }
inline size_t token_tiles_bytes(const Shape& s) {
  return (size_t)s.chunks * s.G * 2 * (s.bf16 ? 1 : 2) * kC * padded_n(s.N) * 2;
}

}  // namespace delta
}  // namespace ssd
