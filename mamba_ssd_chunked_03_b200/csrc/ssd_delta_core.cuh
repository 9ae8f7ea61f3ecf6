// The chunk machinery that the gated delta rule's walks share: the tiles of a
// 32-token chunk in shared memory and the warps that make them.
//
// Within a chunk, with cs_t the cumulative sum of g, Gam_ts = exp(cs_t - cs_s)
// for s <= t, S the state that enters and C = 32:
//
//   forward walk   E = (I + A)^-1 (V - exp(cs) K S^T),  A_ts = Gam_ts beta_s k_t.k_s  (s < t)
//                  U = beta E:  y = scale exp(cs) Q S^T + M U,  M_ts = scale Gam_ts q_t.k_s  (s <= t)
//                  S' = exp(cs_C) S + sum_s exp(cs_C - cs_s) u_s k_s^T
//   reverse walk   D = (I + A)^-T (M^T dY + exp(cs_C - cs) K dS^T),  A_ts = Gam_ts beta_t k_t.k_s
//                  dS' = exp(cs_C) dS + sum_t (scale exp(cs_t) dy_t q_t^T - beta_t exp(cs_t) d_t k_t^T)
//
// (E is v minus what the state already answers to k; D is the gradient of u.)
// (I + A)^-1, M and the factors need no state: four warps of a CTA make them
// one chunk ahead of the warps that carry the state.
#pragma once

#include "ssd_delta.cuh"

namespace ssd {
namespace delta {

constexpr int kPrepWarps = 4, kPrepThreads = 32 * kPrepWarps;
constexpr int kStateWarps = 4, kStateThreads = 32 * kStateWarps;
constexpr int kThreads = kPrepThreads + kStateThreads;
constexpr int kP = 16 * kStateWarps;  // headdim rows of a CTA, 16 a warp
constexpr int kAP = 36;               // row pitch of the fp32 scratch tiles

struct WalkArgs {
  int64_t L, H, G, P, N, hpg;
  int slices;       // CTAs over headdim
  int n_units;      // (run, head, slice) units
  float scale;
  const void* q;
  const void* k;
  const void* v;    // forward: v; reverse: dy
  const float* g;
  const float* beta;
  const float* s0;  // state a run starts from (reverse: gradient of the final state), or null
  const Run* runs;  // or null: a run for each row
  void* out;        // forward: y; state walk: E (fp32); reverse: dv
  float* out_f;     // reverse: D (fp32)
  float* check;     // state at every 64th token of a run (state walk, reverse)
  float* fin;       // final state (forward) or gradient of the initial state (reverse), or null
  int qk_vec, v_vec, out_vec;  // rows start on 16-byte boundaries
};

template <typename T, int NT, bool STAGED>
struct Tiles {
  static constexpr int kTerms = sizeof(T) == 2 ? 1 : 2;  // fp16 terms of q, k and M
  static constexpr int kVP = sizeof(T) == 2 ? kP + 8 : kP + 4;  // row pitch of the V tile
  static constexpr int kTile = kC * NT * 2;
  static constexpr int kSq = kC * kC * 2;
  static constexpr int kK = 0;                               // [2 buffers][terms]
  static constexpr int kQ = kK + 2 * kTerms * kTile;
  static constexpr int kT = kQ + 2 * kTerms * kTile;         // [2][hi, lo]
  static constexpr int kM = kT + 2 * 2 * kSq;                // [2][hi, lo]
  static constexpr int kV = kM + 2 * 2 * kSq;                // [3]
  static constexpr int kVTile = kC * kVP * (int)sizeof(T);
  static constexpr int kRaw = kV + 3 * kVTile;               // [2][k, q]
  static constexpr int kRawTile = STAGED ? kC * NT * (int)sizeof(T) : 0;
  static constexpr int kA = kRaw + 4 * kRawTile;             // fp32 scratch, two tiles
  static constexpr int kStage = kA + 2 * kC * kAP * 4;       // a warp's output tile, fp32 pitch 20
  static constexpr int kFac = kStage + kStateWarps * kC * 20 * 4;  // [2] Factors
  static constexpr int kBytes = kFac + 2 * 1024 + 768;
};

// Per-token factors of a chunk (the powers of two of the operand rows are in them).
struct alignas(16) Factors {
  float kc[kC];   // forward: exp(cs) / k scale;  reverse: exp(cs_C - cs) / k scale
  float qc[kC];   // forward: scale exp(cs) / q scale;  reverse: the same
  float uc[kC];   // forward: exp(cs_C - cs) beta / k scale;  reverse: -beta exp(cs) / k scale
  float tau[kC];  // 1 / scale of the rows of (I + A)^-1
  float mu[kC];   // 1 / scale of the rows of M
  float beta[kC];
  float whole;    // exp(cs_C)
};
static_assert(sizeof(Factors) <= 1024, "Factors overlap");

struct PrepScratch {
  double cs[kC];
  float ik[kC], iq[kC];
  float beta[kC];
};
static_assert(sizeof(PrepScratch) <= 768, "PrepScratch overlaps");

__device__ __forceinline__ void prep_sync() { sm100::named_barrier_sync(1, kPrepThreads); }

// What the prep warps know of their run.
template <typename T>
struct PrepSrc {
  const T* k;  // rows of the run's first token, this head's group
  const T* q;
  const T* v;  // this head, this slice's first column
  const float* g;
  const float* beta;
  int len, P;  // columns of V that exist in this slice
};

// Enqueue the copies of chunk j's raw tiles (k and q when STAGED, v always);
// rows behind the run's end and columns behind N or P become zeros.
template <typename T, int NT, bool STAGED>
__device__ __forceinline__ void prep_issue(const WalkArgs& a, const PrepSrc<T>& s, int j, char* sm, uint32_t smu, int pt) {
  using L = Tiles<T, NT, STAGED>;
  constexpr int E = 16 / (int)sizeof(T);
  const int n = s.len - j * kC;  // rows that exist (<= 0: none)
  if (STAGED && n > 0) {
    constexpr int PC = NT / E;
#pragma unroll 4
    for (int i = pt; i < kC * PC; i += kPrepThreads) {
      const int row = i / PC, c = i % PC;
      const bool ok = row < n && c * E < a.N;
      const int64_t off = ok ? (int64_t)(j * kC + row) * a.G * a.N + c * E : 0;
      const uint32_t dst = smu + L::kRaw + (j & 1) * 2 * L::kRawTile + i * 16;
      cp_async16(dst, s.k + off, ok);
      cp_async16(dst + L::kRawTile, s.q + off, ok);
    }
  }
  if (n > 0) {
    const uint32_t vo = L::kV + (j % 3) * L::kVTile;
    if (a.v_vec) {
      constexpr int PC = kP / E;
#pragma unroll 2
      for (int i = pt; i < kC * PC; i += kPrepThreads) {
        const int row = i / PC, c = i % PC;
        const bool ok = row < n && c * E < s.P;
        const int64_t off = ok ? (int64_t)(j * kC + row) * a.H * a.P + c * E : 0;
        cp_async16(smu + vo + (row * L::kVP + c * E) * (int)sizeof(T), s.v + off, ok);
      }
    } else {
      T* dst = reinterpret_cast<T*>(sm + vo);
      for (int i = pt; i < kC * kP; i += kPrepThreads) {
        const int row = i / kP, p = i % kP;
        dst[row * L::kVP + p] =
            row < n && p < s.P ? s.v[(int64_t)(j * kC + row) * a.H * a.P + p] : from_f<T>(0.f);
      }
    }
  }
  cp_async_commit();
}

// One row of q or k as fp16 terms; returns 1 / its scale (the same in every lane).
template <typename T, int NT, bool STAGED>
__device__ __forceinline__ float prep_row(const T* src, bool exists, int64_t N, int vec, char* tile, int row, int lane) {
  using L = Tiles<T, NT, STAGED>;
  constexpr int E = NT / 32;  // columns of a lane
  float x[E];
  const int n0 = lane * E;
  if constexpr (STAGED) {
    if constexpr (E == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(src + n0);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src + n0 + e);
        x[e] = __uint_as_float(w << 16), x[e + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (exists) {
      bool done = false;
      if constexpr (sizeof(T) == 4) {
        if (vec) {
          done = true;
          if constexpr (E >= 4) {
#pragma unroll
            for (int e = 0; e < E; e += 4)
              if (n0 + e < N) {
                const float4 f = *reinterpret_cast<const float4*>(src + n0 + e);
                x[e] = f.x, x[e + 1] = f.y, x[e + 2] = f.z, x[e + 3] = f.w;
              }
          } else if (n0 < N) {
            const float2 f = *reinterpret_cast<const float2*>(src + n0);
            x[0] = f.x, x[1] = f.y;
          }
        }
      }
      if (!done) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (n0 + e < N) x[e] = to_f(src[n0 + e]);
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(x[e]));
  float inv;
  const float sc = pow2_scale(warp_absmax(m), inv);
  uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    if constexpr (L::kTerms == 1) hi[e] = pack2(x[2 * e] * sc, x[2 * e + 1] * sc);
    else split2(x[2 * e] * sc, x[2 * e + 1] * sc, hi[e], lo[e]);
  }
#pragma unroll
  for (int t = 0; t < L::kTerms; ++t) {
    char* d = tile + t * L::kTile + tile_off<NT>(row, n0);
    const uint32_t* w = t ? lo : hi;
    if constexpr (E == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(d) = w[0];
  }
  return inv;
}

// (I + A)^-1 of a 32 x 32 unit lower triangular matrix by one warp: the two
// 16 x 16 diagonal blocks by forward substitution, a column in each lane of a
// half warp, then T21 = -T22 A21 T11.  A is read below its diagonal only.
__device__ __forceinline__ void inverse32(const float* A, float* Tm, int lane) {
  const int j = lane & 15, h = lane >> 4;
  const float* Ah = A + h * (16 * kAP + 16);
  float t[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int s = 0; s < r; ++s) {
      const float av = Ah[r * kAP + s];
      if (s & 1) s1 = fmaf(av, t[s], s1);
      else s0 = fmaf(av, t[s], s0);
    }
    t[r] = (r == j ? 1.f : 0.f) - (s0 + s1);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) Tm[(16 * h + r) * kAP + 16 * h + j] = t[r];
  __syncwarp();
  // X = A21 T11: this lane's column j, rows 8h..8h+7
  float x[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) x[r] = 0.f;
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    const float ts = Tm[s * kAP + j];
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = fmaf(A[(16 + 8 * h + r) * kAP + s], ts, x[r]);
  }
  float y[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) y[r] = 0.f;
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    const float xs = __shfl_sync(0xffffffffu, x[s & 7], (s >> 3) * 16 + j);
#pragma unroll
    for (int r = 0; r < 8; ++r) y[r] = fmaf(Tm[(16 + 8 * h + r) * kAP + 16 + s], xs, y[r]);
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) Tm[(16 + 8 * h + r) * kAP + j] = -y[r];
}

// Everything of chunk j that needs no state, into buffer j & 1.  Called by the
// prep warps after chunk j's copies; ends without a barrier.
template <typename T, int NT, bool STAGED, bool REV, bool WITH_Q>
__device__ __forceinline__ void prep_chunk(const WalkArgs& a, const PrepSrc<T>& s, int j, float gv, float bv, char* sm,
                                           uint32_t smu, int pw, int lane) {
  using L = Tiles<T, NT, STAGED>;
  const int buf = j & 1, n = s.len - j * kC;
  Factors& f = reinterpret_cast<Factors*>(sm + L::kFac)[buf];
  PrepScratch& ps = *reinterpret_cast<PrepScratch*>(sm + L::kFac + 2 * sizeof(Factors));
  char* kt = sm + L::kK + buf * L::kTerms * L::kTile;
  char* qt = sm + L::kQ + buf * L::kTerms * L::kTile;
  if (pw == 0) {  // cumulative decays, in 64 bits: only their differences are used
    double c = decay_log(gv);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += up;
    }
    ps.cs[lane] = c;
    ps.beta[lane] = bv;
    f.beta[lane] = bv;
  }
#pragma unroll 4
  for (int r = pw; r < kC; r += kPrepWarps) {
    const T* kr;
    const T* qr;
    if constexpr (STAGED) {
      kr = reinterpret_cast<const T*>(sm + L::kRaw + buf * 2 * L::kRawTile) + r * NT;
      qr = reinterpret_cast<const T*>(sm + L::kRaw + (buf * 2 + 1) * L::kRawTile) + r * NT;
    } else {
      kr = s.k + (int64_t)(j * kC + r) * a.G * a.N;
      qr = s.q + (int64_t)(j * kC + r) * a.G * a.N;
    }
    const float ik = prep_row<T, NT, STAGED>(kr, r < n, a.N, a.qk_vec, kt, r, lane);
    if (lane == 0) ps.ik[r] = ik;
    if constexpr (WITH_Q) {
      const float iq = prep_row<T, NT, STAGED>(qr, r < n, a.N, a.qk_vec, qt, r, lane);
      if (lane == 0) ps.iq[r] = iq;
    }
  }
  prep_sync();
  float* As = reinterpret_cast<float*>(sm + L::kA);
  float* Ts = As + kC * kAP;
  // k k^T by warps 0, 1 and q k^T by warps 2, 3: 16 rows each, below the diagonal
  const bool isq = pw >= 2;
  const int mt = pw & 1;
  if (WITH_Q || !isq) {
    const uint32_t at = smu + (isq ? L::kQ : L::kK) + buf * L::kTerms * L::kTile;
    const uint32_t bt = smu + L::kK + buf * L::kTerms * L::kTile;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    const int ar = mt * 16 + (lane & 15), ac = (lane >> 4) * 8;
    const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
#pragma unroll 2
    for (int kk = 0; kk < NT; kk += 16) {
      uint32_t A[L::kTerms][4];
#pragma unroll
      for (int t = 0; t < L::kTerms; ++t) ldsm4(at + t * L::kTile + tile_off<NT>(ar, kk + ac), A[t]);
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        if (np > mt) break;
        uint32_t B[L::kTerms][4];
#pragma unroll
        for (int t = 0; t < L::kTerms; ++t) ldsm4(bt + t * L::kTile + tile_off<NT>(np * 16 + br, kk + bc), B[t]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma(acc[2 * np + i], A[0], B[0][2 * i], B[0][2 * i + 1]);
          if constexpr (L::kTerms == 2) {
            mma(acc[2 * np + i], A[0], B[1][2 * i], B[1][2 * i + 1]);
            mma(acc[2 * np + i], A[1], B[0][2 * i], B[0][2 * i + 1]);
          }
        }
      }
    }
    // Gam and the factors of rows and columns
    const int r0 = mt * 16 + (lane >> 2);
    float rmax[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= 2 * mt + 2) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = r0 + (e >> 1) * 8, c = i * 8 + 2 * (lane & 3) + (e & 1);
        float w = 0.f;
        if (isq ? c <= t : c < t) {
          w = expf((float)(ps.cs[t] - ps.cs[c])) * acc[i][e] * ps.ik[c];
          if (isq) w *= a.scale * ps.iq[t] * (REV ? 1.f : ps.beta[c]);
          else w *= ps.ik[t] * (REV ? ps.beta[t] : ps.beta[c]);
        }
        acc[i][e] = w;
        rmax[e >> 1] = fmaxf(rmax[e >> 1], fabsf(w));
      }
    }
    if (!isq) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= 2 * mt + 2) break;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          *reinterpret_cast<float2*>(As + (r0 + 8 * hh) * kAP + i * 8 + 2 * (lane & 3)) =
              make_float2(acc[i][2 * hh], acc[i][2 * hh + 1]);
      }
    } else {
      char* mtile = sm + L::kM + buf * 2 * L::kSq;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float inv;
        const float sc = pow2_scale(quad_max(rmax[hh]), inv);
        if ((lane & 3) == 0) f.mu[r0 + 8 * hh] = inv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= 2 * mt + 2) break;
          uint32_t hi, lo;
          split2(acc[i][2 * hh] * sc, acc[i][2 * hh + 1] * sc, hi, lo);
          const uint32_t o = tile_off<32>(r0 + 8 * hh, i * 8 + 2 * (lane & 3));
          *reinterpret_cast<uint32_t*>(mtile + o) = hi;
          if (REV || L::kTerms == 2) *reinterpret_cast<uint32_t*>(mtile + L::kSq + o) = lo;
        }
      }
    }
  }
  prep_sync();
  if (pw == 0) {
    inverse32(As, Ts, lane);
  } else if (pw == 1) {
    const double c = ps.cs[lane], end = ps.cs[31];
    const float into = expf((float)c), outof = expf((float)(end - c)), ik = ps.ik[lane], bt = ps.beta[lane];
    f.kc[lane] = (REV ? outof : into) * ik;
    if constexpr (WITH_Q) f.qc[lane] = a.scale * into * ps.iq[lane];
    f.uc[lane] = (REV ? -into : outof) * bt * ik;
    if (lane == 0) f.whole = expf((float)end);
  }
  prep_sync();
  // rows of the inverse as hi + lo
  char* tt = sm + L::kT + buf * 2 * L::kSq;
#pragma unroll
  for (int i = 0; i < kC / kPrepWarps; ++i) {
    const int r = pw + i * kPrepWarps;
    const float w = r < 16 && lane >= 16 ? 0.f : Ts[r * kAP + lane];
    float inv;
    const float sc = pow2_scale(warp_absmax(fabsf(w)), inv);
    const __half hi = __float2half_rn(w * sc);
    const __half lo = __float2half_rn(w * sc - __half2float(hi));
    const uint32_t o = tile_off<32>(r, lane);
    *reinterpret_cast<__half*>(tt + o) = hi;
    *reinterpret_cast<__half*>(tt + L::kSq + o) = lo;
    if (lane == 0) f.tau[r] = inv;
  }
}

}  // namespace delta
}  // namespace ssd
