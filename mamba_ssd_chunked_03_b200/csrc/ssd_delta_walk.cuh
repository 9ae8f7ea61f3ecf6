// The forward walk of the gated delta rule (see ssd_delta_core.cuh for the
// formulas): one CTA carries 64 rows (headdim) of one head's state through one
// sequence, 32 tokens at a time.
//
// Each of four state warps owns 16 rows p of the state for all N columns, in
// registers, as the accumulator tiles of the matrix instruction.  Every
// product of a chunk has m = p, so the result of one is the operand of the
// next without leaving the warp: K S^T (A = S), E (A = R), y (A = S and E),
// S' (A = U).  The warps share only the chunk's tiles, which four further
// warps prepare one chunk ahead; one barrier a chunk is all the
// synchronisation there is.
#pragma once

#include "ssd_delta_core.cuh"

namespace ssd {
namespace delta {

enum WalkMode { kForward = 0, kStates = 1 };

// The 16 x 32 (p x t) tile of a warp, held as accumulators, to rows t of `out`
// (row stride `stride` elements, `cols` of the 16 columns exist, n rows).
template <typename O>
__device__ __forceinline__ void store_tile(const float (&y)[4][4], char* stage, O* out, int64_t stride, int n, int cols,
                                           bool vec, int lane) {
  __syncwarp();
  if constexpr (sizeof(O) == 2) {
    const uint32_t base = sm100::smem_u32(stage);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t r[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * x + (m >> 1)][2 * (m & 1)], y[2 * x + (m >> 1)][2 * (m & 1) + 1]);
        r[m] = *reinterpret_cast<const uint32_t*>(&h);
      }
      const int m = lane >> 3;
      sm100::stmatrix_x4_trans(base + (8 * (2 * x + (m >> 1)) + (lane & 7)) * 48 + (m & 1) * 16, r);
    }
    __syncwarp();
    if (lane < n) {
      O* o = out + lane * stride;
      const char* s = stage + lane * 48;
#pragma unroll
      for (int c = 0; c < 16; c += 8) {
        if (vec && c + 8 <= cols) {
          *reinterpret_cast<uint4*>(o + c) = *reinterpret_cast<const uint4*>(s + c * 2);
        } else {
#pragma unroll 1
          for (int e = c; e < c + 8 && e < cols; ++e) o[e] = reinterpret_cast<const O*>(s)[e];
        }
      }
    }
  } else {
    float* s = reinterpret_cast<float*>(stage);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[(8 * i + 2 * (lane & 3) + (e & 1)) * 20 + (lane >> 2) + 8 * (e >> 1)] = y[i][e];
    __syncwarp();
    if (lane < n) {
      O* o = out + lane * stride;
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        if (vec && c + 4 <= cols) {
          *reinterpret_cast<float4*>(o + c) = *reinterpret_cast<const float4*>(s + lane * 20 + c);
        } else {
#pragma unroll 1
          for (int e = c; e < c + 4 && e < cols; ++e) o[e] = s[lane * 20 + e];
        }
      }
    }
  }
}

// State tiles from or to row-major (P, N) fp32 at `base` (row p0's first element).
template <int NT>
__device__ __forceinline__ void load_state(float (&S)[NT / 8][4], const float* base, int64_t N, int rows, int lane) {
#pragma unroll
  for (int i = 0; i < NT / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = (lane >> 2) + 8 * (e >> 1), n = 8 * i + 2 * (lane & 3) + (e & 1);
      S[i][e] = p < rows && n < N ? base[p * N + n] : 0.f;
    }
}
template <int NT>
__device__ __forceinline__ void store_state(const float (&S)[NT / 8][4], float s0, float s1, float* base, int64_t N,
                                            int rows, int lane) {
  const bool pair = N % 2 == 0 && reinterpret_cast<uintptr_t>(base) % 8 == 0;
#pragma unroll
  for (int i = 0; i < NT / 8; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = (lane >> 2) + 8 * h, n = 8 * i + 2 * (lane & 3);
      if (p >= rows || n >= N) continue;
      const float sc = h ? s1 : s0;
      float* d = base + p * N + n;
      if (pair) {
        *reinterpret_cast<float2*>(d) = make_float2(S[i][2 * h] * sc, S[i][2 * h + 1] * sc);
      } else {
        d[0] = S[i][2 * h] * sc;
        if (n + 1 < N) d[1] = S[i][2 * h + 1] * sc;
      }
    }
}

// The 16 x 32 (p x t) accumulator tile as scaled fp16 operand tiles (two k
// steps of 16 tokens), hi and, if asked for, lo; returns 1 / scale of rows r, r + 8.
template <bool LO>
__device__ __forceinline__ float2 to_operand(const float (&x)[4][4], uint32_t (&hi)[2][4], uint32_t (&lo)[2][4]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m0 = fmaxf(m0, fmaxf(fabsf(x[i][0]), fabsf(x[i][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(x[i][2]), fabsf(x[i][3])));
  }
  float2 inv;
  const float s0 = pow2_scale(quad_max(m0), inv.x), s1 = pow2_scale(quad_max(m1), inv.y);
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float s = a & 1 ? s1 : s0;
      const float u = x[2 * ks + (a >> 1)][2 * (a & 1)] * s, v = x[2 * ks + (a >> 1)][2 * (a & 1) + 1] * s;
      if constexpr (LO) split2(u, v, hi[ks][a], lo[ks][a]);
      else hi[ks][a] = pack2(u, v);
    }
  return inv;
}

// The V (or dY) tile as the accumulator layout: v[i][e] at (p, t).
template <typename T, int VP>
__device__ __forceinline__ void load_v(float (&v)[4][4], const char* tile, int p0, int lane) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t base = sm100::smem_u32(tile);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int m = lane >> 3;
      uint32_t r[4];
      ldsm4t(base + ((8 * (2 * x + (m >> 1)) + (lane & 7)) * VP + p0 + 8 * (m & 1)) * 2, r);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * x + (q >> 1)][2 * (q & 1)] = __uint_as_float(r[q] << 16);
        v[2 * x + (q >> 1)][2 * (q & 1) + 1] = __uint_as_float(r[q] & 0xffff0000u);
      }
    }
  } else {
    const float* s = reinterpret_cast<const float*>(tile);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[i][e] = s[(8 * i + 2 * (lane & 3) + (e & 1)) * VP + p0 + (lane >> 2) + 8 * (e >> 1)];
  }
}

__device__ __forceinline__ void zero(float (&x)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
}

// Row scales that bring the state to fp16 range: the scale, and 1 / scale.
template <int NT>
__device__ __forceinline__ void state_max(const float (&S)[NT / 8][4], float& m0, float& m1) {
  m0 = m1 = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 8; ++i) {
    m0 = fmaxf(m0, fmaxf(fabsf(S[i][0]), fabsf(S[i][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(S[i][2]), fabsf(S[i][3])));
  }
  m0 = quad_max(m0), m1 = quad_max(m1);
}

// S += Uhi/lo (p x t) times a 32 x NT tile of tokens (k or q; TERMS fp16 terms).
template <int NT, int TERMS>
__device__ __forceinline__ void state_add(float (&S)[NT / 8][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4],
                                          uint32_t tile, int lane) {
  constexpr int kTile = kC * NT * 2;
  const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, nc = (lane >> 4) * 8;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int np = 0; np < NT / 16; ++np) {
      uint32_t B[4];
      ldsm4t(tile + tile_off<NT>(16 * ks + tr, 16 * np + nc), B);
      mma(S[2 * np], hi[ks], B[0], B[1]);
      mma(S[2 * np + 1], hi[ks], B[2], B[3]);
      mma(S[2 * np], lo[ks], B[0], B[1]);
      mma(S[2 * np + 1], lo[ks], B[2], B[3]);
      if constexpr (TERMS == 2) {
        ldsm4t(tile + kTile + tile_off<NT>(16 * ks + tr, 16 * np + nc), B);
        mma(S[2 * np], hi[ks], B[0], B[1]);
        mma(S[2 * np + 1], hi[ks], B[2], B[3]);
      }
    }
}

template <typename T, int NT, bool STAGED, int MODE>
__global__ void __launch_bounds__(kThreads, NT <= 128 && sizeof(T) == 2 ? 2 : 1) k_delta_walk(const WalkArgs a) {
  using L = Tiles<T, NT, STAGED>;
  constexpr bool kY = MODE == kForward;
  extern __shared__ __align__(1024) char sm[];
  const uint32_t smu = sm100::smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices;
  const int64_t rh = blockIdx.x / a.slices, h = rh % a.H, ri = rh / a.H;
  Run run;
  if (a.runs) {
    run = a.runs[ri];
  } else {
    run.tok = ri * a.L, run.len = (int)a.L, run.fin = run.h0 = (int)ri;
    run.slot = ri * ((a.L + kCheck - 1) / kCheck);
  }
  const int nc = (run.len + kC - 1) / kC;
  const int p_cta = slice * kP;
  if (warp >= kStateWarps) {  // ---- the warps that prepare the tiles
    const int pw = warp - kStateWarps, pt = threadIdx.x - kStateThreads;
    const int64_t grp = h / a.hpg;
    PrepSrc<T> s;
    s.k = static_cast<const T*>(a.k) + (run.tok * a.G + grp) * a.N;
    s.q = static_cast<const T*>(a.q) + (run.tok * a.G + grp) * a.N;
    s.v = static_cast<const T*>(a.v) + (run.tok * a.H + h) * a.P + p_cta;
    s.g = a.g + run.tok * a.H + h;
    s.beta = a.beta + run.tok * a.H + h;
    s.len = run.len;
    s.P = (int)(a.P - p_cta < kP ? a.P - p_cta : kP);
    const auto gate = [&](int j, const float* src) {
      const int t = j * kC + lane;
      return pw == 0 && t < run.len ? src[t * a.H] : 0.f;
    };
    float gv = gate(0, s.g), bv = gate(0, s.beta);
    if (nc > 0) {
      prep_issue<T, NT, STAGED>(a, s, 0, sm, smu, pt);
      prep_issue<T, NT, STAGED>(a, s, 1, sm, smu, pt);
      cp_async_wait<1>();
      prep_sync();
      prep_chunk<T, NT, STAGED, false, kY>(a, s, 0, gv, bv, sm, smu, pw, lane);
    }
    gv = gate(1, s.g), bv = gate(1, s.beta);
    __syncthreads();
    for (int j = 0; j < nc; ++j) {
      if (j + 1 < nc) {
        const float g1 = gate(j + 2, s.g), b1 = gate(j + 2, s.beta);
        prep_issue<T, NT, STAGED>(a, s, j + 2, sm, smu, pt);
        cp_async_wait<1>();
        prep_sync();
        prep_chunk<T, NT, STAGED, false, kY>(a, s, j + 1, gv, bv, sm, smu, pw, lane);
        gv = g1, bv = b1;
      }
      __syncthreads();
    }
    return;
  }
  // ---- the warps that carry the state: rows p0..p0+15
  const int p0 = p_cta + 16 * warp;
  const int rows = a.P - p0 < 16 ? (int)(a.P - p0) : 16;  // may be negative: nothing is read or written
  float S[NT / 8][4];
  float sig0 = 1.f, sig1 = 1.f;  // the state's rows are S times these
  if (a.s0 && run.h0 >= 0) {
    load_state<NT>(S, a.s0 + (((int64_t)run.h0 * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
  } else {
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
  }
  char* stage = sm + L::kStage + warp * (kC * 20 * 4);
  const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
  __syncthreads();
  for (int j = 0; j < nc; ++j) {
    if (rows <= 0) {  // no such rows: only keep step
      __syncthreads();
      continue;
    }
    const int buf = j & 1;
    const Factors& f = reinterpret_cast<const Factors*>(sm + L::kFac)[buf];
    const uint32_t kt = smu + L::kK + buf * L::kTerms * L::kTile, qt = smu + L::kQ + buf * L::kTerms * L::kTile;
    const uint32_t tt = smu + L::kT + buf * 2 * L::kSq, mt = smu + L::kM + buf * 2 * L::kSq;
    if constexpr (MODE == kStates) {
      if ((j & 1) == 0)
        store_state<NT>(S, sig0, sig1, a.check + (((run.slot + (j >> 1)) * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
    }
    float m0, m1, inv0, inv1;
    state_max<NT>(S, m0, m1);
    const float sc0 = pow2_scale(m0, inv0), sc1 = pow2_scale(m1, inv1);
    inv0 *= sig0, inv1 *= sig1;
    float acc[4][4], yq[4][4];
    zero(acc);
    zero(yq);
#pragma unroll
    for (int ks = 0; ks < NT / 16; ++ks) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float sc = x & 1 ? sc1 : sc0;
        split2(S[2 * ks + (x >> 1)][2 * (x & 1)] * sc, S[2 * ks + (x >> 1)][2 * (x & 1) + 1] * sc, hi[x], lo[x]);
      }
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        uint32_t B[4];
        ldsm4(kt + tile_off<NT>(16 * np + br, 16 * ks + bc), B);
        mma(acc[2 * np], hi, B[0], B[1]);
        mma(acc[2 * np + 1], hi, B[2], B[3]);
        mma(acc[2 * np], lo, B[0], B[1]);
        mma(acc[2 * np + 1], lo, B[2], B[3]);
        if constexpr (L::kTerms == 2) {
          ldsm4(kt + L::kTile + tile_off<NT>(16 * np + br, 16 * ks + bc), B);
          mma(acc[2 * np], hi, B[0], B[1]);
          mma(acc[2 * np + 1], hi, B[2], B[3]);
        }
        if constexpr (kY) {
          ldsm4(qt + tile_off<NT>(16 * np + br, 16 * ks + bc), B);
          mma(yq[2 * np], hi, B[0], B[1]);
          mma(yq[2 * np + 1], hi, B[2], B[3]);
          if constexpr (L::kTerms == 2) {
            mma(yq[2 * np], lo, B[0], B[1]);
            mma(yq[2 * np + 1], lo, B[2], B[3]);
            ldsm4(qt + L::kTile + tile_off<NT>(16 * np + br, 16 * ks + bc), B);
            mma(yq[2 * np], hi, B[0], B[1]);
            mma(yq[2 * np + 1], hi, B[2], B[3]);
          }
        }
      }
    }
    const int tc = 2 * (lane & 3);
    uint32_t hi[2][4], lo[2][4];
    float e[4][4];
    float2 iv;
    {  // R = V - exp(cs) K S^T
      float v[4][4];
      load_v<T, L::kVP>(v, sm + L::kV + (j % 3) * L::kVTile, 16 * warp, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 kc = *reinterpret_cast<const float2*>(f.kc + 8 * i + tc);
        v[i][0] = fmaf(-(acc[i][0] * inv0), kc.x, v[i][0]);
        v[i][1] = fmaf(-(acc[i][1] * inv0), kc.y, v[i][1]);
        v[i][2] = fmaf(-(acc[i][2] * inv1), kc.x, v[i][2]);
        v[i][3] = fmaf(-(acc[i][3] * inv1), kc.y, v[i][3]);
      }
      iv = to_operand<true>(v, hi, lo);
    }
    zero(e);  // E = R (I + A)^-T, its lower triangle
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int np = ks; np < 2; ++np) {
        uint32_t B[4];
        ldsm4(tt + tile_off<32>(16 * np + br, 16 * ks + bc), B);
        mma(e[2 * np], hi[ks], B[0], B[1]);
        mma(e[2 * np + 1], hi[ks], B[2], B[3]);
        mma(e[2 * np], lo[ks], B[0], B[1]);
        mma(e[2 * np + 1], lo[ks], B[2], B[3]);
        ldsm4(tt + L::kSq + tile_off<32>(16 * np + br, 16 * ks + bc), B);
        mma(e[2 * np], hi[ks], B[0], B[1]);
        mma(e[2 * np + 1], hi[ks], B[2], B[3]);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 tau = *reinterpret_cast<const float2*>(f.tau + 8 * i + tc);
      e[i][0] *= iv.x * tau.x, e[i][1] *= iv.x * tau.y, e[i][2] *= iv.y * tau.x, e[i][3] *= iv.y * tau.y;
    }
    const int n = run.len - j * kC < kC ? run.len - j * kC : kC;
    const int64_t row0 = ((run.tok + (int64_t)j * kC) * a.H + h) * a.P + p0;
    if constexpr (kY) {
      iv = to_operand<L::kTerms == 2>(e, hi, lo);
      zero(acc);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int np = ks; np < 2; ++np) {
          uint32_t B[4];
          ldsm4(mt + tile_off<32>(16 * np + br, 16 * ks + bc), B);
          mma(acc[2 * np], hi[ks], B[0], B[1]);
          mma(acc[2 * np + 1], hi[ks], B[2], B[3]);
          if constexpr (L::kTerms == 2) {
            mma(acc[2 * np], lo[ks], B[0], B[1]);
            mma(acc[2 * np + 1], lo[ks], B[2], B[3]);
            ldsm4(mt + L::kSq + tile_off<32>(16 * np + br, 16 * ks + bc), B);
            mma(acc[2 * np], hi[ks], B[0], B[1]);
            mma(acc[2 * np + 1], hi[ks], B[2], B[3]);
          }
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 qc = *reinterpret_cast<const float2*>(f.qc + 8 * i + tc);
        const float2 mu = *reinterpret_cast<const float2*>(f.mu + 8 * i + tc);
        yq[i][0] = fmaf(yq[i][0] * inv0, qc.x, acc[i][0] * iv.x * mu.x);
        yq[i][1] = fmaf(yq[i][1] * inv0, qc.y, acc[i][1] * iv.x * mu.y);
        yq[i][2] = fmaf(yq[i][2] * inv1, qc.x, acc[i][2] * iv.y * mu.x);
        yq[i][3] = fmaf(yq[i][3] * inv1, qc.y, acc[i][3] * iv.y * mu.y);
      }
      store_tile<T>(yq, stage, static_cast<T*>(a.out) + row0, a.H * a.P, n, rows, a.out_vec, lane);
    } else {
      store_tile<float>(e, stage, static_cast<float*>(a.out) + row0, a.H * a.P, n, rows, a.out_vec, lane);
    }
    // S' = exp(cs_C) S + U K, in units in which U fills fp16's range and S stays below 2^35
    float u0 = 0.f, u1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 uc = *reinterpret_cast<const float2*>(f.uc + 8 * i + tc);
      e[i][0] *= uc.x, e[i][1] *= uc.y, e[i][2] *= uc.x, e[i][3] *= uc.y;
      u0 = fmaxf(u0, fmaxf(fabsf(e[i][0]), fabsf(e[i][1])));
      u1 = fmaxf(u1, fmaxf(fabsf(e[i][2]), fabsf(e[i][3])));
    }
    u0 = fmaxf(quad_max(u0), m0 * sig0 * 0x1p-20f), u1 = fmaxf(quad_max(u1), m1 * sig1 * 0x1p-20f);
    float n0, n1;
    const float su0 = pow2_scale(u0, n0), su1 = pow2_scale(u1, n1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float s = x & 1 ? su1 : su0;
        split2(e[2 * ks + (x >> 1)][2 * (x & 1)] * s, e[2 * ks + (x >> 1)][2 * (x & 1) + 1] * s, hi[ks][x], lo[ks][x]);
      }
    const float w0 = f.whole * sig0 * su0, w1 = f.whole * sig1 * su1;
#pragma unroll
    for (int i = 0; i < NT / 8; ++i) S[i][0] *= w0, S[i][1] *= w0, S[i][2] *= w1, S[i][3] *= w1;
    sig0 = n0, sig1 = n1;
    state_add<NT, L::kTerms>(S, hi, lo, kt, lane);
    __syncthreads();
  }
  if (a.fin && run.fin >= 0)
    store_state<NT>(S, sig0, sig1, a.fin + (((int64_t)run.fin * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
}

template <typename T, int NT, bool STAGED, int MODE>
cudaError_t launch_walk(const WalkArgs& a, cudaStream_t stream) {
  constexpr int smem = Tiles<T, NT, STAGED>::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(k_delta_walk<T, NT, STAGED, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_delta_walk<T, NT, STAGED, MODE><<<(unsigned)a.n_units, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch_walk_any(const WalkArgs& a, cudaStream_t stream) {
  // 16-byte copies need rows on 16-byte boundaries; fp32 tiles are read where they lie
  const bool staged = sizeof(T) == 2 && a.qk_vec;
  if constexpr (sizeof(T) == 2) {
    if (staged) {
      if (a.N <= 64) return launch_walk<T, 64, true, MODE>(a, stream);
      if (a.N <= 128) return launch_walk<T, 128, true, MODE>(a, stream);
      return launch_walk<T, 256, true, MODE>(a, stream);
    }
  }
  if (a.N <= 64) return launch_walk<T, 64, false, MODE>(a, stream);
  if (a.N <= 128) return launch_walk<T, 128, false, MODE>(a, stream);
  return launch_walk<T, 256, false, MODE>(a, stream);
}

}  // namespace delta
}  // namespace ssd
