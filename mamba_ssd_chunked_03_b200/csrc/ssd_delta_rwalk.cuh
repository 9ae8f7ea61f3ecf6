// The reverse walk of the gated delta rule's backward (ssd_delta_prep.cuh has
// the formulas): the gradient of the state carried from a sequence's last
// chunk to its first, laid out and scaled as the forward walk carries the
// state.  Per chunk: dU = M^T dY + exp(cs_C - cs) K dS^T, D = (I + A)^-T dU,
// and dS' from dY with q and D with k.  It leaves dv = beta D, D, and dS at
// every checkpoint.
#pragma once

#include "ssd_delta_walk.cuh"

namespace ssd {
namespace delta {

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 128 ? 3 : 2) k_delta_rwalk(const WalkArgs a) {
  using B = Buffers<T, NT, true, 2>;
  using X = TokenTiles<T, NT>;
  using Hd = HeadTiles<2>;
  constexpr int kTerms = X::kTerms;
  extern __shared__ __align__(128) char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices;
  const int64_t rh = blockIdx.x / a.slices, h = rh % a.H, ri = rh / a.H;
  const Run run = a.runs ? a.runs[ri] : row_run(ri, a.L);
  const int nc = (run.len + kC - 1) / kC;
  const int p_cta = slice * kP, p0 = p_cta + 16 * warp;
  const int cols = (int)(a.P - p_cta < kP ? a.P - p_cta : kP);
  const int rows = a.P - p0 < 16 ? (int)(a.P - p0) : 16;
  const int64_t vstride = a.H * a.P, tstride = a.G * X::kBytes, hstride = a.H * Hd::kBytes;
  const char* tok = a.tokens + (run.chunk * a.G + h / a.hpg) * X::kBytes;
  const char* head = a.heads + (run.chunk * a.H + h) * Hd::kBytes;
  const T* v = static_cast<const T*>(a.v) + (run.tok * a.H + h) * a.P + p_cta;
  float S[NT / 8][4];
  float sig0 = 1.f, sig1 = 1.f;
  if (a.s0 && run.fin >= 0) {
    load_state<NT>(S, a.s0 + (((int64_t)run.fin * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
  } else {
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
  }
  char* stage = sm + B::kStage + warp * (kC * 20 * 4);
  sm100::griddep_wait();
  const auto fetch = [&](int j) {
    const int n = run.len - j * kC;
    fetch_chunk<T, NT, true, 2>(tok + j * tstride, head + j * hstride, v + (int64_t)j * kC * vstride, vstride, n, cols,
                                a.v_vec, sm + (j & 1) * B::kBuf);
  };
  if (nc > 0) fetch(nc - 1);
  for (int j = nc - 1; j >= 0; --j) {
    cp_async_wait<0>();
    __syncthreads();
    if (j > 0) fetch(j - 1);
    if (rows <= 0) continue;
    char* const buf = sm + (j & 1) * B::kBuf;
    const Factors& f = *reinterpret_cast<const Factors*>(buf + B::kHead + Hd::kF);
    const uint32_t kt = sm100::smem_u32(buf), qt = kt + kTerms * X::kTile;
    const uint32_t tt = kt + B::kHead, mt = tt + Hd::kM;
    float m0, m1, inv0, inv1;
    state_max<NT>(S, m0, m1);
    if ((j & 1) == 1 || j == nc - 1) {
      const int64_t at = (run.slot + (j >> 1)) * a.H + h;
      store_state<NT>(S, sig0, sig1, a.check + (at * a.P + p0) * a.N, a.N, rows, lane);
      const float m = warp_absmax(fmaxf(m0 * sig0, m1 * sig1));
      if (lane == 0) a.max_check[at * a.pg + p0 / 16] = m;
    }
    const float sc0 = pow2_scale(m0, inv0), sc1 = pow2_scale(m1, inv1);
    inv0 *= sig0, inv1 *= sig1;
    float acc[4][4], d[4][4], y[4][4];
    zero(acc);
#pragma unroll
    for (int ks = 0; ks < NT / 16; ++ks) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        split2(mul2(S[2 * ks + (x >> 1)][2 * (x & 1)], S[2 * ks + (x >> 1)][2 * (x & 1) + 1], x & 1 ? sc1 : sc0), hi[x], lo[x]);
      tokens_mma<NT, kTerms, true>(acc, hi, lo, kt, ks, lane);
    }
    const int tc = 2 * (lane & 3);
    const int64_t at = ((run.chunk + j) * a.H + h) * a.pg + p0 / 16;
    uint32_t hi[2][4], lo[2][4];
    float2 iv;
    load_v<T, B::kVP>(y, buf + B::kV, 16 * warp, lane);
    {
      const float m = warp_absmax(tile_max(y));
      if (lane == 0) a.max_v[at] = m;
    }
    // M^T dY: the scales of M's rows are powers of two, so bf16 values stay exact in one term
    float e[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 mu = *reinterpret_cast<const float2*>(f.mu + 8 * i + tc);
      e[i][0] = y[i][0] * mu.x, e[i][1] = y[i][1] * mu.y, e[i][2] = y[i][2] * mu.x, e[i][3] = y[i][3] * mu.y;
    }
    iv = to_operand<kTerms == 2>(e, hi, lo);
    zero(d);
    lower_mma_t<kTerms == 2>(d, hi, lo, mt, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // dU, with the scales of the inverse's rows
      const float2 kc = *reinterpret_cast<const float2*>(f.kc + 8 * i + tc);
      const float2 tau = *reinterpret_cast<const float2*>(f.tau + 8 * i + tc);
      e[i][0] = fmaf(acc[i][0] * inv0, kc.x, d[i][0] * iv.x) * tau.x;
      e[i][1] = fmaf(acc[i][1] * inv0, kc.y, d[i][1] * iv.x) * tau.y;
      e[i][2] = fmaf(acc[i][2] * inv1, kc.x, d[i][2] * iv.y) * tau.x;
      e[i][3] = fmaf(acc[i][3] * inv1, kc.y, d[i][3] * iv.y) * tau.y;
    }
    iv = to_operand<true>(e, hi, lo);
    zero(d);
    lower_mma_t<true>(d, hi, lo, tt, lane);
    const int n = run.len - j * kC < kC ? run.len - j * kC : kC;
    const int64_t row0 = ((run.tok + (int64_t)j * kC) * a.H + h) * a.P + p0;
    float u0 = 0.f, u1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i][0] *= iv.x, d[i][1] *= iv.x, d[i][2] *= iv.y, d[i][3] *= iv.y;
      const float2 be = *reinterpret_cast<const float2*>(f.beta + 8 * i + tc);
      e[i][0] = d[i][0] * be.x, e[i][1] = d[i][1] * be.y, e[i][2] = d[i][2] * be.x, e[i][3] = d[i][3] * be.y;
    }
    {
      const float m = warp_absmax(tile_max(d));
      if (lane == 0) a.max_out[at] = m;
    }
    store_tile<float>(d, stage, a.out_f + row0, a.H * a.P, n, rows, a.P % 4 == 0, lane);
    store_tile<T>(e, stage, static_cast<T*>(a.out) + row0, a.H * a.P, n, rows, a.out_vec, lane);
    // dS' = exp(cs_C) dS + (scale exp(cs) dY) q - (beta exp(cs) D) k, in common units
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 qc = *reinterpret_cast<const float2*>(f.qc + 8 * i + tc);
      const float2 uc = *reinterpret_cast<const float2*>(f.uc + 8 * i + tc);
      y[i][0] *= qc.x, y[i][1] *= qc.y, y[i][2] *= qc.x, y[i][3] *= qc.y;
      d[i][0] *= uc.x, d[i][1] *= uc.y, d[i][2] *= uc.x, d[i][3] *= uc.y;
      u0 = fmaxf(u0, fmaxf(fmaxf(fabsf(y[i][0]), fabsf(y[i][1])), fmaxf(fabsf(d[i][0]), fabsf(d[i][1]))));
      u1 = fmaxf(u1, fmaxf(fmaxf(fabsf(y[i][2]), fabsf(y[i][3])), fmaxf(fabsf(d[i][2]), fabsf(d[i][3]))));
    }
    u0 = fmaxf(quad_max(u0), m0 * sig0 * 0x1p-20f), u1 = fmaxf(quad_max(u1), m1 * sig1 * 0x1p-20f);
    float n0, n1;
    const float su0 = pow2_scale(u0, n0), su1 = pow2_scale(u1, n1);
    const float w0 = f.whole * sig0 * su0, w1 = f.whole * sig1 * su1;
#pragma unroll
    for (int i = 0; i < NT / 8; ++i) {
      const float2 x = mul2(S[i][0], S[i][1], w0), z = mul2(S[i][2], S[i][3], w1);
      S[i][0] = x.x, S[i][1] = x.y, S[i][2] = z.x, S[i][3] = z.y;
    }
    sig0 = n0, sig1 = n1;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 2 * ks + (x >> 1), c = 2 * (x & 1);
          split2(w ? mul2(d[r][c], d[r][c + 1], x & 1 ? su1 : su0) : mul2(y[r][c], y[r][c + 1], x & 1 ? su1 : su0), hi[ks][x],
                 lo[ks][x]);
        }
      state_add<NT, kTerms>(S, hi, lo, w ? kt : qt, lane);
    }
  }
  if (a.fin && run.h0 >= 0)
    store_state<NT>(S, sig0, sig1, a.fin + (((int64_t)run.h0 * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
}

template <typename T, int NT>
cudaError_t launch_rwalk_nt(const WalkArgs& a, cudaStream_t stream) {
  constexpr int smem = Buffers<T, NT, true, 2>::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  return launch_after(k_delta_rwalk<T, NT>, (unsigned)a.units, smem, a, stream);
}

template <typename T>
cudaError_t launch_rwalk(const WalkArgs& a, cudaStream_t stream) {
  if (a.N <= 64) return launch_rwalk_nt<T, 64>(a, stream);
  if (a.N <= 128) return launch_rwalk_nt<T, 128>(a, stream);
  return launch_rwalk_nt<T, 256>(a, stream);
}

}  // namespace delta
}  // namespace ssd
