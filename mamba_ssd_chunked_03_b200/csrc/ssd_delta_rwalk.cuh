// The reverse walk of the gated delta rule's backward (ssd_delta_prep.cuh has
// the formulas): the gradient of the state carried from a sequence's last
// chunk to its first, laid out and scaled as the forward walk carries the
// state.  Per chunk: dU = M^T dY + exp(cs_C - cs) K dS^T, D = (I + A)^-T dU,
// and dS' from dY with q and D with k.  It leaves dv = beta D, D, and dS at
// every checkpoint.  Bound as the forward walk is, by the chain of a warp's
// chunk: b4 L2048 H32 P64 N128, one CTA an SM, 200 us (3.1 us a chunk), 32 %
// of it with the matrix pipe busy.
#pragma once

#include "ssd_delta_walk.cuh"

namespace ssd {
namespace delta {

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 128 ? 3 : 2) k_delta_rwalk(const WalkArgs a) {
  using B = Buffers<T, NT, true, 2>;
  using X = TokenTiles<T, NT>;
  using Hd = RevTiles;
  constexpr int kTerms = X::kTerms;
  extern __shared__ __align__(128) char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices;
  const int64_t rh = blockIdx.x / a.slices, h = rh % a.H, ri = rh / a.H;
  const Run run = a.runs ? a.runs[ri] : row_run(ri, a.L);
  const int nc = (run.len + kC - 1) / kC;
  const int p_cta = slice * kP, p0 = p_cta + 16 * warp;
  const int cols = (int)(a.pv - p_cta < kP ? a.pv - p_cta : kP);
  const int rows = a.P - p0 < 16 ? (int)(a.P - p0) : 16;
  const int64_t vstride = a.H * a.pv, tstride = a.G * X::kBytes, hstride = a.H * Hd::kStride;
  const char* tok = a.tokens + (run.chunk * a.G + h / a.hpg) * X::kBytes;
  const char* head = a.heads + (run.chunk * a.H + h) * Hd::kStride;
  const T* v = static_cast<const T*>(a.v) + (run.tok * a.H + h) * a.pv + p_cta;
  float S[NT / 8][4];
  if (a.s0 && run.fin >= 0 && nc > 0) {
    load_state<NT>(S, a.s0 + (((int64_t)run.fin * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
  } else {
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
  }
  Unit unit;
  unit.init<NT>(S);
  char* stage = sm + B::kStage + warp * (kC * 20 * 4);
  sm100::griddep_wait();
  const auto fetch = [&](int j) {
    const int n = run.len - j * kC;
    fetch_chunk<T, NT, true, 2>(tok + j * tstride, head + j * hstride, v + (int64_t)j * kC * vstride, vstride, n, cols,
                                sm + (j & 1) * B::kBuf);
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
    if ((j & 1) == 1 || j == nc - 1) {
      const int64_t at = (run.slot + (j >> 1)) * a.H + h;
      store_state<NT>(S, unit.sig.x, unit.sig.y, a.check + (at * a.P + p0) * a.N, a.N, rows, lane);
      const float m = warp_absmax(fmaxf(unit.bnd.x * unit.sig.x, unit.bnd.y * unit.sig.y));
      if (lane == 0) a.max_check[at * a.pg + p0 / 16] = m;
    }
    float acc[4][4], d[4][4], y[4][4], e[4][4];
    state_times<NT, kTerms, false>(S, acc, kt, acc, 0, lane);
    const int64_t at = ((run.chunk + j) * a.H + h) * a.pg + p0 / 16;
    uint32_t hi[2][4], lo[2][4];
    load_v<T, B::kVP>(y, buf + B::kV, 16 * warp, lane);
    const float ymax = warp_absmax(tile_max(y));
    if (lane == 0) a.max_v[at] = ymax;
    // M^T dY: the scales of M's rows are powers of two, so bf16 values stay exact in one term
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) e[i][x] = y[i][x];
    scale_tile(e, f.mu, make_float2(1.f, 1.f), lane);
    float2 iv = to_operand<kTerms == 2>(e, hi, lo);
    zero(d);
    lower_mma_t<kTerms == 2>(d, hi, lo, mt, lane);
    // dU, with the scales of the inverse's rows
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i][0] *= iv.x, d[i][1] *= iv.x, d[i][2] *= iv.y, d[i][3] *= iv.y;
    add_scaled(d, acc, f.kc, unit.sig, lane);
    scale_tile(d, f.tau, make_float2(1.f, 1.f), lane);
    iv = to_operand<true>(d, hi, lo);
    zero(d);
    lower_mma_t<true>(d, hi, lo, tt, lane);
    // D: at most 32 products of two operands below 2^15 and a power of two
    const int n = run.len - j * kC < kC ? run.len - j * kC : kC;
    const int64_t th = (run.tok + (int64_t)j * kC) * a.H + h, row0 = th * a.P + p0, rowe = th * a.pe + p0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i][0] *= iv.x, d[i][1] *= iv.x, d[i][2] *= iv.y, d[i][3] *= iv.y;
      e[i][0] = d[i][0], e[i][1] = d[i][1], e[i][2] = d[i][2], e[i][3] = d[i][3];
    }
    scale_tile(e, f.beta, make_float2(1.f, 1.f), lane);
    const float2 db = make_float2(iv.x * 0x1p35f, iv.y * 0x1p35f);
    {
      const float m = warp_absmax(tile_max(d));
      if (lane == 0) a.max_out[at] = m;
    }
    store_tile<float>(d, stage, a.out_f + rowe, a.H * a.pe, n, (rows + 3) & ~3, true, lane);
    store_tile<T>(e, stage, static_cast<T*>(a.out) + row0, a.H * a.P, n, rows, a.out_vec, lane);
    // dS' = exp(cs_C) dS + (scale exp(cs) dY) q - (beta exp(cs) D) k
    const float yb = ymax * f.qcm;
    const float2 is = unit.step<NT>(S, f.whole, make_float2(fmaf(db.x, f.ucm, yb), fmaf(db.y, f.ucm, yb)), (j & 7) == 0);
    scale_tile(y, f.qc, is, lane);
    as_operand<true>(y, hi, lo);
    state_add<NT, kTerms>(S, hi, lo, qt, lane);
    scale_tile(d, f.uc, is, lane);
    as_operand<true>(d, hi, lo);
    state_add<NT, kTerms>(S, hi, lo, kt, lane);
  }
  if (a.fin && run.h0 >= 0)
    store_state<NT>(S, unit.sig.x, unit.sig.y, a.fin + (((int64_t)run.h0 * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
}

template <typename T, int NT>
cudaError_t launch_rwalk_nt(const WalkArgs& a, cudaStream_t stream) {
  constexpr int smem = Buffers<T, NT, true, 2>::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> seen{0};
  return launch_kernel(k_delta_rwalk<T, NT>, seen, (unsigned)a.units, kThreads, smem, smem, true, stream, a);
}

template <typename T>
cudaError_t launch_rwalk(const WalkArgs& a, cudaStream_t stream) {
  if (a.N <= 64) return launch_rwalk_nt<T, 64>(a, stream);
  if (a.N <= 128) return launch_rwalk_nt<T, 128>(a, stream);
  return launch_rwalk_nt<T, 256>(a, stream);
}

}  // namespace delta
}  // namespace ssd
