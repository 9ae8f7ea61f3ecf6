// One token of the gated delta rule per batch row, on a state the caller keeps:
//     u = beta (v - exp(g) S k),  S <- exp(g) S + u k^T,  y = scale S q
//
// Bound by HBM on the state, read and written once (8 b H P N bytes).  Both
// products are taken with the state as it is loaded, S k and S q in one pass,
// and y = scale (exp(g) S q + u (k . q)): the row never has to be read again
// after u is known.  A row of the state lies across LP lanes, four consecutive
// values each (float4), so short rows share a warp; a lane holds kRows rows at
// once, all loaded before any is used.
//
// 256 rows of H80 P64 N128 (671 MB of state): 201 to 212 us from box to box, 6.3
// to 6.7 TB/s, a plain copy's rate.  CTAs of 256 threads took 251 us (the loads of a CTA
// come in one burst, and half as many CTAs overlap), four rows a lane 223 us,
// sixteen 667 us; without the streaming hints 208 us.  The hints cost nothing
// where the state stays in L2 (21 MB: 7.6 us with or without).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxN = 256;

struct Args {
  int64_t H, P, N, hpg, G;
  int slices;  // CTAs over headdim
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* state;
  void* y;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LP lanes a row (4 LP >= N, or 32 lanes and NK pieces of 128 columns), kRows
// rows a lane.
template <typename T, int LP, int NK, int kRows>
__global__ void __launch_bounds__(kThreads) k_delta_step(const Args a) {
  constexpr int RW = 32 / LP;                       // rows a warp takes at once
  constexpr int kCta = RW * kRows * (kThreads / 32);  // rows of a CTA
  const int slice = blockIdx.x % a.slices;
  const int64_t bh = blockIdx.x / a.slices, b = bh / a.H, grp = (bh % a.H) / a.hpg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane % LP;
  const int64_t p0 = (int64_t)slice * kCta + warp * (RW * kRows) + lane / LP;
  float* __restrict__ S = a.state + bh * a.P * a.N;
  float4 s[kRows][NK];
  float vv[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t p = p0 + r * RW;
    vv[r] = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      const int n = 4 * col + 128 * c;
      s[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < a.P && n < a.N) s[r][c] = __ldcs(reinterpret_cast<const float4*>(S + p * a.N + n));
    }
    if (p < a.P) vv[r] = to_f(static_cast<const T*>(a.v)[bh * a.P + p]);
  }
  const T* kp = static_cast<const T*>(a.k) + (b * a.G + grp) * a.N;
  const T* qp = static_cast<const T*>(a.q) + (b * a.G + grp) * a.N;
  float4 kv[NK], qv[NK];
  float kq = 0.f;
#pragma unroll
  for (int c = 0; c < NK; ++c) {
    const int n = 4 * col + 128 * c;
    kv[c] = n < a.N ? load4(kp + n) : make_float4(0.f, 0.f, 0.f, 0.f);
    qv[c] = n < a.N ? load4(qp + n) : make_float4(0.f, 0.f, 0.f, 0.f);
    kq = dot4(kv[c], qv[c], kq);
  }
  const float decay = expf(a.g[bh]), beta = a.beta[bh];
  kq = group_sum<LP>(kq);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t p = p0 + r * RW;
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c) sk = dot4(s[r][c], kv[c], sk), sq = dot4(s[r][c], qv[c], sq);
    sk = group_sum<LP>(sk), sq = group_sum<LP>(sq);
    const float u = beta * fmaf(-decay, sk, vv[r]);
    if (p < a.P) {
#pragma unroll
      for (int c = 0; c < NK; ++c) {
        const int n = 4 * col + 128 * c;
        if (n >= a.N) continue;
        float4 t = s[r][c];
        t.x = fmaf(decay, t.x, u * kv[c].x), t.y = fmaf(decay, t.y, u * kv[c].y);
        t.z = fmaf(decay, t.z, u * kv[c].z), t.w = fmaf(decay, t.w, u * kv[c].w);
        __stcs(reinterpret_cast<float4*>(S + p * a.N + n), t);
      }
      if (col == 0) from_f(static_cast<T*>(a.y) + bh * a.P + p, a.scale * fmaf(decay, sq, u * kq));
    }
  }
}

template <typename T, int LP, int NK>
cudaError_t launch(Args& a, int64_t units, cudaStream_t st) {
  // Few rows: two a lane instead of eight, so that four times the CTAs share the
  // loads (of the small variant at most 4 x 2 x 148; of the other a CTA takes 16
  // rows or more, which bounds the grid before the launch).
  constexpr int kFew = 2, kMany = NK == 1 ? 8 : 4;
  const int64_t few = (int64_t)(32 / LP) * kFew * (kThreads / 32), many = few / kFew * kMany;
  const bool small = units * ((a.P + many - 1) / many) < 2 * 148;
  const int64_t cta = small ? few : many;
  a.slices = (int)((a.P + cta - 1) / cta);
  const unsigned grid = (unsigned)(units * a.slices);
  if (small) k_delta_step<T, LP, NK, kFew><<<grid, kThreads, 0, st>>>(a);
  else k_delta_step<T, LP, NK, kMany><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_any(Args& a, int64_t units, cudaStream_t st) {
  if (a.N <= 16) return launch<T, 4, 1>(a, units, st);
  if (a.N <= 32) return launch<T, 8, 1>(a, units, st);
  if (a.N <= 64) return launch<T, 16, 1>(a, units, st);
  if (a.N <= 128) return launch<T, 32, 1>(a, units, st);
  return launch<T, 32, 2>(a, units, st);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace ssd

extern "C" SSD_API ssd_status ssd_delta_step(const ssd_delta_step_args* a, void* stream) {
  using namespace ssd;
  if (!a) return SSD_ERR_INVALID_ARG;
  if (a->batch <= 0 || a->nheads <= 0 || a->headdim <= 0 || a->dstate <= 0 || a->ngroups <= 0)
    return SSD_ERR_INVALID_ARG;
  if (a->nheads % a->ngroups != 0) return SSD_ERR_INVALID_ARG;
  if (a->dtype != SSD_F32 && a->dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->state || !a->y) return SSD_ERR_INVALID_ARG;
  const size_t esz = a->dtype == SSD_BF16 ? 2 : 4;
  if (!aligned(a->state, 16) || !aligned(a->q, 4 * esz) || !aligned(a->k, 4 * esz) || !aligned(a->v, esz) ||
      !aligned(a->y, esz) || !aligned(a->g, 4) || !aligned(a->beta, 4))
    return SSD_ERR_INVALID_ARG;
  if (a->dstate % 4 != 0 || a->dstate > kMaxN || a->headdim > 65536) return SSD_ERR_UNSUPPORTED;
  // a CTA takes 16 rows at least where the grid is large: it stays below 2^31
  if ((double)a->batch * (double)a->nheads * (double)((a->headdim + 15) / 16) >= 2147483647.0)
    return SSD_ERR_UNSUPPORTED;
  Args s;
  s.H = a->nheads, s.P = a->headdim, s.N = a->dstate, s.G = a->ngroups, s.hpg = a->nheads / a->ngroups;
  s.slices = 1, s.scale = a->scale;
  s.q = a->q, s.k = a->k, s.v = a->v, s.g = a->g, s.beta = a->beta, s.state = a->state, s.y = a->y;
  const int64_t units = a->batch * a->nheads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == SSD_BF16 ? launch_any<__nv_bfloat16>(s, units, st) : launch_any<float>(s, units, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
