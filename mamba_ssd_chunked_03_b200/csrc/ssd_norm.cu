// Layer norm over the last axis with the block's gate, forward and backward:
//     y = ((x - mean) rstd w + b) SiLU(z)
//     dx = rstd (hw - mean(hw) - n mean(hw n)),  n = (x - mean) rstd, hw = dout SiLU(z) w
//     dw = sum_rows dout SiLU(z) n,  db = sum_rows dout SiLU(z)
//     dz = dout (n w + b) SiLU'(z)
//
// Bound by HBM: every tensor is read once and every output written once.  A
// row belongs to a group of GT threads (part of a warp, or a whole CTA), which
// holds it in registers: the mean first, then the mean square of the
// differences, so that a large mean costs no accuracy.  Groups walk the rows
// with a fixed stride and load the next row before they work on this one;
// weights, biases and the sums of their gradients stay in registers all the
// way.  The backward's partial sums (one set a CTA) are added by a second
// kernel in a fixed order.  Rows wider than the registers hold are swept
// several times from memory instead, with the column sums in a pass of their
// own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kSMs = 148;
constexpr int kThreads = 256;     // CTA of the kernels whose rows share one
constexpr int kMostThreads = 512;  // CTA of one row, as many as it needs
constexpr int kParts = 3 * kSMs;  // most CTAs of the backward, each with its partial sums

struct Args {
  int64_t rows, cols;
  float eps;
  const void* x;
  const float* w;
  const float* b;
  const void* z;
  const void* dout;
  void* out;    // forward: y; backward: dx
  void* dz;
  float* part;  // backward: [2][kParts][cols] partial sums of dw, db, or null
  float* stat;  // wide rows: [rows][2] mean, rstd
};

// E consecutive elements as they are loaded and stored
template <typename T, int E>
struct Pack;
template <>
struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(p); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = r; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(r); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The hardware exponential and an approximate divide: off by a few 2^-23.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
// z sigmoid(z); 0 at z = -inf
__device__ __forceinline__ float silu(float v) { return v < -1e30f ? 0.f : v * sigmoid(v); }

// Sums of N values over the GT threads of a group (GT > 32: the CTA's threads,
// however many), the same bits in each of them.
template <int GT>
struct GroupSum {
  float4 (*red)[kMostThreads / 32];  // two sets, taken in turn: one barrier a sum
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int o = (GT < 32 ? GT : 32) / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (GT > 32) {
      if ((threadIdx.x & 31) == 0)
        red[turn][threadIdx.x >> 5] = make_float4(v[0], v[N > 1 ? 1 : 0], v[N > 2 ? 2 : 0], v[N > 3 ? 3 : 0]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll 4
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        const float4 x = red[turn][w];
        v[0] += x.x;
        if constexpr (N > 1) v[1] += x.y;
        if constexpr (N > 2) v[2] += x.z;
        if constexpr (N > 3) v[3] += x.w;
      }
      turn ^= 1;
    }
  }
};

// Rows held in registers: VPL packs of E elements for each of the GT threads of
// a row (GT > 32: the CTA's threads, however many up to BT).
template <typename T, int E, int GT, int VPL, int BT, int MINB, bool BWD, bool GATE>
__global__ void __launch_bounds__(BT, MINB) k_norm(const Args a) {
  using Pk = Pack<T, E>;
  constexpr int GC = GT > 32 ? 1 : kThreads / GT;  // groups of a CTA
  __shared__ float4 red[2][kMostThreads / 32];
  GroupSum<GT> sum{red};
  const int gt = GT > 32 ? blockDim.x : GT;  // threads of a row
  const int g = GT > 32 ? 0 : threadIdx.x / GT, l = GT > 32 ? threadIdx.x : threadIdx.x % GT;
  const int64_t cols = a.cols;
  const float inv_cols = 1.f / (float)cols;
  const auto col = [&](int v) { return (int64_t)(v * gt + l) * E; };
  float w[VPL][E], b[VPL][E], dw[VPL][E], db[VPL][E];
#pragma unroll
  for (int v = 0; v < VPL; ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = col(v) < cols;
      w[v][e] = a.w && in ? a.w[col(v) + e] : 1.f;
      b[v][e] = a.b && in ? a.b[col(v) + e] : 0.f;
      dw[v][e] = db[v][e] = 0.f;
    }
  Pk xr[VPL], zr[VPL], dr[VPL];
  const auto fetch = [&](int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (col(v) < cols) {
        xr[v].load(static_cast<const T*>(a.x) + r * cols + col(v));
        if constexpr (GATE) zr[v].load(static_cast<const T*>(a.z) + r * cols + col(v));
        if constexpr (BWD) dr[v].load(static_cast<const T*>(a.dout) + r * cols + col(v));
      }
  };
  const int64_t stride = (int64_t)gridDim.x * GC;
  fetch((int64_t)blockIdx.x * GC + g);
  for (int64_t r0 = (int64_t)blockIdx.x * GC; r0 < a.rows; r0 += stride) {  // the same trips for all threads
    const int64_t r = r0 + g;
    const bool live = r < a.rows;
    float x[VPL][E], z[VPL][E], d[VPL][E];  // x - mean, the gate, and dout: then dout SiLU(z)
    float s0[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool in = live && col(v) < cols;
      xr[v].get(x[v]);
      if constexpr (GATE) zr[v].get(z[v]);
      if constexpr (BWD) dr[v].get(d[v]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[v][e] = in ? x[v][e] : 0.f;
        if constexpr (GATE) z[v][e] = in ? z[v][e] : 0.f;
        if constexpr (BWD) d[v][e] = in ? d[v][e] : 0.f;
        s0[0] += x[v][e];
      }
    }
    fetch(r + stride);
    sum(s0);
    const float mean = s0[0] * inv_cols;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[v][e] = col(v) < cols ? x[v][e] - mean : 0.f;
        sq[0] = fmaf(x[v][e], x[v][e], sq[0]);
      }
    sum(sq);
    const float rstd = 1.f / sqrtf(fmaf(sq[0], inv_cols, a.eps));
    if constexpr (!BWD) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          y[e] = fmaf(x[v][e] * rstd, w[v][e], b[v][e]);
          if constexpr (GATE) y[e] *= silu(z[v][e]);
        }
        if (live && col(v) < cols) Pk::store(static_cast<T*>(a.out) + r * cols + col(v), y);
      }
    } else {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float dz[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float n = x[v][e] * rstd;
          float h = d[v][e];
          if constexpr (GATE) {
            const float sg = sigmoid(z[v][e]);
            dz[e] = h * fmaf(n, w[v][e], b[v][e]) * (sg * fmaf(z[v][e], 1.f - sg, 1.f));
            h *= z[v][e] * sg;
          }
          dw[v][e] = fmaf(h, n, dw[v][e]);
          db[v][e] += h;
          d[v][e] = h * w[v][e];
          m[0] += d[v][e];
          m[1] = fmaf(d[v][e], n, m[1]);
        }
        if constexpr (GATE)
          if (live && col(v) < cols) Pk::store(static_cast<T*>(a.dz) + r * cols + col(v), dz);
      }
      sum(m);
      const float m1 = m[0] * inv_cols, m2 = m[1] * inv_cols * rstd;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = rstd * (fmaf(-x[v][e], m2, d[v][e]) - m1);
        if (live && col(v) < cols) Pk::store(static_cast<T*>(a.out) + r * cols + col(v), y);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // the CTA's groups added in order, one set of partial sums a CTA
    float* pw = a.part + blockIdx.x * cols;
    float* pb = pw + (int64_t)kParts * cols;
    if constexpr (GC == 1) {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (col(v) < cols) {
#pragma unroll
          for (int e = 0; e < E; ++e) pw[col(v) + e] = dw[v][e], pb[col(v) + e] = db[v][e];
        }
    } else {
      // groups of a warp by shuffles, then the warps through shared memory
      __shared__ float2 all[kThreads / 32][32][E];
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float p = dw[v][e], q = db[v][e];
#pragma unroll
          for (int o = GT; o < 32; o <<= 1) {
            p += __shfl_xor_sync(0xffffffffu, p, o);
            q += __shfl_xor_sync(0xffffffffu, q, o);
          }
          all[threadIdx.x >> 5][threadIdx.x & 31][e] = make_float2(p, q);
        }
        __syncthreads();
        if (threadIdx.x < GT && col(v) < cols) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float p = 0.f, q = 0.f;
            for (int i = 0; i < kThreads / 32; ++i) p += all[i][threadIdx.x][e].x, q += all[i][threadIdx.x][e].y;
            pw[col(v) + e] = p, pb[col(v) + e] = q;
          }
        }
      }
    }
  }
}

// Rows of bf16 that take a CTA.
//
// Such a row costs a barrier for every sum that waits for another one, so all
// of its sums are taken at once, of the differences to K, the mean of the
// row's first pack: x - mean = (x - K) - mean(x - K), var = mean((x - K)^2) -
// mean(x - K)^2.  K is off the mean by at most sqrt(cols / 8) deviations, since
// its elements are part of the row, and by less than one in all but contrived
// rows; what cancels in var is then cols / 8 x 2^-24 at the very most, far
// below the rounding of the outputs.  The row stays packed in registers and is
// unpacked again after the sums; weight and bias lie in shared memory: that
// leaves room for a second CTA's rows.
template <int VPL, int BT, int MINB, bool BWD, bool GATE>
__global__ void __launch_bounds__(BT, MINB) k_norm_row(const Args a) {
  using T = __nv_bfloat16;
  constexpr int E = 8;
  using Pk = Pack<T, E>;
  extern __shared__ __align__(16) float wb[];  // weight, bias
  __shared__ float4 red[2][kMostThreads / 32];
  GroupSum<64> sum{red};
  const int l = threadIdx.x, gt = blockDim.x, cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const auto col = [&](int v) { return (v * gt + l) * E; };
  for (int c = l; c < cols; c += gt) {
    wb[c] = a.w ? a.w[c] : 1.f;
    if constexpr (GATE || !BWD) wb[cols + c] = a.b ? a.b[c] : 0.f;
  }
  __syncthreads();
  const auto weights = [&](int c, float (&w)[E]) {
    const float4 p = *reinterpret_cast<const float4*>(wb + c), q = *reinterpret_cast<const float4*>(wb + c + 4);
    w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w, w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
  };
  float dw[BWD ? VPL : 1][E], db[BWD ? VPL : 1][E];
#pragma unroll
  for (int v = 0; v < (BWD ? VPL : 1); ++v)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[v][e] = db[v][e] = 0.f;
  Pk xn[VPL], zn[VPL], dn[VPL], kn;
  const auto fetch = [&](int64_t r) {
    if (r >= a.rows) return;
    const int64_t o = r * cols;
    kn.load(static_cast<const T*>(a.x) + o);
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (col(v) < cols) {
        xn[v].load(static_cast<const T*>(a.x) + o + col(v));
        if constexpr (GATE) zn[v].load(static_cast<const T*>(a.z) + o + col(v));
        if constexpr (BWD) dn[v].load(static_cast<const T*>(a.dout) + o + col(v));
      }
  };
  fetch(blockIdx.x);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    Pk xr[VPL], zr[VPL], dr[VPL];
    float K = 0.f;
    {
      float k[E];
      kn.get(k);
#pragma unroll
      for (int e = 0; e < E; ++e) K += k[e];
      K *= 1.f / E;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      xr[v] = xn[v];
      if constexpr (GATE) zr[v] = zn[v];
      if constexpr (BWD) dr[v] = dn[v];
    }
    fetch(r + gridDim.x);
    float t[BWD ? 4 : 2] = {};
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (col(v) >= cols) continue;
      float x[E], d[E], z[E], w[E];
      xr[v].get(x);
      if constexpr (BWD) {
        dr[v].get(d);
        weights(col(v), w);
      }
      if constexpr (BWD && GATE) zr[v].get(z);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] -= K;
        t[0] += x[e];
        t[1] = fmaf(x[e], x[e], t[1]);
        if constexpr (BWD) {
          float h = d[e] * w[e];
          if constexpr (GATE) h *= z[e] * sigmoid(z[e]);
          t[2] += h;
          t[3] = fmaf(h, x[e], t[3]);
        }
      }
    }
    sum(t);
    const float dm = t[0] * inv_cols, mean = K + dm;
    const float rstd = 1.f / sqrtf(fmaxf(fmaf(t[1], inv_cols, -dm * dm), 0.f) + a.eps);
    float m1 = 0.f, m2 = 0.f;
    if constexpr (BWD) m1 = t[2] * inv_cols, m2 = rstd * (t[3] - dm * t[2]) * inv_cols;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (col(v) >= cols) continue;
      float x[E], d[E], z[E], w[E], b[E], dz[E];
      xr[v].get(x);
      if constexpr (BWD) dr[v].get(d);
      if constexpr (GATE) zr[v].get(z);
      weights(col(v), w);
      if constexpr (GATE || !BWD) weights(cols + col(v), b);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float n = (x[e] - mean) * rstd;
        if constexpr (!BWD) {
          x[e] = fmaf(n, w[e], b[e]);
          if constexpr (GATE) x[e] *= silu(z[e]);
        } else {
          float h = d[e];
          if constexpr (GATE) {
            const float sg = sigmoid(z[e]);
            dz[e] = h * fmaf(n, w[e], b[e]) * (sg * fmaf(z[e], 1.f - sg, 1.f));
            h *= z[e] * sg;
          }
          dw[v][e] = fmaf(h, n, dw[v][e]);
          db[v][e] += h;
          x[e] = rstd * (fmaf(-n, m2, h * w[e]) - m1);
        }
      }
      Pk::store(static_cast<T*>(a.out) + r * cols + col(v), x);
      if constexpr (BWD && GATE) Pk::store(static_cast<T*>(a.dz) + r * cols + col(v), dz);
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    float* pw = a.part + (int64_t)blockIdx.x * cols;
    float* pb = pw + (int64_t)kParts * cols;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (col(v) < cols) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          *reinterpret_cast<float4*>(pw + col(v) + e) = make_float4(dw[v][e], dw[v][e + 1], dw[v][e + 2], dw[v][e + 3]);
          *reinterpret_cast<float4*>(pb + col(v) + e) = make_float4(db[v][e], db[v][e + 1], db[v][e + 2], db[v][e + 3]);
        }
      }
  }
}

// Rows too wide for registers: one CTA a row at a time, swept from memory.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) k_norm_wide(const Args a) {
  __shared__ float4 red[2][kMostThreads / 32];
  GroupSum<kThreads> sum{red};
  const int64_t cols = a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * cols;
    const T* z = a.z ? static_cast<const T*>(a.z) + r * cols : nullptr;
    float s[1] = {0.f}, q[1] = {0.f};
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) s[0] += to_f(x[c]);
    sum(s);
    const float mean = s[0] / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
      const float d = to_f(x[c]) - mean;
      q[0] = fmaf(d, d, q[0]);
    }
    sum(q);
    const float rstd = 1.f / sqrtf(q[0] / (float)cols + a.eps);
    if constexpr (!BWD) {
      T* y = static_cast<T*>(a.out) + r * cols;
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        float v = fmaf((to_f(x[c]) - mean) * rstd, a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f);
        if (z) v *= silu(to_f(z[c]));
        put(y + c, v);
      }
    } else {
      const T* dout = static_cast<const T*>(a.dout) + r * cols;
      float m[2] = {0.f, 0.f};
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = (to_f(x[c]) - mean) * rstd;
        float h = to_f(dout[c]);
        const float w = a.w ? a.w[c] : 1.f;
        if (z) {
          const float zv = to_f(z[c]), sg = sigmoid(zv);
          put(static_cast<T*>(a.dz) + r * cols + c,
              h * fmaf(n, w, a.b ? a.b[c] : 0.f) * (sg * fmaf(zv, 1.f - sg, 1.f)));
          h *= zv * sg;
        }
        m[0] += h * w;
        m[1] = fmaf(h * w, n, m[1]);
      }
      sum(m);
      const float m1 = m[0] / (float)cols, m2 = m[1] / (float)cols;
      if (threadIdx.x == 0) a.stat[2 * r] = mean, a.stat[2 * r + 1] = rstd;
      T* dx = static_cast<T*>(a.out) + r * cols;
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = (to_f(x[c]) - mean) * rstd;
        float h = to_f(dout[c]);
        if (z) h *= silu(to_f(z[c]));
        put(dx + c, rstd * (h * (a.w ? a.w[c] : 1.f) - m1 - n * m2));
      }
    }
  }
}

// Wide rows: the column sums of one stripe of rows (blockIdx.y) for 256
// columns, with the statistics that k_norm_wide left.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_wide_cols(const Args a) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, cols = a.cols;
  if (c >= cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float n = (to_f(static_cast<const T*>(a.x)[r * cols + c]) - a.stat[2 * r]) * a.stat[2 * r + 1];
    float h = to_f(static_cast<const T*>(a.dout)[r * cols + c]);
    if (a.z) h *= silu(to_f(static_cast<const T*>(a.z)[r * cols + c]));
    dw = fmaf(h, n, dw);
    db += h;
  }
  a.part[blockIdx.y * cols + c] = dw;
  a.part[((int64_t)kParts + blockIdx.y) * cols + c] = db;
}

// dw and db from the partial sums: 32 columns a CTA, eight strands of parts
// each, the strands added in order.
__global__ void __launch_bounds__(kThreads) k_norm_sum(const float* __restrict__ part, int parts, int64_t cols,
                                                       float* dw, float* db) {
  __shared__ double s[2][8][32];
  const int l = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  double p = 0., q = 0.;
  if (c < cols) {
#pragma unroll 4
    for (int i = g; i < parts; i += 8) {
      p += part[i * cols + c];
      q += part[((int64_t)kParts + i) * cols + c];
    }
  }
  s[0][g][l] = p, s[1][g][l] = q;
  __syncthreads();
  if (g < 2 && c < cols) {
    double t = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[g][i][l];
    if (g == 0 && dw) dw[c] = (float)t;
    if (g == 1 && db) db[c] = (float)t;
  }
}

// MINB CTAs an SM, which the kernel's registers allow, and one grid of them.
// `threads`: of a CTA that takes one row; else GT threads take one.
template <typename T, int E, int GT, int VPL, int BT, int MINB, bool BWD>
cudaError_t launch(const Args& a, cudaStream_t st, int* parts, int threads = kThreads) {
  constexpr int GC = GT > 32 ? 1 : kThreads / GT;
  const int64_t need = (a.rows + GC - 1) / GC, most = MINB * kSMs;
  static_assert(!BWD || MINB * kSMs <= kParts, "partial sums");
  const unsigned grid = (unsigned)(need < most ? need : most);
  *parts = (int)grid;
  if (a.z) k_norm<T, E, GT, VPL, BT, MINB, BWD, true><<<grid, threads, 0, st>>>(a);
  else k_norm<T, E, GT, VPL, BT, MINB, BWD, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}
template <int VPL, int BT, int MINB, bool BWD>
cudaError_t launch_row(const Args& a, cudaStream_t st, int* parts) {
  const int64_t most = MINB * kSMs;
  const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
  *parts = (int)grid;
  const int threads = (int)((a.cols / 8 + 32 * VPL - 1) / (32 * VPL) * 32);
  const size_t smem = (size_t)a.cols * (BWD && !a.z ? 4 : 8);  // at most 64 KB
  const auto kern = a.z ? k_norm_row<VPL, BT, MINB, BWD, true> : k_norm_row<VPL, BT, MINB, BWD, false>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, threads, smem, st>>>(a);
  return cudaGetLastError();
}

// The group by the row's packs: part of a warp up to 64 packs (no barrier),
// else a CTA of as many threads as the row needs with one or two packs each.
template <typename T, bool BWD>
cudaError_t launch_rows(const Args& a, bool vec, cudaStream_t st, int* parts, bool* wide) {
  constexpr int E = 16 / (int)sizeof(T), kB = BWD ? 2 : 4;
  *wide = false;
  const auto warps = [](int64_t n) { return (int)((n + 31) / 32 * 32); };
  if (vec) {
    const int64_t n = a.cols / E;
    if (n <= 4) return launch<T, E, 4, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 8) return launch<T, E, 8, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 16) return launch<T, E, 16, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 32) return launch<T, E, 32, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 64) return launch<T, E, 32, 2, 256, 2, BWD>(a, st, parts);
    if constexpr (sizeof(T) == 2) {
      if (n <= 256) return launch_row<1, 256, BWD ? 3 : 4, BWD>(a, st, parts);
      if (n <= 640) return launch_row<2, 320, BWD ? 2 : 3, BWD>(a, st, parts);
      if (n <= 1024) return launch_row<2, 512, 1, BWD>(a, st, parts);
    } else {
      if (n <= 256) return launch<T, E, 64, 1, 256, kB, BWD>(a, st, parts, warps(n));
      if (n <= 1024) return launch<T, E, 64, 2, 512, 1, BWD>(a, st, parts, warps((n + 1) / 2));
    }
  } else {
    if (a.cols <= 8) return launch<T, 1, 8, 1, 256, kB, BWD>(a, st, parts);
    if (a.cols <= 32) return launch<T, 1, 32, 1, 256, kB, BWD>(a, st, parts);
    if (a.cols <= 160) return launch<T, 1, 32, 5, 256, BWD ? 3 : 4, BWD>(a, st, parts);
    if (a.cols <= 1024) return launch<T, 1, 64, 4, 256, kB, BWD>(a, st, parts, warps((a.cols + 3) / 4));
    if (a.cols <= 4096) return launch<T, 1, 64, 8, 512, 1, BWD>(a, st, parts, warps((a.cols + 7) / 8));
  }
  *wide = true;
  const unsigned grid = (unsigned)(a.rows < 4 * kSMs ? a.rows : 4 * kSMs);
  k_norm_wide<T, BWD><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

ssd_status check(int64_t rows, int64_t cols, ssd_dtype dtype, float eps) {
  if (rows <= 0 || cols <= 0 || (dtype != SSD_F32 && dtype != SSD_BF16) || !(eps >= 0.f)) return SSD_ERR_INVALID_ARG;
  if (rows >= ((int64_t)1 << 31) || cols >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

size_t bwd_workspace(int64_t rows, int64_t cols) {
  return align_up((size_t)2 * kParts * (size_t)cols * 4, kWsAlign) + align_up((size_t)rows * 8, kWsAlign);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" SSD_API ssd_status ssd_layer_norm(const ssd_norm_args* a, void* stream) {
  if (!a) return SSD_ERR_INVALID_ARG;
  const ssd_status c = check(a->rows, a->cols, a->dtype, a->eps);
  if (c != SSD_OK) return c;
  if (!a->x || !a->out) return SSD_ERR_INVALID_ARG;
  const size_t esz = a->dtype == SSD_BF16 ? 2 : 4;
  if (!aligned(a->x, esz) || !aligned(a->out, esz) || !aligned(a->z, esz)) return SSD_ERR_INVALID_ARG;
  Args k = {};
  k.rows = a->rows, k.cols = a->cols, k.eps = a->eps;
  k.x = a->x, k.w = a->weight, k.b = a->bias, k.z = a->z, k.out = a->out;
  const bool vec = a->cols * esz % 16 == 0 && aligned(a->x, 16) && aligned(a->z, 16) && aligned(a->out, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int parts;
  bool wide;
  const cudaError_t e = a->dtype == SSD_BF16 ? launch_rows<__nv_bfloat16, false>(k, vec, st, &parts, &wide)
                                             : launch_rows<float, false>(k, vec, st, &parts, &wide);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

extern "C" SSD_API size_t ssd_layer_norm_bwd_workspace_size(const ssd_norm_bwd_args* a) {
  return a && check(a->rows, a->cols, a->dtype, a->eps) == SSD_OK ? bwd_workspace(a->rows, a->cols) : 0;
}

extern "C" SSD_API ssd_status ssd_layer_norm_bwd(const ssd_norm_bwd_args* a, void* stream) {
  if (!a) return SSD_ERR_INVALID_ARG;
  const ssd_status c = check(a->rows, a->cols, a->dtype, a->eps);
  if (c != SSD_OK) return c;
  if (!a->x || !a->dout || !a->dx || (a->z == nullptr) != (a->dz == nullptr)) return SSD_ERR_INVALID_ARG;
  const size_t esz = a->dtype == SSD_BF16 ? 2 : 4, need = bwd_workspace(a->rows, a->cols);
  for (const void* p : {a->x, a->dout, (const void*)a->dx, a->z, (const void*)a->dz})
    if (!aligned(p, esz)) return SSD_ERR_INVALID_ARG;
  if (!a->workspace || a->workspace_bytes < need) return SSD_ERR_WORKSPACE;
  if (!aligned(a->workspace, kWsAlign)) return SSD_ERR_INVALID_ARG;
  Args k = {};
  k.rows = a->rows, k.cols = a->cols, k.eps = a->eps;
  k.x = a->x, k.w = a->weight, k.b = a->bias, k.z = a->z, k.dout = a->dout, k.out = a->dx, k.dz = a->dz;
  float* part = static_cast<float*>(a->workspace);
  const bool sums = a->dweight || a->dbias;
  k.part = sums ? part : nullptr;
  k.stat = reinterpret_cast<float*>(static_cast<char*>(a->workspace) +
                                    align_up((size_t)2 * kParts * (size_t)a->cols * 4, kWsAlign));
  bool vec = a->cols * esz % 16 == 0;
  for (const void* p : {a->x, a->dout, (const void*)a->dx, a->z, (const void*)a->dz}) vec = vec && aligned(p, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int parts = 0;
  bool wide = false;
  const bool bf16 = a->dtype == SSD_BF16;
  const cudaError_t e = bf16 ? launch_rows<__nv_bfloat16, true>(k, vec, st, &parts, &wide)
                             : launch_rows<float, true>(k, vec, st, &parts, &wide);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  if (!sums) return SSD_OK;
  if (wide) {
    parts = (int)(a->rows < kParts ? a->rows : kParts);
    const dim3 grid((unsigned)((a->cols + kThreads - 1) / kThreads), (unsigned)parts);
    if (bf16) k_norm_wide_cols<__nv_bfloat16><<<grid, kThreads, 0, st>>>(k);
    else k_norm_wide_cols<float><<<grid, kThreads, 0, st>>>(k);
    if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;
  }
  k_norm_sum<<<(unsigned)((a->cols + 31) / 32), kThreads, 0, st>>>(part, parts, a->cols, a->dweight, a->dbias);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
