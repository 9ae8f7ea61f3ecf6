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
constexpr int kThreads = 256;     // CTA of the row kernels
constexpr int kParts = 2 * kSMs;  // CTAs of the backward, each with its partial sums

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

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }
// z sigmoid(z), 0 at z = -inf
__device__ __forceinline__ float silu(float v) { return v == -INFINITY ? 0.f : v * sigmoid(v); }

// Sums over the GT threads of a group, the same bits in each of them.
template <int GT>
struct GroupSum {
  float2 (*red)[kThreads / 32];  // two sets, taken in turn: one barrier a sum
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = (GT < 32 ? GT : 32) / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (GT > 32) {
      if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = make_float2(a, b);
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int w = 0; w < GT / 32; ++w) {
        const float2 v = red[turn][w];
        a += v.x, b += v.y;
      }
      turn ^= 1;
    }
    return make_float2(a, b);
  }
};

// Rows held in registers: VPL packs of E elements a thread.
template <typename T, int E, int GT, int VPL, bool BWD, bool GATE>
__global__ void __launch_bounds__(kThreads) k_norm(const Args a) {
  using Pk = Pack<T, E>;
  constexpr int GC = kThreads / GT;  // groups of a CTA
  __shared__ float2 red[2][kThreads / 32];
  GroupSum<GT> sum{red};
  const int g = threadIdx.x / GT, l = threadIdx.x % GT;
  const int64_t cols = a.cols;
  const float inv_cols = 1.f / (float)cols;
  const auto col = [&](int v) { return (int64_t)(v * GT + l) * E; };
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
    float x[VPL][E], z[VPL][E], d[VPL][E];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool in = live && col(v) < cols;
      xr[v].get(x[v]);
      if constexpr (GATE) zr[v].get(z[v]);
      if constexpr (BWD) dr[v].get(d[v]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!in) x[v][e] = 0.f, z[v][e] = 0.f, d[v][e] = 0.f;
        s += x[v][e];
      }
    }
    fetch(r + stride);
    const float mean = sum(s, 0.f).x * inv_cols;
    s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[v][e] = col(v) < cols ? x[v][e] - mean : 0.f;
        s = fmaf(x[v][e], x[v][e], s);
      }
    const float rstd = 1.f / sqrtf(fmaf(sum(s, 0.f).x, inv_cols, a.eps));
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
      float s1 = 0.f, s2 = 0.f;
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
          const float hw = h * w[v][e];
          s1 += hw;
          s2 = fmaf(hw, n, s2);
          x[v][e] = n, d[v][e] = hw;
        }
        if constexpr (GATE)
          if (live && col(v) < cols) Pk::store(static_cast<T*>(a.dz) + r * cols + col(v), dz);
      }
      const float2 m = sum(s1, s2);
      const float m1 = m.x * inv_cols, m2 = m.y * inv_cols;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = rstd * (d[v][e] - m1 - x[v][e] * m2);
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

// Rows too wide for registers: one CTA a row at a time, swept from memory.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) k_norm_wide(const Args a) {
  __shared__ float2 red[2][kThreads / 32];
  GroupSum<kThreads> sum{red};
  const int64_t cols = a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * cols;
    const T* z = a.z ? static_cast<const T*>(a.z) + r * cols : nullptr;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) s += to_f(x[c]);
    const float mean = sum(s, 0.f).x / (float)cols;
    s = 0.f;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
      const float d = to_f(x[c]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(sum(s, 0.f).x / (float)cols + a.eps);
    if constexpr (!BWD) {
      T* y = static_cast<T*>(a.out) + r * cols;
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        float v = fmaf((to_f(x[c]) - mean) * rstd, a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f);
        if (z) v *= silu(to_f(z[c]));
        put(y + c, v);
      }
    } else {
      const T* dout = static_cast<const T*>(a.dout) + r * cols;
      float s1 = 0.f, s2 = 0.f;
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
        s1 += h * w;
        s2 = fmaf(h * w, n, s2);
      }
      const float2 m = sum(s1, s2);
      const float m1 = m.x / (float)cols, m2 = m.y / (float)cols;
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

template <typename T, int E, int GT, int VPL, bool BWD>
cudaError_t launch(const Args& a, cudaStream_t st, int* parts) {
  constexpr int GC = kThreads / GT;
  const int64_t need = (a.rows + GC - 1) / GC, most = BWD ? kParts : 8 * kSMs;
  const unsigned grid = (unsigned)(need < most ? need : most);
  *parts = (int)grid;
  if (a.z) k_norm<T, E, GT, VPL, BWD, true><<<grid, kThreads, 0, st>>>(a);
  else k_norm<T, E, GT, VPL, BWD, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// The group and the packs of a thread by the row's packs: part of a warp up to
// 128 packs (no barrier), else a CTA.
template <typename T, bool BWD>
cudaError_t launch_rows(const Args& a, bool vec, cudaStream_t st, int* parts, bool* wide) {
  constexpr int E = 16 / (int)sizeof(T);
  *wide = false;
  if (vec) {
    const int64_t n = (a.cols + E - 1) / E;
    if (n <= 4) return launch<T, E, 4, 1, BWD>(a, st, parts);
    if (n <= 8) return launch<T, E, 8, 1, BWD>(a, st, parts);
    if (n <= 16) return launch<T, E, 16, 1, BWD>(a, st, parts);
    if (n <= 32) return launch<T, E, 32, 1, BWD>(a, st, parts);
    if (n <= 64) return launch<T, E, 32, 2, BWD>(a, st, parts);
    if (n <= 256) return launch<T, E, 256, 1, BWD>(a, st, parts);
    if (n <= 512) return launch<T, E, 256, 2, BWD>(a, st, parts);
    if (n <= 768) return launch<T, E, 256, 3, BWD>(a, st, parts);
    if (n <= 1024) return launch<T, E, 256, 4, BWD>(a, st, parts);
  } else {
    if (a.cols <= 8) return launch<T, 1, 8, 1, BWD>(a, st, parts);
    if (a.cols <= 32) return launch<T, 1, 32, 1, BWD>(a, st, parts);
    if (a.cols <= 160) return launch<T, 1, 32, 5, BWD>(a, st, parts);
    if (a.cols <= 1024) return launch<T, 1, 256, 4, BWD>(a, st, parts);
    if (a.cols <= 4096) return launch<T, 1, 256, 16, BWD>(a, st, parts);
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
