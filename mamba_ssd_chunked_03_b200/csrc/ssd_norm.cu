// Layer norm over the last axis with the block's gate, forward and backward:
//     y = ((x - mean) rstd w + b) SiLU(z)
//     dx = rstd (hw - mean(hw) - n mean(hw n)),  n = (x - mean) rstd, hw = dout SiLU(z) w
//     dw = sum_rows dout SiLU(z) n,  db = sum_rows dout SiLU(z)
//     dz = dout (n w + b) SiLU'(z)
//
// Bound by HBM: every tensor is read once and every output written once, but for
// rows that are swept from memory (below).  A
// row belongs to a group of GT threads (part of a warp, or a whole CTA), which
// holds it in registers: the mean first, then the mean square of the
// differences to it, so that a large mean costs no accuracy.  In fp32 the
// differences' own mean is taken out of them again: it is what the rounding of
// the mean is off by.  In bf16 the sum of equal values is exact (8 bits each), so
// a mean divided without error leaves zeros, and other rows deviate by more than
// the mean's rounding shows.  Groups walk the rows with a fixed stride and load
// the next row before they work on this one; weights, biases and the sums of
// their gradients stay in registers all the way.  The backward's partial sums (one set a CTA) are added by a second
// kernel in a fixed order.  Rows wider than the registers hold are swept
// several times from memory instead, with the column sums in a pass of their
// own.  1.3 M rows of 64, gated, bf16: 86 us, 5.8 TB/s (the call 91); 100003
// rows of 129, gated, fp32, backward: 70 us, 3.7 TB/s (bound by the instructions
// of its four-byte loads and of the gate); 7 rows of 5120: 3.7 us, a chain of
// latencies.
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
constexpr int kParts = 3 * kSMs;  // most CTAs of the backward whose rows do not each take a CTA

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
  float* part;  // backward: [2][CTAs][cols] partial sums of dw, db, or null
  float* stat;  // wide rows: [rows][3] mean, rstd, and what the mean's rounding takes off n
};

// Arithmetic on one value or on two at once (half the instructions).
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float total(float a) { return a; }
__device__ __forceinline__ float total(float2 a) { return a.x + a.y; }
template <typename V>
__device__ __forceinline__ V all(float v);
template <>
__device__ __forceinline__ float all<float>(float v) { return v; }
template <>
__device__ __forceinline__ float2 all<float2>(float v) { return make_float2(v, v); }

// E consecutive elements as they are loaded and stored, and as EV values of type V.
template <typename T, int E>
struct Pack;
template <>
struct Pack<float, 4> {
  using V = float2;
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[2]) const { f[0] = make_float2(r.x, r.y), f[1] = make_float2(r.z, r.w); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void store(float* p, const float2 (&f)[2]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  using V = float2;
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __float22bfloat162_rn(f[i]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Pack<float, 2> {
  using V = float2;
  float2 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[1]) const { f[0] = r; }
  __device__ __forceinline__ void zero() { r = make_float2(0.f, 0.f); }
  static __device__ __forceinline__ void store(float* p, const float2 (&f)[1]) { *reinterpret_cast<float2*>(p) = f[0]; }
};
template <>
struct Pack<__nv_bfloat16, 2> {
  using V = float2;
  uint32_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void get(float2 (&f)[1]) const {
    f[0] = make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  __device__ __forceinline__ void zero() { r = 0; }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[1]) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(f[0]);
  }
};
template <>
struct Pack<float, 1> {
  using V = float;
  float r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(p); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = r; }
  __device__ __forceinline__ void zero() { r = 0.f; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  using V = float;
  __nv_bfloat16 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(r); }
  __device__ __forceinline__ void zero() { r = __float2bfloat16_rn(0.f); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// In fp32 by e^-|v|, so that nothing overflows and a far negative v keeps its
// relative accuracy, with a divisor between 1 and 2: off by a few 2^-23 of the
// value.  For a result in bf16 the hardware exponential, whose relative error
// grows with |v| (some |v| 2^-23: 2^-16 at -87, where its rounding is 2^-8), and
// which the divide takes for infinite below -87.3: zero there in place of 1e-36.
// (The fp32 form on bf16 rows of 64 takes 110 us against 91; on fp32 rows of 129,
// backward, 76 against 70.)
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-v));
  const float t = expf(-fabsf(v));
  return __fdividef(v < 0.f ? t : 1.f, 1.f + t);
}
// The gate bounded below where SiLU and its derivative are zero: -inf would
// give 0 x inf.  NaN stays NaN.
__device__ __forceinline__ float bounded(float v) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(-1e30f));
  return v;
}
__device__ __forceinline__ float2 bounded(float2 v) { return make_float2(bounded(v.x), bounded(v.y)); }
template <typename T>
__device__ __forceinline__ float2 sigmoid(float2 v) { return make_float2(sigmoid<T>(v.x), sigmoid<T>(v.y)); }
// z sigmoid(z)
template <typename T>
__device__ __forceinline__ float silu(float v) {
  v = bounded(v);
  return v * sigmoid<T>(v);
}
template <typename T>
__device__ __forceinline__ float2 silu(float2 v) { return make_float2(silu<T>(v.x), silu<T>(v.y)); }

// (var + eps)^-1/2, for a variance that rounding may have taken below zero.  NaN
// stays NaN, so that a row with an infinity or a NaN is NaN throughout.
__device__ __forceinline__ float inv_dev(float var, float eps) { return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps); }

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
  constexpr bool kTwice = sizeof(T) == 4;          // the differences' mean is taken out too
  __shared__ float4 red[2][kMostThreads / 32];
  GroupSum<GT> sum{red};
  const int gt = GT > 32 ? blockDim.x : GT;  // threads of a row
  const int g = GT > 32 ? 0 : threadIdx.x / GT, l = GT > 32 ? threadIdx.x : threadIdx.x % GT;
  const int64_t cols = a.cols;
  const float inv_cols = 1.f / (float)cols;
  const auto col = [&](int v) { return (int64_t)(v * gt + l) * E; };
  using V = typename Pk::V;
  constexpr int EV = E * (int)sizeof(float) / (int)sizeof(V);  // values of type V
  V w[VPL][EV], b[VPL][EV], dw[VPL][EV], db[VPL][EV];
  Pk xr[VPL], zr[VPL], dr[VPL];  // zeros for ever where the row has no columns
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float wv[E], bv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = col(v) < cols;
      wv[e] = a.w && in ? a.w[col(v) + e] : 1.f;
      bv[e] = a.b && in ? a.b[col(v) + e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      w[v][e] = *reinterpret_cast<const V*>(wv + e * (E / EV)), b[v][e] = *reinterpret_cast<const V*>(bv + e * (E / EV));
      dw[v][e] = db[v][e] = all<V>(0.f);
    }
    xr[v].zero(), zr[v].zero(), dr[v].zero();
  }
  const auto fetch = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (r < a.rows) {
        if (col(v) < cols) {
          xr[v].load(static_cast<const T*>(a.x) + r * cols + col(v));
          if constexpr (GATE) zr[v].load(static_cast<const T*>(a.z) + r * cols + col(v));
          if constexpr (BWD) dr[v].load(static_cast<const T*>(a.dout) + r * cols + col(v));
        }
      } else if constexpr (BWD) {
        dr[v].zero();  // no such row: it must not count
      }
    }
  };
  const int64_t stride = (int64_t)gridDim.x * GC;
  fetch((int64_t)blockIdx.x * GC + g);
  for (int64_t r0 = (int64_t)blockIdx.x * GC; r0 < a.rows; r0 += stride) {  // the same trips for all threads
    const int64_t r = r0 + g;
    const bool live = r < a.rows;
    V x[VPL][EV], z[VPL][EV], d[VPL][EV];  // x - mean, the gate, and dout: then dout SiLU(z)
    V s0 = all<V>(0.f), s1 = all<V>(0.f), sq = all<V>(0.f);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      xr[v].get(x[v]);
      if constexpr (GATE) zr[v].get(z[v]);
      if constexpr (BWD) dr[v].get(d[v]);
#pragma unroll
      for (int e = 0; e < EV; ++e) s0 = add(s0, x[v][e]);
    }
    fetch(r + stride);
    float t[1] = {total(s0)};
    sum(t);
    float mean = t[0] * inv_cols;
    if constexpr (!kTwice) mean = fmaf(fmaf(-mean, (float)cols, t[0]), inv_cols, mean);
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        x[v][e] = add(x[v][e], all<V>(col(v) < cols ? -mean : 0.f));
        if constexpr (kTwice) s1 = add(s1, x[v][e]);
        sq = fma_(x[v][e], x[v][e], sq);
      }
    float u[kTwice ? 2 : 1] = {total(sq)}, dm = 0.f;
    if constexpr (kTwice) u[1] = total(s1);
    sum(u);
    if constexpr (kTwice) dm = u[1] * inv_cols;
    const float rstd = live ? inv_dev(fmaf(u[0], inv_cols, -dm * dm), a.eps) : 0.f;
    const V scale = all<V>(rstd), shift = all<V>(-dm * rstd);
    const auto normed = [&](V c) {
      if constexpr (kTwice) return fma_(c, scale, shift);
      else return mul(c, scale);
    };
    if constexpr (!BWD) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        V y[EV];
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          y[e] = fma_(normed(x[v][e]), w[v][e], b[v][e]);
          if constexpr (GATE) y[e] = mul(y[e], silu<T>(z[v][e]));
        }
        if (live && col(v) < cols) Pk::store(static_cast<T*>(a.out) + r * cols + col(v), y);
      }
    } else {
      V p1 = all<V>(0.f), p2 = all<V>(0.f);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        V dz[EV];
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          x[v][e] = normed(x[v][e]);
          V h = d[v][e];
          if constexpr (GATE) {  // SiLU' = s + z s (1 - s)
            const V zb = bounded(z[v][e]), sg = sigmoid<T>(zb), zs = mul(zb, sg);
            dz[e] = mul(mul(h, fma_(x[v][e], w[v][e], b[v][e])), fma_(zs, fma_(sg, all<V>(-1.f), all<V>(1.f)), sg));
            h = mul(h, zs);
          }
          dw[v][e] = fma_(h, x[v][e], dw[v][e]);
          db[v][e] = add(db[v][e], h);
          d[v][e] = mul(h, w[v][e]);
          p1 = add(p1, d[v][e]);
          p2 = fma_(d[v][e], x[v][e], p2);
        }
        if constexpr (GATE)
          if (live && col(v) < cols) Pk::store(static_cast<T*>(a.dz) + r * cols + col(v), dz);
      }
      float m[2] = {total(p1), total(p2)};
      sum(m);
      const V m1 = all<V>(-m[0] * inv_cols), m2 = all<V>(-m[1] * inv_cols);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        V y[EV];
#pragma unroll
        for (int e = 0; e < EV; ++e) y[e] = mul(all<V>(rstd), add(fma_(x[v][e], m2, d[v][e]), m1));
        if (live && col(v) < cols) Pk::store(static_cast<T*>(a.out) + r * cols + col(v), y);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // the CTA's groups added in order, one set of partial sums a CTA
    float* pw = a.part + blockIdx.x * cols;
    float* pb = pw + (int64_t)gridDim.x * cols;
    const auto at = [](const V (&x)[EV], int e) { return reinterpret_cast<const float*>(&x)[e]; };
    if constexpr (GC == 1) {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (col(v) < cols) {
#pragma unroll
          for (int e = 0; e < E; ++e) pw[col(v) + e] = at(dw[v], e), pb[col(v) + e] = at(db[v], e);
        }
    } else {
      // groups of a warp by shuffles, then the warps through shared memory
      __shared__ float2 all[kThreads / 32][32][E];
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float p = at(dw[v], e), q = at(db[v], e);
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

__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}

// Rows of bf16 that take a CTA.
//
// Such a row costs a barrier for every sum that waits for another one, so all
// of its sums are taken at once, of the differences to K, the mean of the
// row's first pack: x - mean = (x - K) - mean(x - K), var = mean((x - K)^2) -
// mean(x - K)^2.  K is off the mean by at most sqrt(cols / 8) deviations, since
// its elements are part of the row, and by less than one in all but contrived
// rows; what cancels in var is then cols / 8 x 2^-24 at the very most, far
// below the rounding of the outputs.  A thread copies its packs of the next
// rows into a ring of its own in shared memory, where a second look at them
// after the sums costs nothing; weight and bias lie there too.  That leaves the
// registers to the column sums, and room for two rows at a time where a row has
// two tensors at most: what takes the time is the chain of a row's sums through
// the barrier, and two rows share one.  (16384 rows of 5120, backward: 138 us
// with rows held in registers, 122 us from the ring one at a time, 117 us two
// at a time: 4.3 TB/s.  Three CTAs an SM with half the ring took 133 us.
// Forward, the same rows: 100 us, with the gate 154, 0.5 of a copy's rate.)
template <int VPL, bool BWD, bool GATE>
struct RowRing {
  static constexpr int kTensors = 1 + GATE + BWD;
  static constexpr int kRows = kTensors == 3 ? 1 : 2;  // at a time; as many again are on their way
  static constexpr size_t bytes(int threads, int64_t cols) {
    return (size_t)2 * kRows * kTensors * VPL * threads * 16 + (size_t)cols * (BWD && !GATE ? 4 : 8);
  }
};
template <int VPL, int BT, int MINB, bool BWD, bool GATE>
__global__ void __launch_bounds__(BT, MINB) k_norm_row(const Args a) {
  using T = __nv_bfloat16;
  constexpr int E = 8;
  using Pk = Pack<T, E>;
  using R = RowRing<VPL, BWD, GATE>;
  extern __shared__ __align__(16) uint4 ring[];  // [row][tensor][pack][thread]
  constexpr int NR = R::kRows, NS = BWD ? 4 : 2;
  float* const wb = reinterpret_cast<float*>(ring + 2 * NR * R::kTensors * VPL * blockDim.x);  // weight, bias
  __shared__ float4 red[2][NR][kMostThreads / 32];  // two sets, taken in turn
  const int l = threadIdx.x, gt = blockDim.x, cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const auto col = [&](int v) { return (v * gt + l) * E; };
  for (int c = l; c < cols; c += gt) {
    wb[c] = a.w ? a.w[c] : 1.f;
    if constexpr (GATE || !BWD) wb[cols + c] = a.b ? a.b[c] : 0.f;
  }
  __syncthreads();
  using V = float2;
  constexpr int EV = E / 2;
  const auto weights = [&](int c, V (&w)[EV]) {
    const float4 p = *reinterpret_cast<const float4*>(wb + c), q = *reinterpret_cast<const float4*>(wb + c + 4);
    w[0] = make_float2(p.x, p.y), w[1] = make_float2(p.z, p.w), w[2] = make_float2(q.x, q.y), w[3] = make_float2(q.z, q.w);
  };
  V dw[BWD ? VPL : 1][EV], db[BWD ? VPL : 1][EV];
#pragma unroll
  for (int v = 0; v < (BWD ? VPL : 1); ++v)
#pragma unroll
    for (int e = 0; e < EV; ++e) dw[v][e] = db[v][e] = all<V>(0.f);
  // x, dout, z: tensor t of row q of the rows at hand (set 0 or 1)
  const auto place = [&](int set, int q, int t, int v) { return ring + (((set * NR + q) * R::kTensors + t) * VPL + v) * gt + l; };
  const auto fetch = [&](int64_t r0, int set) {
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int64_t r = r0 + (int64_t)q * gridDim.x, o = r * cols;
      if (r >= a.rows) continue;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (col(v) < cols) {
          copy16(place(set, q, 0, v), static_cast<const T*>(a.x) + o + col(v));
          if constexpr (BWD) copy16(place(set, q, 1, v), static_cast<const T*>(a.dout) + o + col(v));
          if constexpr (GATE) copy16(place(set, q, 1 + BWD, v), static_cast<const T*>(a.z) + o + col(v));
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Pk kn[NR];
  const auto first = [&](int64_t r0) {
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int64_t r = r0 + (int64_t)q * gridDim.x;
      if (r < a.rows) kn[q].load(static_cast<const T*>(a.x) + r * cols);
      else kn[q].zero();
    }
  };
  const int64_t step = (int64_t)NR * gridDim.x;
  first(blockIdx.x);
  fetch(blockIdx.x, 0);
  int set = 0;
  for (int64_t r0 = blockIdx.x; r0 < a.rows; r0 += step, set ^= 1) {
    fetch(r0 + step, set ^ 1);
    float K[NR];
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      V k[EV];
      kn[q].get(k);
      K[q] = total(add(add(k[0], k[1]), add(k[2], k[3]))) * (1.f / E);
    }
    first(r0 + step);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const auto see = [&](int q, int t, int v, V (&f)[EV]) {
      Pk p;
      p.r = *place(set, q, t, v);
      p.get(f);
    };
    float t[NR][NS];
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      V p0 = all<V>(0.f), p1 = p0, p2 = p0, p3 = p0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        if (col(v) >= cols || r0 + (int64_t)q * gridDim.x >= a.rows) continue;
        V x[EV], d[EV], z[EV], w[EV];
        see(q, 0, v, x);
        if constexpr (BWD) {
          see(q, 1, v, d);
          weights(col(v), w);
        }
        if constexpr (BWD && GATE) see(q, 1 + BWD, v, z);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          x[e] = add(x[e], all<V>(-K[q]));
          p0 = add(p0, x[e]);
          p1 = fma_(x[e], x[e], p1);
          if constexpr (BWD) {
            V h = mul(d[e], w[e]);
            if constexpr (GATE) h = mul(h, silu<T>(z[e]));
            p2 = add(p2, h);
            p3 = fma_(h, x[e], p3);
          }
        }
      }
      t[q][0] = total(p0), t[q][1] = total(p1);
      if constexpr (BWD) t[q][2] = total(p2), t[q][3] = total(p3);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int i = 0; i < NS; ++i) t[q][i] += __shfl_xor_sync(0xffffffffu, t[q][i], o);
    if ((l & 31) == 0) {
#pragma unroll
      for (int q = 0; q < NR; ++q) red[set][q][l >> 5] = make_float4(t[q][0], t[q][1], t[q][NS - 2], t[q][NS - 1]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NR; ++q) {
#pragma unroll
      for (int i = 0; i < NS; ++i) t[q][i] = 0.f;
#pragma unroll 5
      for (int i = 0; i < (gt >> 5); ++i) {
        const float4 x = red[set][q][i];
        t[q][0] += x.x, t[q][1] += x.y;
        if constexpr (BWD) t[q][2] += x.z, t[q][3] += x.w;
      }
    }
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int64_t r = r0 + (int64_t)q * gridDim.x;
      if (r >= a.rows) continue;
      const float dm = t[q][0] * inv_cols;
      const float rstd = inv_dev(fmaf(t[q][1], inv_cols, -dm * dm), a.eps);
      float m1 = 0.f, m2 = 0.f;
      if constexpr (BWD) m1 = t[q][2] * inv_cols, m2 = rstd * (t[q][3] - dm * t[q][2]) * inv_cols;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        if (col(v) >= cols) continue;
        V x[EV], d[EV], z[EV], w[EV], b[EV], dz[EV];
        see(q, 0, v, x);
        if constexpr (BWD) see(q, 1, v, d);
        if constexpr (GATE) see(q, 1 + BWD, v, z);
        weights(col(v), w);
        if constexpr (GATE || !BWD) weights(cols + col(v), b);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const V n = fma_(add(x[e], all<V>(-K[q])), all<V>(rstd), all<V>(-dm * rstd));
          if constexpr (!BWD) {
            x[e] = fma_(n, w[e], b[e]);
            if constexpr (GATE) x[e] = mul(x[e], silu<T>(z[e]));
          } else {
            V h = d[e];
            if constexpr (GATE) {
              const V zb = bounded(z[e]), sg = sigmoid<T>(zb), zs = mul(zb, sg);
              dz[e] = mul(mul(h, fma_(n, w[e], b[e])), fma_(zs, fma_(sg, all<V>(-1.f), all<V>(1.f)), sg));
              h = mul(h, zs);
            }
            dw[v][e] = fma_(h, n, dw[v][e]);
            db[v][e] = add(db[v][e], h);
            x[e] = mul(all<V>(rstd), add(fma_(n, all<V>(-m2), mul(h, w[e])), all<V>(-m1)));
          }
        }
        Pk::store(static_cast<T*>(a.out) + r * cols + col(v), x);
        if constexpr (BWD && GATE) Pk::store(static_cast<T*>(a.dz) + r * cols + col(v), dz);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    float* pw = a.part + (int64_t)blockIdx.x * cols;
    float* pb = pw + (int64_t)gridDim.x * cols;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (col(v) < cols) {
#pragma unroll
        for (int e = 0; e < EV; e += 2) {
          *reinterpret_cast<float4*>(pw + col(v) + 2 * e) = make_float4(dw[v][e].x, dw[v][e].y, dw[v][e + 1].x, dw[v][e + 1].y);
          *reinterpret_cast<float4*>(pb + col(v) + 2 * e) = make_float4(db[v][e].x, db[v][e].y, db[v][e + 1].x, db[v][e + 1].y);
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
    float s[1] = {0.f}, q[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) s[0] += to_f(x[c]);
    sum(s);
    const float mean = s[0] / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
      const float d = to_f(x[c]) - mean;
      q[0] += d, q[1] = fmaf(d, d, q[1]);
    }
    sum(q);
    const float dm = q[0] / (float)cols;
    const float rstd = inv_dev(q[1] / (float)cols - dm * dm, a.eps), shift = -dm * rstd;
    if constexpr (!BWD) {
      T* y = static_cast<T*>(a.out) + r * cols;
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        float v = fmaf(fmaf(to_f(x[c]) - mean, rstd, shift), a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f);
        if (z) v *= silu<T>(to_f(z[c]));
        put(y + c, v);
      }
    } else {
      const T* dout = static_cast<const T*>(a.dout) + r * cols;
      float m[2] = {0.f, 0.f};
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = fmaf(to_f(x[c]) - mean, rstd, shift);
        float h = to_f(dout[c]);
        const float w = a.w ? a.w[c] : 1.f;
        if (z) {
          const float zv = bounded(to_f(z[c])), sg = sigmoid<T>(zv);
          put(static_cast<T*>(a.dz) + r * cols + c,
              h * fmaf(n, w, a.b ? a.b[c] : 0.f) * (sg * fmaf(zv, 1.f - sg, 1.f)));
          h *= zv * sg;
        }
        m[0] += h * w;
        m[1] = fmaf(h * w, n, m[1]);
      }
      sum(m);
      const float m1 = m[0] / (float)cols, m2 = m[1] / (float)cols;
      if (threadIdx.x == 0) a.stat[3 * r] = mean, a.stat[3 * r + 1] = rstd, a.stat[3 * r + 2] = shift;
      T* dx = static_cast<T*>(a.out) + r * cols;
      for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
        const float n = fmaf(to_f(x[c]) - mean, rstd, shift);
        float h = to_f(dout[c]);
        if (z) h *= silu<T>(to_f(z[c]));
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
    const float n = fmaf(to_f(static_cast<const T*>(a.x)[r * cols + c]) - a.stat[3 * r], a.stat[3 * r + 1], a.stat[3 * r + 2]);
    float h = to_f(static_cast<const T*>(a.dout)[r * cols + c]);
    if (a.z) h *= silu<T>(to_f(static_cast<const T*>(a.z)[r * cols + c]));
    dw = fmaf(h, n, dw);
    db += h;
  }
  a.part[blockIdx.y * cols + c] = dw;
  a.part[((int64_t)gridDim.y + blockIdx.y) * cols + c] = db;
}

// dw and db from the partial sums: 32 columns a CTA, 32 strands of parts each,
// the strands added in order.
constexpr int kSumThreads = 1024, kStrands = kSumThreads / 32;
__global__ void __launch_bounds__(kSumThreads) k_norm_sum(const float* __restrict__ part, int parts, int64_t cols,
                                                       float* dw, float* db) {
  __shared__ double s[2][kStrands][32];
  const int l = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  double p = 0., q = 0.;
  if (c < cols) {
#pragma unroll 4
    for (int i = g; i < parts; i += kStrands) {
      p += part[i * cols + c];
      q += part[((int64_t)parts + i) * cols + c];
    }
  }
  s[0][g][l] = p, s[1][g][l] = q;
  __syncthreads();
  if (g < 2 && c < cols) {
    double t = 0.;
#pragma unroll
    for (int i = 0; i < kStrands; ++i) t += s[g][i][l];
    if (g == 0 && dw) dw[c] = (float)t;
    if (g == 1 && db) db[c] = (float)t;
  }
}

// CTAs of a grid with `threads` an SM (at most 16 an SM).
int64_t ctas(int per_sm, int threads) {
  const int n = per_sm / threads;
  return (int64_t)kSMs * (n < 1 ? 1 : n > 16 ? 16 : n);
}
constexpr int kRowParts = 16384;  // CTAs of an SM times columns, where a row takes a CTA, are at most this

// One grid of the CTAs that registers allow: MINB of BT threads an SM, or more of
// fewer.  (The ring of a wide row can allow fewer still: two of three at 5120
// columns forward, one with the gate, and the grid then runs in two or three
// parts.)  `threads`: of a CTA that takes one row;
// else GT threads take one.
template <typename T, int E, int GT, int VPL, int BT, int MINB, bool BWD>
cudaError_t launch(const Args& a, cudaStream_t st, int* parts, int threads = kThreads) {
  constexpr int GC = GT > 32 ? 1 : kThreads / GT;
  const int64_t need = (a.rows + GC - 1) / GC, most = ctas(MINB * BT, threads);
  static_assert(!BWD || (GT > 32 ? MINB * BT * E * VPL <= kRowParts : MINB * kSMs <= kParts), "partial sums");
  const unsigned grid = (unsigned)(need < most ? need : most);
  *parts = (int)grid;
  if (a.z) k_norm<T, E, GT, VPL, BT, MINB, BWD, true><<<grid, threads, 0, st>>>(a);
  else k_norm<T, E, GT, VPL, BT, MINB, BWD, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}
template <int VPL, int BT, int MINB, bool BWD>
cudaError_t launch_row(const Args& a, cudaStream_t st, int* parts) {
  const unsigned threads = (unsigned)((a.cols / 8 + 32 * VPL - 1) / (32 * VPL) * 32);
  const int64_t most = ctas(MINB * BT, (int)threads);
  static_assert(!BWD || MINB * BT * 8 * VPL <= kRowParts, "partial sums");
  const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
  *parts = (int)grid;
  constexpr int kMost = BT * VPL * 8;  // columns
  static std::atomic<uint64_t> seen[2] = {};
  if (a.z) {
    using R = RowRing<VPL, BWD, true>;
    return launch_kernel(k_norm_row<VPL, BT, MINB, BWD, true>, seen[1], grid, threads, R::bytes(threads, a.cols),
                         R::bytes(BT, kMost), false, st, a);
  }
  using R = RowRing<VPL, BWD, false>;
  return launch_kernel(k_norm_row<VPL, BT, MINB, BWD, false>, seen[0], grid, threads, R::bytes(threads, a.cols),
                       R::bytes(BT, kMost), false, st, a);
}

// Rows that 16-byte packs do not divide, in pairs or single elements: half a
// row to an eighth of the loads' width.  Up to 160 of them lie in one warp, five a
// lane, and cost no barrier; then in a CTA of four, then eight a thread.
template <typename T, int E, bool BWD>
cudaError_t launch_narrow(const Args& a, cudaStream_t st, int* parts, bool* wide) {
  constexpr int kB = BWD ? 2 : 4;
  const int64_t n = a.cols / E;
  const auto warps = [](int64_t n) { return (int)((n + 31) / 32 * 32); };
  if (n <= 8) return launch<T, E, 8, 1, 256, kB, BWD>(a, st, parts);
  if (n <= 32) return launch<T, E, 32, 1, 256, kB, BWD>(a, st, parts);
  if (n <= 64) return launch<T, E, 32, 2, 256, kB, BWD>(a, st, parts);
  if (n <= 160) return launch<T, E, 32, 5, 256, BWD ? (E == 1 ? 3 : 2) : (E == 1 ? 4 : 3), BWD>(a, st, parts);
  if (n <= 1024) return launch<T, E, 64, 4, 256, kB, BWD>(a, st, parts, warps((n + 3) / 4));
  if (n <= 4096) return launch<T, E, 64, 8, 512, BWD || E == 2 ? 1 : 2, BWD>(a, st, parts, warps((n + 7) / 8));
  *wide = true;
  return cudaSuccess;
}

// The group by the row's packs: part of a warp up to 64 packs (no barrier),
// else a CTA of as many threads as the row needs with one or two packs each.  The
// steps between them are where a CTA's threads run out at the registers that its
// packs take: 256 of one pack, 320 of two with two CTAs an SM left (three forward),
// 512 of two with one.
// `vec`: elements to which every row is aligned (E, 2 or 1).  Where a row's
// registers or its ring end, at 1024 packs, 4096 pairs or 4096 single elements, it
// is swept from memory.  In fp32 that puts aligned rows of 4100 to 8192 columns
// behind those that only pairs divide: 16384 rows of 5120 take 193 us forward, 442
// gated, 397 and 922 backward, where 5122 columns take 170, 258, 328 and 956;
// packs held beyond 1024 are not built.  bf16 rows of 10240 (8192 of them): 190,
// 385, 416 and 786 us, 0.16 to 0.27 of a copy's rate.
template <typename T, bool BWD>
cudaError_t launch_rows(const Args& a, int vec, cudaStream_t st, int* parts, bool* wide) {
  constexpr int E = 16 / (int)sizeof(T), kB = BWD ? 2 : 4;
  *wide = false;
  const auto warps = [](int64_t n) { return (int)((n + 31) / 32 * 32); };
  const int64_t n = a.cols / E;
  if (vec == E && n <= 1024) {
    if (n <= 4) return launch<T, E, 4, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 8) return launch<T, E, 8, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 16) return launch<T, E, 16, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 32) return launch<T, E, 32, 1, 256, kB, BWD>(a, st, parts);
    if (n <= 64) return launch<T, E, 32, 2, 256, 2, BWD>(a, st, parts);
    if constexpr (sizeof(T) == 2) {
      if (n <= 256) return launch_row<1, 256, BWD ? 3 : 4, BWD>(a, st, parts);
      if (n <= 640) return launch_row<2, 320, BWD ? 2 : 3, BWD>(a, st, parts);
      return launch_row<2, 512, 1, BWD>(a, st, parts);
    } else {
      if (n <= 256) return launch<T, E, 64, 1, 256, kB, BWD>(a, st, parts, warps(n));
      return launch<T, E, 64, 2, 512, 1, BWD>(a, st, parts, warps((n + 1) / 2));
    }
  }
  if (vec != E) {
    const cudaError_t e =
        vec == 2 ? launch_narrow<T, 2, BWD>(a, st, parts, wide) : launch_narrow<T, 1, BWD>(a, st, parts, wide);
    if (!*wide) return e;
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

// Partial sums, one set for each CTA (no more of them than rows), then the
// statistics of rows that are swept from memory: none of up to 4096 columns is,
// wherever they start.
size_t part_bytes(int64_t rows, int64_t cols) {
  const int64_t grid = kParts * cols, row = (int64_t)kSMs * kRowParts, all = rows * cols, most = grid > row ? grid : row;
  return align_up((size_t)(all < most ? all : most) * 2 * 4, kWsAlign);
}
size_t bwd_workspace(int64_t rows, int64_t cols) {
  return part_bytes(rows, cols) + (cols > 4096 ? align_up((size_t)rows * 12, kWsAlign) : 0);
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
  if (!aligned(a->x, esz) || !aligned(a->out, esz) || !aligned(a->z, esz) || !aligned(a->weight, 4) || !aligned(a->bias, 4))
    return SSD_ERR_INVALID_ARG;
  Args k = {};
  k.rows = a->rows, k.cols = a->cols, k.eps = a->eps;
  k.x = a->x, k.w = a->weight, k.b = a->bias, k.z = a->z, k.out = a->out;
  const auto all_at = [&](size_t n) {
    return a->cols * esz % n == 0 && aligned(a->x, n) && aligned(a->z, n) && aligned(a->out, n);
  };
  const int vec = all_at(16) ? (int)(16 / esz) : all_at(2 * esz) ? 2 : 1;
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
  for (const void* p : {(const void*)a->weight, (const void*)a->bias, (const void*)a->dweight, (const void*)a->dbias})
    if (!aligned(p, 4)) return SSD_ERR_INVALID_ARG;
  if (!a->workspace || a->workspace_bytes < need) return SSD_ERR_WORKSPACE;
  if (!aligned(a->workspace, kWsAlign)) return SSD_ERR_INVALID_ARG;
  Args k = {};
  k.rows = a->rows, k.cols = a->cols, k.eps = a->eps;
  k.x = a->x, k.w = a->weight, k.b = a->bias, k.z = a->z, k.dout = a->dout, k.out = a->dx, k.dz = a->dz;
  float* part = static_cast<float*>(a->workspace);
  const bool sums = a->dweight || a->dbias;
  k.part = sums ? part : nullptr;
  k.stat = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + part_bytes(a->rows, a->cols));
  const auto all_at = [&](size_t n) {
    bool is = a->cols * esz % n == 0;
    for (const void* p : {a->x, a->dout, (const void*)a->dx, a->z, (const void*)a->dz}) is = is && aligned(p, n);
    return is;
  };
  const int vec = all_at(16) ? (int)(16 / esz) : all_at(2 * esz) ? 2 : 1;
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
  k_norm_sum<<<(unsigned)((a->cols + 31) / 32), kSumThreads, 0, st>>>(part, parts, a->cols, a->dweight, a->dbias);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
