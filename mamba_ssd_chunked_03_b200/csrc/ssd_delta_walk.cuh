// The forward walk of the gated delta rule (ssd_delta_prep.cuh has the
// formulas): one CTA carries 64 rows (headdim) of one head's state through one
// sequence, 32 tokens at a time.
//
// Each of its four warps owns 16 rows p of the state for all N columns, in
// registers, as the accumulator tiles of the matrix instruction.  Every
// product of a chunk has m = p, so the result of one is the operand of the
// next without leaving the warp: K S^T (A = S), E (A = R), y (A = S and E),
// S' (A = U).  The warps share only the chunk's tiles, copied one chunk ahead
// into the other of two buffers; one barrier a chunk is all the
// synchronisation there is.
//
// Units.  A row of the state is S times a power of two, sig, with |S| <= bnd
// <= 2^15: S is an fp16 operand as it stands (hi + lo).  A chunk decays S and
// moves it to the units in which the bound of what comes out, bnd exp(cs_C) +
// 64 max|U| (32 tokens, k below 2), lies in [2^14, 2^15); U is brought to the
// same units and the products are added to S in place.  The bound is some
// 2^10 above the values, which leaves them 2^4 or so, 2^29 above fp16's last
// place; every eighth chunk it starts anew from the true maximum, so that it
// does not run away where nothing decays.  Taking the maximum in every chunk
// was measured too: 130 clocks a chunk and warp of 2970.
//
// Bound by the chain of a warp's chunk, about 1250 instructions that mostly
// wait for one another: alone on its scheduler (128 CTAs: b4 L2048 H32 P64
// N128, without y: 149 us) a warp issues in 29 % of the clocks and holds the
// matrix pipe for 28 %.  Three CTAs an SM fill the gaps of one another: b8
// L2048 H80 P64 N128 takes 530 us; the matrix instructions by themselves (228 a
// warp and chunk, 8 clocks each) would take 265 us there.  A third of them are
// y's.  With one term of S, U and M for y in bf16 (184 instructions, errors of
// 2^-12 before y's own rounding) the walk took 460 us; it is not kept, so that y
// is the rounding of a value held to 32 bits.  Warp-level instructions run at a
// quarter of the rate of tcgen05 (557 TFLOP/s measured), but their results go
// from product to product in registers; on tcgen05 each of the five dependent
// products would pass through TMEM and shared memory.  That form was not built, so how
// it compares is not known.  Measured and not kept: issuing the
// next chunk's copies between the products of this one (471 us), two warps for
// 16 rows, half of the columns each, for calls of few CTAs (their exchange and
// the products that both make cost more than the halves save: 16 chunks of
// fp32 take 45 us against 34, the reverse walk 263 against 220), an explicit
// order of loads before their use, units brought up to date only when they
// run out (both no change), V read element by element where it is unaligned
// (4.1 us a chunk; see k_delta_pad).
#pragma once

#include "ssd_delta_prep.cuh"

namespace ssd {
namespace delta {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kP = 16 * kWarps;  // headdim rows of a CTA, 16 a warp

struct WalkArgs {
  int64_t L, H, G, P, N, hpg;
  int slices;          // CTAs over headdim
  int64_t units;       // (run, head, slice)
  const char* tokens;  // [chunk][group] TokenTiles
  const char* heads;   // [chunk][head] HeadTiles
  const void* v;       // forward: v; reverse: dy; rows of `pv` elements on 16-byte boundaries
  const float* s0;     // state a run starts from (reverse: gradient of the final state), or null
  const Run* runs;     // or null: a run for each row
  void* out;           // forward: y; state walk: E (fp32); reverse: dv
  float* out_f;        // reverse: D (fp32)
  float* check;        // state at every 64th token of a run (state walk, reverse)
  float* max_v;        // largest magnitude of each 16 rows of V in each chunk (reverse), of
  float* max_out;      // E or D there, and of the state at each checkpoint: [.][head][pg],
  float* max_check;    // for the kernel that turns them into operands
  int pg;              // sixteens of headdim
  float* fin;          // final state (forward) or gradient of the initial state (reverse), or null
  int64_t pv;          // row pitch of v
  int64_t pe;          // row pitch of E and D: headdim rounded up to fours
  int out_vec;         // rows of y or dv start on 16-byte boundaries
};

// A chunk's tiles in shared memory, two buffers.
template <typename T, int NT, bool Q, int MTERMS>
struct Buffers {
  using X = TokenTiles<T, NT>;
  using Hd = HeadTiles<MTERMS>;
  static constexpr int kTok = Q ? X::kBytes : X::kBytes / 2;  // k, and q where it is used
  static constexpr int kVP = sizeof(T) == 2 ? kP + 8 : kP + 4;  // row pitch of the V tile
  static constexpr int kHead = kTok, kV = kHead + Hd::kBytes;
  static constexpr int kBuf = kV + kC * kVP * (int)sizeof(T);
  static constexpr int kStage = 2 * kBuf;  // a warp's output tile, fp32 pitch 20
  static constexpr int kBytes = kStage + kWarps * kC * 20 * 4;
  static_assert(kBuf % 16 == 0, "16-byte copies");
};

// Rows of v or dy that do not start on 16-byte boundaries are copied, by a
// kernel before the walk, to rows that do, with zeros behind headdim: reading
// them element by element in the walk, between two chunks, took it from 2.0 to
// 4.1 us a chunk.
template <typename T>
__global__ void __launch_bounds__(256) k_delta_pad(const T* __restrict__ from, T* __restrict__ to, int64_t rows, int64_t P,
                                                   int64_t pitch) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pitch; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pitch, c = i - r * pitch;
    to[i] = c < P ? from[r * P + c] : from_f<T>(0.f);
  }
}
template <typename T>
cudaError_t launch_pad(const void* from, void* to, int64_t rows, int64_t P, int64_t pitch, cudaStream_t stream) {
  const int64_t need = (rows * pitch + 255) / 256;
  k_delta_pad<T><<<(unsigned)(need < 8 * 148 ? need : 8 * 148), 256, 0, stream>>>(static_cast<const T*>(from),
                                                                                   static_cast<T*>(to), rows, P, pitch);
  return cudaGetLastError();
}
// Row pitch of v as the walks read it, and bytes of its padded copy (0: it is read where it lies).
inline int64_t pitch_of(const Shape& s) {
  const int64_t e = s.bf16 ? 8 : 4;
  return (s.P + e - 1) / e * e;
}
inline size_t pad_bytes(const Shape& s, const void* v) {
  const size_t esz = s.bf16 ? 2 : 4;
  return s.P == pitch_of(s) && aligned(v, 16) ? 0 : (size_t)s.b * s.L * s.H * pitch_of(s) * esz;
}

// Enqueue the copies of one chunk: the group's tiles, the head's, and its rows
// of V (n of them exist, `cols` columns; the rest become zeros).
template <typename T, int NT, bool Q, int MTERMS>
__device__ __forceinline__ void fetch_chunk(const char* tok, const char* head, const T* v, int64_t vstride, int n, int cols,
                                            char* buf) {
  using B = Buffers<T, NT, Q, MTERMS>;
  const uint32_t d = sm100::smem_u32(buf);
#pragma unroll
  for (int x = 0; x < B::kTok / (16 * kThreads); ++x) {
    const int o = (x * kThreads + threadIdx.x) * 16;
    cp_async16(d + o, tok + o, true);
  }
  constexpr int kHeadVec = B::Hd::kBytes / 16;
#pragma unroll
  for (int x = 0; x < (kHeadVec + kThreads - 1) / kThreads; ++x) {
    const int i = x * kThreads + threadIdx.x;
    if (i < kHeadVec) cp_async16(d + B::kHead + i * 16, head + i * 16, true);
  }
  constexpr int E = 16 / (int)sizeof(T), PC = kP / E, kStep = kThreads / PC;
  const int row0 = threadIdx.x / PC, c = (threadIdx.x % PC) * E;
#pragma unroll
  for (int x = 0; x < kC / kStep; ++x) {
    const int row = row0 + x * kStep;
    const bool ok = row < n && c < cols;
    const uint32_t o = B::kV + (row * B::kVP + c) * (int)sizeof(T);
    cp_async16(d + o, ok ? v + row * vstride + c : v, ok);
  }
  cp_async_commit();
}

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
      const float2 u = mul2(x[2 * ks + (a >> 1)][2 * (a & 1)], x[2 * ks + (a >> 1)][2 * (a & 1) + 1], s);
      if constexpr (LO) split2(u, hi[ks][a], lo[ks][a]);
      else hi[ks][a] = pack2(u);
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

// The largest magnitude of a thread's tile, and of the warp's.
__device__ __forceinline__ float tile_max(const float (&x)[4][4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[i][e]));
  return m;
}
__device__ __forceinline__ float warp_absmax(float m) { return absmax_bits(__float_as_uint(m)); }

__device__ __forceinline__ void zero(float (&x)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
}

// Row maxima of the state.
template <int NT>
__device__ __forceinline__ float2 state_max(const float (&S)[NT / 8][4]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 8; ++i) {
    m0 = fmaxf(m0, fmaxf(fabsf(S[i][0]), fabsf(S[i][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(S[i][2]), fabsf(S[i][3])));
  }
  return make_float2(quad_max(m0), quad_max(m1));
}
template <int NT>
__device__ __forceinline__ void state_scale(float (&S)[NT / 8][4], float2 f) {
#pragma unroll
  for (int i = 0; i < NT / 8; ++i) {
    const float2 x = mul2(S[i][0], S[i][1], f.x), y = mul2(S[i][2], S[i][3], f.y);
    S[i][0] = x.x, S[i][1] = x.y, S[i][2] = y.x, S[i][3] = y.y;
  }
}

// The units of a thread's two rows of the state.
struct Unit {
  float2 sig, bnd;

  // The power of two that brings a bound to [2^14, 2^15) (zero: 1), and its inverse.
  static __device__ __forceinline__ float of(float b, float& inv) {
    int e = (int)(__float_as_uint(b) >> 23);
    e = e < 15 ? 15 : e > 253 ? 253 : e;
    e = b > 0.f ? e : 141;
    inv = __uint_as_float((uint32_t)(268 - e) << 23);
    return __uint_as_float((uint32_t)(e - 14) << 23);
  }
  // A state as it was loaded: true values.
  template <int NT>
  __device__ __forceinline__ void init(float (&S)[NT / 8][4]) {
    const float2 m = state_max<NT>(S);
    float2 inv;
    sig = make_float2(of(m.x, inv.x), of(m.y, inv.y));
    bnd = make_float2(m.x * inv.x, m.y * inv.y);
    state_scale<NT>(S, inv);
  }
  // Decay the state by `whole` and bring it to units that also hold 32 tokens'
  // addends of at most `add` (times k, below 2).  Returns 1 / sig.
  template <int NT>
  __device__ __forceinline__ float2 step(float (&S)[NT / 8][4], float whole, float2 add, bool look) {
    if (look) bnd = state_max<NT>(S);
    const float2 want = make_float2(sig.x * whole, sig.y * whole);
    const float2 b = make_float2(fmaf(bnd.x, want.x, 64.f * add.x), fmaf(bnd.y, want.y, 64.f * add.y));
    float2 inv;
    sig = make_float2(of(b.x, inv.x), of(b.y, inv.y));
    bnd = make_float2(b.x * inv.x, b.y * inv.y);
    state_scale<NT>(S, make_float2(want.x * inv.x, want.y * inv.y));
    return inv;
  }
};

// x (p x t) times row and column factors: f.x, f.y for the two rows, c for the columns.
__device__ __forceinline__ void scale_tile(float (&x)[4][4], const float* c, float2 f, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = *reinterpret_cast<const float2*>(c + 8 * i + 2 * (lane & 3));
    const float2 a = __fmul2_rn(make_float2(x[i][0], x[i][1]), mul2(v.x, v.y, f.x));
    const float2 b = __fmul2_rn(make_float2(x[i][2], x[i][3]), mul2(v.x, v.y, f.y));
    x[i][0] = a.x, x[i][1] = a.y, x[i][2] = b.x, x[i][3] = b.y;
  }
}
// to = x c f + to
__device__ __forceinline__ void add_scaled(float (&to)[4][4], const float (&x)[4][4], const float* c, float2 f, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = *reinterpret_cast<const float2*>(c + 8 * i + 2 * (lane & 3));
    const float2 a = __ffma2_rn(make_float2(x[i][0], x[i][1]), mul2(v.x, v.y, f.x), make_float2(to[i][0], to[i][1]));
    const float2 b = __ffma2_rn(make_float2(x[i][2], x[i][3]), mul2(v.x, v.y, f.y), make_float2(to[i][2], to[i][3]));
    to[i][0] = a.x, to[i][1] = a.y, to[i][2] = b.x, to[i][3] = b.y;
  }
}
// A tile whose values fit fp16 as they are, as operand tiles.
template <bool LO>
__device__ __forceinline__ void as_operand(const float (&x)[4][4], uint32_t (&hi)[2][4], uint32_t (&lo)[2][4]) {
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float2 u = make_float2(x[2 * ks + (a >> 1)][2 * (a & 1)], x[2 * ks + (a >> 1)][2 * (a & 1) + 1]);
      if constexpr (LO) split2(u, hi[ks][a], lo[ks][a]);
      else hi[ks][a] = pack2(u);
    }
}
// S += Uhi/lo (p x t) times a 32 x NT tile of tokens (k or q; TERMS fp16
// terms).  Four tiles at a time, so that an accumulator is not needed again
// before its last product is done.
template <int NT, int TERMS>
__device__ __forceinline__ void state_add(float (&S)[NT / 8][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4],
                                          uint32_t tile, int lane) {
  constexpr int kTile = kC * NT * 2;
  const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, nc = (lane >> 4) * 8;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int np = 0; np < NT / 16; np += 2) {
      uint32_t B[2][4];
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) ldsm4t(tile + t * kTile + tile_off<NT>(16 * ks + tr, 16 * (np + x) + nc), B[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) mma(S[2 * np + x], hi[ks], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
        if (t == 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x) mma(S[2 * np + x], lo[ks], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
        }
      }
    }
}

// d (p x t) += A (p x NT, hi and lo of one 16-column step) times rows of a
// 32 x NT tile of tokens; LO: with A's lo term.
template <int NT, int TERMS, bool LO>
__device__ __forceinline__ void tokens_mma(float (&d)[4][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint32_t tile,
                                           int ks, int lane) {
  constexpr int kTile = kC * NT * 2;
  const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
  uint32_t B[2][4];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) ldsm4(tile + t * kTile + tile_off<NT>(16 * x + br, 16 * ks + bc), B[x]);
#pragma unroll
    for (int x = 0; x < 4; ++x) mma(d[x], hi, B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    if (LO && t == 0) {
#pragma unroll
      for (int x = 0; x < 4; ++x) mma(d[x], lo, B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    }
  }
}

// acc (p x t) = S (in its units) times the rows of a tile of tokens; Y: and y of another tile.
template <int NT, int TERMS, bool Y>
__device__ __forceinline__ void state_times(const float (&S)[NT / 8][4], float (&acc)[4][4], uint32_t kt, float (&y)[4][4],
                                            uint32_t qt, int lane) {
  zero(acc);
  if constexpr (Y) zero(y);
#pragma unroll
  for (int ks = 0; ks < NT / 16; ++ks) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      split2(make_float2(S[2 * ks + (x >> 1)][2 * (x & 1)], S[2 * ks + (x >> 1)][2 * (x & 1) + 1]), hi[x], lo[x]);
    tokens_mma<NT, TERMS, true>(acc, hi, lo, kt, ks, lane);
    if constexpr (Y) tokens_mma<NT, TERMS, true>(y, hi, lo, qt, ks, lane);
  }
}

// d (p x t) += X (p x s) W^T for a lower triangular 32 x 32 tile W (t x s):
// X's terms times W's terms, lo times lo left out.
template <bool XLO, int WTERMS>
__device__ __forceinline__ void lower_mma(float (&d)[4][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4],
                                          uint32_t tile, int lane) {
  const int br = (lane & 7) + (lane >> 4) * 8, bc = ((lane >> 3) & 1) * 8;
  uint32_t B[3][4];  // (t, s) blocks of 16: (0, 0), (1, 0), (1, 1)
#pragma unroll
  for (int w = 0; w < WTERMS; ++w) {
#pragma unroll
    for (int x = 0; x < 3; ++x)
      ldsm4(tile + w * kSq + tile_off<32>(16 * (x > 0) + br, 16 * (x == 2) + bc), B[x]);
#pragma unroll
    for (int x = 0; x < 6; ++x)
      mma(d[x < 4 ? x : x - 2], hi[x >> 2], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    if (XLO && w == 0) {
#pragma unroll
      for (int x = 0; x < 6; ++x)
        mma(d[x < 4 ? x : x - 2], lo[x >> 2], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    }
  }
}

// d (p x s) += X (p x t) W for a lower triangular 32 x 32 tile W (t x s).
template <bool XLO>
__device__ __forceinline__ void lower_mma_t(float (&d)[4][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4],
                                            uint32_t tile, int lane) {
  const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, nc = (lane >> 4) * 8;
  uint32_t B[3][4];  // (t, s) blocks of 16: (1, 0), (1, 1), (0, 0)
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int x = 0; x < 3; ++x)
      ldsm4t(tile + w * kSq + tile_off<32>(16 * (x < 2) + tr, 16 * (x == 1) + nc), B[x]);
#pragma unroll
    for (int x = 0; x < 6; ++x) mma(d[x & 3], hi[x < 4], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    if (XLO && w == 0) {
#pragma unroll
      for (int x = 0; x < 6; ++x) mma(d[x & 3], lo[x < 4], B[x >> 1][2 * (x & 1)], B[x >> 1][2 * (x & 1) + 1]);
    }
  }
}

template <typename T, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, NT <= 128 ? 3 : 2) k_delta_walk(const WalkArgs a) {
  constexpr bool kY = MODE == kForward;
  constexpr int kMTerms = kY ? 2 : 0;  // M to 22 bits, as every operand that is a result
  using B = Buffers<T, NT, kY, kMTerms>;
  using X = TokenTiles<T, NT>;
  using Hd = HeadTiles<kMTerms>;
  constexpr int kTerms = X::kTerms;
  extern __shared__ __align__(128) char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices;
  const int64_t rh = blockIdx.x / a.slices, h = rh % a.H, ri = rh / a.H;
  const Run run = a.runs ? a.runs[ri] : row_run(ri, a.L);
  const int nc = (run.len + kC - 1) / kC;
  const int p_cta = slice * kP, p0 = p_cta + 16 * warp;
  const int cols = (int)(a.pv - p_cta < kP ? a.pv - p_cta : kP);
  const int rows = a.P - p0 < 16 ? (int)(a.P - p0) : 16;  // may be negative: nothing is read or written
  const int64_t vstride = a.H * a.pv, tstride = a.G * X::kBytes, hstride = a.H * Hd::kStride;
  const char* tok = a.tokens + (run.chunk * a.G + h / a.hpg) * X::kBytes;
  const char* head = a.heads + (run.chunk * a.H + h) * Hd::kStride;
  const T* v = static_cast<const T*>(a.v) + (run.tok * a.H + h) * a.pv + p_cta;
  float S[NT / 8][4];
  if (a.s0 && run.h0 >= 0) {
    load_state<NT>(S, a.s0 + (((int64_t)run.h0 * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
  } else {
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
  }
  Unit unit;
  unit.init<NT>(S);
  char* stage = sm + B::kStage + warp * (kC * 20 * 4);
  sm100::griddep_wait();  // the tiles
  const auto fetch = [&](int j) {
    const int n = run.len - j * kC;
    fetch_chunk<T, NT, kY, kMTerms>(tok + j * tstride, head + j * hstride, v + (int64_t)j * kC * vstride, vstride, n, cols,
                                    sm + (j & 1) * B::kBuf);
  };
  if (nc > 0) fetch(0);
  for (int j = 0; j < nc; ++j) {
    cp_async_wait<0>();
    __syncthreads();  // chunk j is there, and every warp is done with the other buffer
    if (j + 1 < nc) fetch(j + 1);
    if (rows <= 0) continue;  // no such rows: only keep step
    char* const buf = sm + (j & 1) * B::kBuf;
    const Factors& f = *reinterpret_cast<const Factors*>(buf + B::kHead + Hd::kF);
    const uint32_t kt = sm100::smem_u32(buf), qt = kt + kTerms * X::kTile;
    const uint32_t tt = kt + B::kHead, mt = tt + Hd::kM;
    if constexpr (MODE == kStates) {
      if ((j & 1) == 0) {
        const int64_t at = (run.slot + (j >> 1)) * a.H + h;
        store_state<NT>(S, unit.sig.x, unit.sig.y, a.check + (at * a.P + p0) * a.N, a.N, rows, lane);
        const float m = warp_absmax(fmaxf(unit.bnd.x * unit.sig.x, unit.bnd.y * unit.sig.y));
        if (lane == 0) a.max_check[at * a.pg + p0 / 16] = m;
      }
    }
    float acc[4][4], y[4][4], e[4][4];
    state_times<NT, kTerms, kY>(S, acc, kt, y, qt, lane);
    uint32_t hi[2][4], lo[2][4];
    // R = V - exp(cs) K S^T
    load_v<T, B::kVP>(e, buf + B::kV, 16 * warp, lane);
    add_scaled(e, acc, f.kc, make_float2(-unit.sig.x, -unit.sig.y), lane);
    float2 iv = to_operand<true>(e, hi, lo);
    // E = R (I + A)^-T, in units (1 / iv below) in which it is below 2^15 like R
    zero(e);
    lower_mma<true, 2>(e, hi, lo, tt, lane);
    scale_tile(e, f.tau, make_float2(1.f, 1.f), lane);
    iv.x *= f.norm, iv.y *= f.norm;
    const int n = run.len - j * kC < kC ? run.len - j * kC : kC;
    const int64_t th = (run.tok + (int64_t)j * kC) * a.H + h, row0 = th * a.P + p0, rowe = th * a.pe + p0;
    if constexpr (kY) {
      as_operand<true>(e, hi, lo);
      scale_tile(y, f.qc, unit.sig, lane);
      zero(acc);
      lower_mma<true, kMTerms>(acc, hi, lo, mt, lane);
      add_scaled(y, acc, f.mu, iv, lane);
      store_tile<T>(y, stage, static_cast<T*>(a.out) + row0, a.H * a.P, n, rows, a.out_vec, lane);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i][0] = e[i][0] * iv.x, y[i][1] = e[i][1] * iv.x, y[i][2] = e[i][2] * iv.y, y[i][3] = e[i][3] * iv.y;
      // (zeros in the columns from headdim to the pitch)
      store_tile<float>(y, stage, static_cast<float*>(a.out) + rowe, a.H * a.pe, n, (rows + 3) & ~3, true, lane);
      const float m = warp_absmax(32768.f * fmaxf(iv.x, iv.y));
      if (lane == 0) a.max_out[((run.chunk + j) * a.H + h) * a.pg + p0 / 16] = m;
    }
    // S' = exp(cs_C) S + U K
    const float ub = 32768.f * f.ucm;
    const float2 is = unit.step<NT>(S, f.whole, make_float2(iv.x * ub, iv.y * ub), (j & 7) == 7);
    scale_tile(e, f.uc, make_float2(iv.x * is.x, iv.y * is.y), lane);
    as_operand<true>(e, hi, lo);
    state_add<NT, kTerms>(S, hi, lo, kt, lane);
  }
  if (a.fin && run.fin >= 0)
    store_state<NT>(S, unit.sig.x, unit.sig.y, a.fin + (((int64_t)run.fin * a.H + h) * a.P + p0) * a.N, a.N, rows, lane);
}

template <typename T, int NT, int MODE>
cudaError_t launch_walk_nt(const WalkArgs& a, cudaStream_t stream) {
  constexpr int smem = Buffers<T, NT, MODE == kForward, MODE == kForward ? 2 : 0>::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> seen{0};
  return launch_kernel(k_delta_walk<T, NT, MODE>, seen, (unsigned)a.units, kThreads, smem, smem, true, stream, a);
}

template <typename T, int MODE>
cudaError_t launch_walk(const WalkArgs& a, cudaStream_t stream) {
  if (a.N <= 64) return launch_walk_nt<T, 64, MODE>(a, stream);
  if (a.N <= 128) return launch_walk_nt<T, 128, MODE>(a, stream);
  return launch_walk_nt<T, 256, MODE>(a, stream);
}

}  // namespace delta
}  // namespace ssd
