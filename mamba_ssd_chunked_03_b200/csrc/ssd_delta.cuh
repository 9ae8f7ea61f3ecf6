// Shared pieces of the gated delta rule's kernels (ssd_delta_fwd.cu,
// ssd_delta_bwd.cu): the run list, the warp-level matrix instruction, and the
// operand split that keeps fp32 accuracy on 16-bit matrix instructions.
//
// Operands.  Every matrix operand is held as fp16 after its rows (for the
// gradients: its tile) have been brought into fp16's range by a power of two that
// is folded back into the fp32 result.  A bf16 value is then exact in one term
// (8 bits, down to 2^-17 of the largest, and off by 2^-25 of it below); an
// fp32 one is split in two, hi + lo with 11 bits each, so that a product of an
// exact and a split operand takes two instructions and is off by about 2^-22,
// and one of two split operands takes three (lo * lo is left out: 2^-22
// again).  bf16 terms would need three and six for the same accuracy.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100.cuh"
#include "ssd.h"

namespace ssd {
namespace delta {

constexpr int kC = 32;         // tokens of a chunk
constexpr int kCheck = 64;     // tokens between two state checkpoints of the backward

// One sequence: a row without seq_idx, or one run of equal ids.
struct Run {
  int64_t tok;    // first token, counted over all rows (row * L + t)
  int64_t chunk;  // index of its first chunk among all runs' chunks
  int64_t slot;   // index of its first checkpoint
  int32_t len;    // tokens; 0: an id that does not occur (its final state is zeroed)
  int32_t fin;    // index of its final state, or -1
  int32_t h0;     // row whose initial state it starts from, or -1
  int32_t pad;
};
// A chunk's place: its first token over all rows, and how many of its 32
// tokens exist (0: no such chunk).
struct Chunk {
  int32_t tok, n;
};

// A checkpoint's place: the (up to) 64 tokens it covers, their first chunk.
struct Slot {
  int32_t tok, n, chunk;
};

// ---------------------------------------------------------------- elements
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The power of two that brings a row with largest magnitude m to [2^14, 2^15),
// and its inverse (m = 0, denormal, infinite or NaN: the nearest that exists).
__device__ __forceinline__ float pow2_scale(float m, float& inv) {
  int e = (int)(__float_as_uint(m) >> 23);
  e = e < 15 ? 15 : e > 253 ? 253 : e;
  inv = __uint_as_float((uint32_t)(e - 14) << 23);
  return __uint_as_float((uint32_t)(268 - e) << 23);
}

// The same for rows of q and k, brought to [1, 2): their products with a state
// of up to 2^14 then stay in its units (ssd_delta_walk.cuh).
__device__ __forceinline__ float pow2_unit(float m, float& inv) {
  int e = (int)(__float_as_uint(m) >> 23);
  e = e < 1 ? 1 : e > 253 ? 253 : e;
  inv = __uint_as_float((uint32_t)e << 23);
  return __uint_as_float((uint32_t)(254 - e) << 23);
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ float2 bf16x2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// hi and lo terms of two scaled values
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack2(v);
  lo = pack2(__ffma2_rn(unpack2(hi), make_float2(-1.f, -1.f), v));
}
__device__ __forceinline__ float2 mul2(float a, float b, float s) { return __fmul2_rn(make_float2(a, b), make_float2(s, s)); }

// ---------------------------------------------------------------- matrix instruction
// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).  Thread i of the
// warp holds D at rows i/4 and i/4 + 8, columns 2(i%4) and 2(i%4) + 1; A at
// the same rows and columns (registers 0, 1: columns 0-7; 2, 3: 8-15); B at
// column i/4, rows 2(i%4).. and 2(i%4) + 8...  So a D tile pair is an A tile
// as it stands, and a product can be fed to the next without leaving the
// registers.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) { sm100::ldmatrix_x4_trans(addr, r); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes are zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of (row, column) in a tile of fp16 rows: W columns each, the
// 16-byte pieces of a row permuted by its index so that the eight rows of an
// ldmatrix lie in different banks.
template <int W>
__device__ __forceinline__ uint32_t tile_off(int row, int col) {
  if constexpr (W == 32)
    return (uint32_t)(row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + (col & 7) * 2);
  else
    return (uint32_t)(row * (W * 2) + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

// The largest magnitude over the four threads that share a row of D.
__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// g in powers of two, bounded below where its exponential is zero anyway: a
// decay of -inf (a reset) then leaves the cumulative sums finite.  NaN stays NaN.
__device__ __forceinline__ double decay_log2(float g) {
  return (g < -1.0e4f ? -1.0e4 : (double)g) * 1.4426950408889634074;
}

// 2^c, accurate to fp32 for any c (the fraction is taken in 64 bits).
__device__ __forceinline__ float pow2_of(double c) {
  const double i = rint(c);
  return exp2f((float)(c - i)) * exp2f((float)i);
}

struct Shape {
  int64_t b, L, H, G, P, N, num_seqs;
  int64_t runs;    // units of the run list
  int64_t chunks;  // places of chunks over all runs
  int64_t slots;   // places of checkpoints over all runs
  bool bf16, packed;
  float scale;
};

// A run without a list: row `ri`.
__device__ __forceinline__ Run row_run(int64_t ri, int64_t L) {
  Run r;
  r.tok = ri * L, r.len = (int32_t)L, r.fin = r.h0 = (int32_t)ri, r.pad = 0;
  r.chunk = ri * ((L + kC - 1) / kC), r.slot = ri * ((L + kCheck - 1) / kCheck);
  return r;
}

// The run list's part of the workspace: runs, chunks, and scratch.
struct RunList {
  Run* runs;
  Chunk* chunks;
  Slot* slots;
  int32_t* first;
  int32_t* present;
};
size_t runs_bytes(const Shape& s);
RunList runs_at(const Shape& s, void* ws);
// SSD_FLAG_CHECK_SEQ: the precondition on a host copy of seq (waits for `stream`).
ssd_status check_seq_device(const int32_t* seq, int64_t b, int64_t L, int64_t num_seqs, cudaStream_t stream);
// Enqueue the run list of seq_idx: `s.runs` entries, longest first, ids that
// do not occur as runs of length 0 after them; and the places of the chunks.
cudaError_t launch_runs(const Shape& s, const int32_t* seq, const RunList& r, cudaStream_t stream);

// The sizes and options of a call, checked; SSD_OK, or why not.
ssd_status resolve(const ssd_delta_args* a, Shape* s);

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Whether the inputs start on boundaries of their elements (an access elsewhere faults).
inline bool inputs_aligned(const ssd_delta_args* a) {
  const size_t esz = a->dtype == SSD_BF16 ? 2 : 4;
  return aligned(a->q, esz) && aligned(a->k, esz) && aligned(a->v, esz) && aligned(a->g, 4) && aligned(a->beta, 4) &&
         aligned(a->initial_states, 4) && aligned(a->seq_idx, 4);
}

}  // namespace delta
}  // namespace ssd
