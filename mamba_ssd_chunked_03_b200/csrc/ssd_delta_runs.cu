// The run list of packed sequences for the gated delta rule: one CTA finds
// where the id changes, counts and ranks the runs (longest first, so that the
// last CTAs to start are short), and lists the ids that do not occur, whose
// final states the main kernel zeroes.
//
// Bound by latency, a chain of a few global accesses between barriers: the ids
// are read 32 at a time per warp with eight loads in flight, each warp over its
// own contiguous range, and once only up to 65536 of them.  16384 ids
// in 8 runs: 15.5 us.
#include <vector>

#include "ssd_delta.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace delta {
namespace {

constexpr int kThreads = 1024;
constexpr int kRanked = 2048;  // runs up to which they are ranked (quadratic work)

// Whether a run starts at token i (32-bit arithmetic: a 64-bit remainder for
// each id took most of the kernel's time).
__device__ __forceinline__ bool starts(const int32_t* seq, uint32_t i, uint32_t L, bool rows) {
  if (i == 0 || (rows && i % L == 0)) return true;
  return seq[i] != seq[i - 1];
}

__global__ void __launch_bounds__(kThreads) k_delta_runs(const int32_t* __restrict__ seq, int64_t n, int64_t L,
                                                         int64_t cap, int64_t places, int64_t checks,
                                                         const RunList out) {
  Run* const runs = out.runs;
  Chunk* const chunks = out.chunks;
  Slot* const slots = out.slots;
  int32_t* const present = out.present;
  __shared__ int warp_count[32];
  __shared__ int total, absent;
  __shared__ int lens[kRanked], starts_s[kRanked + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool rows = L < n, small = cap <= kRanked;
  int32_t* const first = small ? starts_s : out.first;
  const int64_t per = ((n + 31) / 32 + 31) / 32 * 32;  // ids per warp, a multiple of 32
  const int64_t i0 = warp * per, i1 = i0 + per < n ? i0 + per : n;
  // eight flags of this lane for each 256 ids of the warp; those of the first
  // 2048 are kept for the second pass
  const auto flags = [&](int64_t i) {
    uint32_t f = 0;
    bool s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      s[u] = i + 32 * u + lane < i1 && starts(seq, (uint32_t)(i + 32 * u + lane), (uint32_t)L, rows);
#pragma unroll
    for (int u = 0; u < 8; ++u) f |= (uint32_t)s[u] << u;
    return f;
  };
  uint64_t kept = 0;
  int count = 0;
  for (int64_t i = i0, it = 0; i < i1; i += 256, ++it) {
    const uint32_t f = flags(i);
    if (it < 8) kept |= (uint64_t)f << (8 * it);
    count += __popc(f);
  }
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) warp_count[warp] = count;
  if (threadIdx.x == 0) absent = 0;
  for (int64_t i = threadIdx.x; i < cap; i += kThreads) {
    present[i] = 0;
    Run r = {};
    r.fin = r.h0 = -1;
    runs[i] = r;
  }
  for (int64_t i = threadIdx.x; i < places; i += kThreads) chunks[i] = Chunk{0, 0};
  for (int64_t i = threadIdx.x; i < checks; i += kThreads) slots[i] = Slot{0, 0, 0};
  __syncthreads();
  if (warp == 0) {
    const int c = warp_count[lane];
    int sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    warp_count[lane] = sum - c;
    if (lane == 31) total = sum;
  }
  __syncthreads();
  int64_t at = warp_count[warp];
  for (int64_t i = i0, it = 0; i < i1; i += 256, ++it) {
    const uint32_t f = it < 8 ? (uint32_t)(kept >> (8 * it)) & 255u : flags(i);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool st = (f >> u) & 1;
      const uint32_t m = __ballot_sync(0xffffffffu, st);
      const int64_t k = at + __popc(m & ((1u << lane) - 1u));
      if (st && k <= cap) first[k] = (int32_t)(i + 32 * u + lane);
      at += __popc(m);
    }
  }
  __syncthreads();
  // more runs than num_seqs (ids that come back): the rest is left out
  const int64_t nr = total < cap ? total : cap;
  const auto len_of = [&](int64_t k) { return (int)((k + 1 < total ? first[k + 1] : n) - first[k]); };
  const bool ranked = nr <= kRanked;
  if (ranked) {
    for (int64_t k = threadIdx.x; k < nr; k += kThreads) lens[k] = len_of(k);
    __syncthreads();
  }
  for (int64_t k = threadIdx.x; k < nr; k += kThreads) {
    const int64_t t = first[k];
    const int id = seq[t], len = ranked ? lens[k] : len_of(k);
    int64_t rank = k;
    if (ranked) {
      rank = 0;
      for (int j = 0; j < nr; ++j) rank += lens[j] > len || (lens[j] == len && j < k);
    }
    Run r;
    r.tok = t;
    r.chunk = t / kC + k;  // at least as many places as the runs before it have chunks
    r.slot = t / kCheck + k;
    r.len = len;
    r.fin = id >= 0 && id < cap ? id : -1;
    r.h0 = t % L == 0 ? (int32_t)(t / L) : -1;
    r.pad = 0;
    runs[rank] = r;
    if (r.fin >= 0) present[r.fin] = 1;
  }
  for (int64_t k = warp; k < nr; k += 32) {
    const int t = first[k], len = ranked ? lens[k] : len_of(k);
    for (int i = lane * kC; i < len; i += 32 * kC)
      chunks[t / kC + k + i / kC] = Chunk{t + i, len - i < kC ? len - i : kC};
    for (int i = lane * kCheck; i < len; i += 32 * kCheck)
      slots[t / kCheck + k + i / kCheck] =
          Slot{t + i, len - i < kCheck ? len - i : kCheck, (int)(t / kC + k + i / kC)};
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < cap; i += kThreads) {
    if (present[i]) continue;
    const int64_t k = nr + atomicAdd(&absent, 1);  // any order: each of them writes zeros
    if (k < cap) runs[k].fin = (int32_t)i;
  }
}

}  // namespace

size_t runs_bytes(const Shape& s) {
  if (!s.packed) return 0;
  return align_up((size_t)s.runs * sizeof(Run), kWsAlign) + align_up((size_t)s.chunks * sizeof(Chunk), kWsAlign) +
         align_up((size_t)s.slots * sizeof(Slot), kWsAlign) +
         2 * align_up((size_t)(s.runs + 1) * 4, kWsAlign);
}

RunList runs_at(const Shape& s, void* ws) {
  if (!s.packed) return RunList{};
  char* p = static_cast<char*>(ws);
  RunList r;
  r.runs = reinterpret_cast<Run*>(p);
  p += align_up((size_t)s.runs * sizeof(Run), kWsAlign);
  r.chunks = reinterpret_cast<Chunk*>(p);
  p += align_up((size_t)s.chunks * sizeof(Chunk), kWsAlign);
  r.slots = reinterpret_cast<Slot*>(p);
  p += align_up((size_t)s.slots * sizeof(Slot), kWsAlign);
  r.first = reinterpret_cast<int32_t*>(p);
  p += align_up((size_t)(s.runs + 1) * 4, kWsAlign);
  r.present = reinterpret_cast<int32_t*>(p);
  return r;
}

cudaError_t launch_runs(const Shape& s, const int32_t* seq, const RunList& r, cudaStream_t stream) {
  k_delta_runs<<<1, kThreads, 0, stream>>>(seq, s.b * s.L, s.L, s.runs, s.chunks, s.slots, r);
  return cudaGetLastError();
}

ssd_status check_seq_device(const int32_t* seq, int64_t b, int64_t L, int64_t num_seqs, cudaStream_t stream) {
  try {
    std::vector<int32_t> host((size_t)(b * L));
    if (cudaMemcpyAsync(host.data(), seq, host.size() * sizeof(int32_t), cudaMemcpyDeviceToHost, stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
      return SSD_ERR_CUDA;
    return ssd_check_seq_idx(host.data(), b, L, num_seqs);
  } catch (...) {  // no host memory for the copy
    return SSD_ERR_UNSUPPORTED;
  }
}

ssd_status resolve(const ssd_delta_args* a, Shape* s) {
  if (!a || a->batch <= 0 || a->seqlen <= 0 || a->nheads <= 0 || a->headdim <= 0 || a->dstate <= 0 || a->ngroups <= 0)
    return SSD_ERR_INVALID_ARG;
  if (a->nheads % a->ngroups != 0 || (a->dtype != SSD_F32 && a->dtype != SSD_BF16)) return SSD_ERR_INVALID_ARG;
  if (a->flags & ~SSD_FLAG_CHECK_SEQ) return SSD_ERR_INVALID_ARG;
  if (a->seq_idx && a->num_seqs <= 0) return SSD_ERR_INVALID_ARG;
  const double most = 2147483647.0, b = (double)a->batch, L = (double)a->seqlen, H = (double)a->nheads;
  const double runs = a->seq_idx ? (double)a->num_seqs : b;
  if (a->dstate > 256 || a->headdim > 65536) return SSD_ERR_UNSUPPORTED;
  // grids (heads of chunks, 32-row slices of runs) and token counts below 2^31
  if (b * L >= most || runs >= most || runs * H * (double)((a->headdim + 31) / 32) >= most ||
      (b * (L / kC + 1) + runs) * H >= most)
    return SSD_ERR_UNSUPPORTED;
  s->b = a->batch, s->L = a->seqlen, s->H = a->nheads, s->G = a->ngroups, s->P = a->headdim, s->N = a->dstate;
  s->packed = a->seq_idx != nullptr, s->bf16 = a->dtype == SSD_BF16, s->scale = a->scale;
  s->num_seqs = s->packed ? a->num_seqs : 0;
  s->runs = s->packed ? a->num_seqs : a->batch;
  const int64_t tokens = s->b * s->L;
  s->chunks = s->packed ? tokens / kC + s->runs : s->b * ((s->L + kC - 1) / kC);
  s->slots = s->packed ? tokens / kCheck + s->runs : s->b * ((s->L + kCheck - 1) / kCheck);
  return SSD_OK;
}

}  // namespace delta
}  // namespace ssd
