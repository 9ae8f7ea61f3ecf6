// Internal declarations shared by the libssd translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ssd.h"

namespace ssd {

// Resolved problem description (validated sizes, typed pointers).
struct Problem {
  int64_t b, L, H, P, N, G, Q, nc;  // nc = ceil(L / Q) chunks per row
  int64_t hpg;                      // heads per group, H / G
  ssd_dtype dtype;
  const void* x;
  const float* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const float* h0;
  const int32_t* seq;
  int64_t num_seqs;
  void* y;
  float* final_states;
  const void* z;  // gate: y * SiLU(z), or null
  bool stall;     // SSD_FLAG_TEST_STALL: the two-head kernel's hand-over waits never succeed
};

constexpr size_t kWsAlign = 256;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Launch a kernel with `smem` bytes of dynamic shared memory, `most` at the most
// over all of its launches.  A kernel's limit is raised to that on the first launch on each device (`seen`: one bit a device, per
// kernel; raising it on every call costs as much as the launch), and once more
// if a launch is refused, as after a device reset.  PDL: the kernel may start
// while the one before it ends, and waits for it itself.  (Up to 40 KB needs no
// limit raised: 48 KB less what a kernel declares itself.)
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kern)(P...), std::atomic<uint64_t>& seen, unsigned grid, unsigned threads, size_t smem,
                          size_t most, bool pdl, cudaStream_t stream, const A&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid), c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at, c.numAttrs = pdl ? 1 : 0;
  for (int attempt = 0;; ++attempt) {
    if (most > 40 * 1024 && (attempt || !(seen.load(std::memory_order_relaxed) & bit))) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != cudaSuccess) return e;
      seen.fetch_or(bit, std::memory_order_relaxed);
    }
    e = cudaLaunchKernelEx(&c, kern, args...);
    if (e != cudaErrorInvalidValue || attempt || most <= 40 * 1024) return e;
    cudaGetLastError();
  }
}

// ---- generic (CUDA-core, fp32) path: ssd_generic.cu ----
size_t generic_workspace_bytes(const Problem& p);
cudaError_t generic_forward(const Problem& p, void* ws, cudaStream_t stream);
int generic_launch_count(const Problem& p);

// ---- fused tensor-core path: ssd_tc.cu ----
bool tc_supported(const Problem& p, uint32_t flags);
size_t tc_workspace_bytes(const Problem& p);
int tc_launch_count(const Problem& p);
// device address of the tensor-core path's error word inside the workspace
const int* tc_error_word(const Problem& p, const void* ws);
// name of the fused kernel the tensor-core path launches for p
const char* tc_main_kernel(const Problem& p);
cudaError_t tc_forward(const Problem& p, void* ws, cudaStream_t stream, cudaEvent_t ev0, cudaEvent_t ev1);

}  // namespace ssd
