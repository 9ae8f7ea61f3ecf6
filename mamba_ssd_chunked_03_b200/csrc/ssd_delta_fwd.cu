// ssd_delta_fwd: the gated delta rule over whole sequences.
#include "ssd_delta_walk.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace delta {
namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

ssd_status resolve(const ssd_delta_args* a, Shape* s) {
  if (!a || a->batch <= 0 || a->seqlen <= 0 || a->nheads <= 0 || a->headdim <= 0 || a->dstate <= 0 || a->ngroups <= 0)
    return SSD_ERR_INVALID_ARG;
  if (a->nheads % a->ngroups != 0 || (a->dtype != SSD_F32 && a->dtype != SSD_BF16)) return SSD_ERR_INVALID_ARG;
  if (a->flags & ~SSD_FLAG_CHECK_SEQ) return SSD_ERR_INVALID_ARG;
  if (a->seq_idx && a->num_seqs <= 0) return SSD_ERR_INVALID_ARG;
  const double most = 2147483647.0, b = (double)a->batch, runs = a->seq_idx ? (double)a->num_seqs : b;
  if (a->dstate > 256 || a->headdim > 65536) return SSD_ERR_UNSUPPORTED;
  if (b * (double)a->seqlen >= most || runs >= most ||
      runs * (double)a->nheads * (double)((a->headdim + kP - 1) / kP) >= most)
    return SSD_ERR_UNSUPPORTED;
  // the largest tensors stay addressable in 64 bits with room to spare
  if (b * (double)a->seqlen * (double)a->nheads * (double)(a->headdim + a->dstate) >= 9.0e17) return SSD_ERR_UNSUPPORTED;
  *s = Shape{a->batch, a->seqlen, a->nheads, a->ngroups, a->headdim, a->dstate, a->seq_idx ? a->num_seqs : 0,
             a->seq_idx ? a->num_seqs : a->batch, 0, a->dtype == SSD_BF16, a->seq_idx != nullptr};
  return SSD_OK;
}

}  // namespace
}  // namespace delta
}  // namespace ssd

using namespace ssd;
using namespace ssd::delta;

extern "C" SSD_API size_t ssd_delta_fwd_workspace_size(const ssd_delta_args* a) {
  Shape s;
  return resolve(a, &s) == SSD_OK ? runs_bytes(s) : 0;
}

extern "C" SSD_API ssd_status ssd_delta_fwd(const ssd_delta_args* a, void* stream) {
  Shape s;
  const ssd_status st = resolve(a, &s);
  if (st != SSD_OK) return st;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->y) return SSD_ERR_INVALID_ARG;
  const size_t need = runs_bytes(s);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  if (need && !aligned(a->workspace, kWsAlign)) return SSD_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.packed && (a->flags & SSD_FLAG_CHECK_SEQ)) {
    const ssd_status c = check_seq_device(a->seq_idx, s.b, s.L, s.num_seqs, cs);
    if (c != SSD_OK) return c;
  }
  WalkArgs w = {};
  w.L = s.L, w.H = s.H, w.G = s.G, w.P = s.P, w.N = s.N, w.hpg = s.H / s.G;
  w.slices = (int)((s.P + kP - 1) / kP);
  w.n_units = (int)(s.runs * s.H * w.slices);
  w.scale = a->scale;
  w.q = a->q, w.k = a->k, w.v = a->v, w.g = a->g, w.beta = a->beta;
  w.s0 = a->initial_states;
  w.runs = s.packed ? static_cast<const Run*>(a->workspace) : nullptr;
  w.out = a->y;
  w.fin = a->final_states;
  const size_t esz = s.bf16 ? 2 : 4;
  w.qk_vec = s.N * esz % 16 == 0 && aligned(a->q, 16) && aligned(a->k, 16);
  w.v_vec = s.P * esz % 16 == 0 && aligned(a->v, 16);
  w.out_vec = s.P * esz % 16 == 0 && aligned(a->y, 16);
  if (s.packed && launch_runs(s, a->seq_idx, a->workspace, cs) != cudaSuccess) return SSD_ERR_CUDA;
  const cudaError_t e =
      s.bf16 ? launch_walk_any<__nv_bfloat16, kForward>(w, cs) : launch_walk_any<float, kForward>(w, cs);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
