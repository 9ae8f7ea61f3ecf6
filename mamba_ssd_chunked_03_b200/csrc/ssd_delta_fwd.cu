// ssd_delta_fwd: the gated delta rule over whole sequences.  The run list (with
// seq_idx), every chunk's tiles, then the walk.
#include "ssd_delta_walk.cuh"
#include "ssd_internal.h"

using namespace ssd;
using namespace ssd::delta;

namespace {

size_t head_tiles_bytes(const Shape& s) {
  return (size_t)s.chunks * s.H * HeadTiles<2>::kStride;
}

}  // namespace

extern "C" SSD_API size_t ssd_delta_fwd_workspace_size(const ssd_delta_args* a) {
  Shape s;
  if (resolve(a, &s) != SSD_OK) return 0;
  return runs_bytes(s) + align_up(token_tiles_bytes(s), kWsAlign) + align_up(head_tiles_bytes(s), kWsAlign) +
         align_up(pad_bytes(s, a->v), kWsAlign);
}

extern "C" SSD_API ssd_status ssd_delta_fwd(const ssd_delta_args* a, void* stream) {
  Shape s;
  const ssd_status st = resolve(a, &s);
  if (st != SSD_OK) return st;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->y) return SSD_ERR_INVALID_ARG;
  if (!inputs_aligned(a) || !aligned(a->y, s.bf16 ? 2 : 4) || !aligned(a->final_states, 4)) return SSD_ERR_INVALID_ARG;
  const size_t need = ssd_delta_fwd_workspace_size(a);
  if (!a->workspace || a->workspace_bytes < need) return SSD_ERR_WORKSPACE;
  if (!aligned(a->workspace, kWsAlign)) return SSD_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.packed && (a->flags & SSD_FLAG_CHECK_SEQ)) {
    const ssd_status c = check_seq_device(a->seq_idx, s.b, s.L, s.num_seqs, cs);
    if (c != SSD_OK) return c;
  }
  const RunList runs = runs_at(s, a->workspace);
  if (s.packed && launch_runs(s, a->seq_idx, runs, cs) != cudaSuccess) return SSD_ERR_CUDA;
  char* ws = static_cast<char*>(a->workspace) + runs_bytes(s);
  const size_t esz = s.bf16 ? 2 : 4;
  const void* v = a->v;
  cudaError_t e = cudaSuccess;
  if (pad_bytes(s, v)) {
    char* to = ws + align_up(token_tiles_bytes(s), kWsAlign) + align_up(head_tiles_bytes(s), kWsAlign);
    const int64_t rows = s.b * s.L * s.H;
    e = s.bf16 ? launch_pad<__nv_bfloat16>(v, to, rows, s.P, pitch_of(s), cs)
               : launch_pad<float>(v, to, rows, s.P, pitch_of(s), cs);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
    v = to;
  }
  PrepArgs p = {};
  p.L = s.L, p.H = s.H, p.G = s.G, p.N = s.N, p.hpg = s.H / s.G;
  p.per_row = (int)((s.L + kC - 1) / kC);
  p.scale = s.scale;
  p.q = a->q, p.k = a->k, p.g = a->g, p.beta = a->beta, p.chunks = runs.chunks;
  p.tokens = ws, p.fwd = ws + align_up(token_tiles_bytes(s), kWsAlign);
  p.vec = s.N * esz % 16 == 0 && aligned(a->q, 16) && aligned(a->k, 16);
  e = s.bf16 ? launch_prep<__nv_bfloat16, true, false>(p, s.chunks, cs)
             : launch_prep<float, true, false>(p, s.chunks, cs);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  WalkArgs w = {};
  w.L = s.L, w.H = s.H, w.G = s.G, w.P = s.P, w.N = s.N, w.hpg = p.hpg;
  w.slices = (int)((s.P + kP - 1) / kP);
  w.units = s.runs * s.H * w.slices;
  w.tokens = p.tokens, w.heads = p.fwd, w.v = v, w.pv = pitch_of(s), w.s0 = a->initial_states, w.runs = runs.runs;
  w.out = a->y, w.fin = a->final_states;
  w.out_vec = s.P * esz % 16 == 0 && aligned(a->y, 16);
  e = s.bf16 ? launch_walk<__nv_bfloat16, kForward>(w, cs) : launch_walk<float, kForward>(w, cs);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
