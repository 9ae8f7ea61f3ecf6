// ssd_delta_bwd: the gated delta rule's backward.  The run list (with seq_idx),
// every chunk's tiles for both walks, the forward walk again (for E and the
// states at checkpoints), the reverse walk (dv, D and the states' gradients at
// checkpoints), then all other gradients, 64 tokens at a time.
#include "ssd_delta_grads.cuh"
#include "ssd_delta_rwalk.cuh"
#include "ssd_internal.h"

using namespace ssd;
using namespace ssd::delta;

namespace {

struct Layout {
  size_t runs, tokens, fwd, rev, e, d, s, ds, max_y, max_e, max_d, max_s, max_ds, part, dg, v, dy, total;
  int nslices, splits, heads, pg;
};

int64_t pitch_e(const Shape& s) { return (s.P + 3) / 4 * 4; }

Layout layout(const Shape& s, const ssd_delta_bwd_args* b) {
  Layout l;
  size_t at = runs_bytes(s);
  l.runs = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, kWsAlign);
    return o;
  };
  const size_t tokens = (size_t)s.b * s.L, hpn = (size_t)s.H * s.P * s.N;
  l.pg = (int)((s.P + 15) / 16);
  l.nslices = s.bf16 ? grad_slices<__nv_bfloat16>(s.N) : grad_slices<float>(s.N);
  // a group's heads in one CTA, whose sums need no second pass; spread over
  // several while there are fewer CTAs than SMs
  const int64_t hpg = s.H / s.G, units = s.slots * s.G * l.nslices;
  int64_t splits = (148 + units - 1) / units;
  splits = splits > hpg ? hpg : splits;
  l.heads = (int)((hpg + splits - 1) / splits);
  l.splits = (int)((hpg + l.heads - 1) / l.heads);
  l.tokens = take(token_tiles_bytes(s));
  l.fwd = take((size_t)s.chunks * s.H * HeadTiles<0>::kStride);
  l.rev = take((size_t)s.chunks * s.H * RevTiles::kStride);
  l.e = take(tokens * s.H * pitch_e(s) * 4);
  l.d = take(tokens * s.H * pitch_e(s) * 4);
  l.s = take((size_t)s.slots * hpn * 4);
  l.ds = take((size_t)s.slots * hpn * 4);
  const size_t cm = (size_t)s.chunks * s.H * l.pg * 4, sm = (size_t)s.slots * s.H * l.pg * 4;
  l.max_y = take(cm), l.max_e = take(cm), l.max_d = take(cm), l.max_s = take(sm), l.max_ds = take(sm);
  l.part = take(l.splits > 1 ? (size_t)l.splits * 2 * tokens * s.G * s.N * 4 : 0);
  l.dg = take(l.nslices > 1 ? (size_t)l.nslices * tokens * s.H * 4 : 0);
  l.v = take(pad_bytes(s, b->fwd.v));
  l.dy = take(pad_bytes(s, b->dy));
  l.total = at;
  return l;
}

template <typename T>
cudaError_t run_all(const ssd_delta_bwd_args* b, const Shape& s, const Layout& l, const RunList& runs, cudaStream_t st) {
  const ssd_delta_args* a = &b->fwd;
  char* ws = static_cast<char*>(b->workspace);
  const auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const size_t esz = sizeof(T);
  PrepArgs p = {};
  p.L = s.L, p.H = s.H, p.G = s.G, p.N = s.N, p.hpg = s.H / s.G, p.per_row = (int)((s.L + kC - 1) / kC);
  p.scale = s.scale, p.q = a->q, p.k = a->k, p.g = a->g, p.beta = a->beta, p.chunks = runs.chunks;
  p.tokens = ws + l.tokens, p.fwd = ws + l.fwd, p.rev = ws + l.rev;
  p.vec = s.N * esz % 16 == 0 && aligned(a->q, 16) && aligned(a->k, 16);
  cudaError_t e = cudaSuccess;
  const int64_t rows = s.b * s.L * s.H, pv = pitch_of(s);
  const void* v = a->v;
  const void* dy = b->dy;
  if (pad_bytes(s, v)) {
    v = ws + l.v;
    if ((e = launch_pad<T>(a->v, ws + l.v, rows, s.P, pv, st)) != cudaSuccess) return e;
  }
  if (pad_bytes(s, dy)) {
    dy = ws + l.dy;
    if ((e = launch_pad<T>(b->dy, ws + l.dy, rows, s.P, pv, st)) != cudaSuccess) return e;
  }
  e = launch_prep<T, true, true>(p, s.chunks, st);
  if (e != cudaSuccess) return e;
  WalkArgs w = {};
  w.pv = pv, w.pe = pitch_e(s);
  w.L = s.L, w.H = s.H, w.G = s.G, w.P = s.P, w.N = s.N, w.hpg = p.hpg;
  w.slices = (int)((s.P + kP - 1) / kP), w.units = s.runs * s.H * w.slices;
  w.tokens = p.tokens, w.heads = p.fwd, w.v = v, w.s0 = a->initial_states, w.runs = runs.runs;
  w.pg = l.pg, w.out = at(l.e), w.max_out = at(l.max_e);
  w.check = at(l.s), w.max_check = at(l.max_s);
  if ((e = launch_walk<T, kStates>(w, st)) != cudaSuccess) return e;
  w.heads = p.rev, w.v = dy, w.s0 = b->dfinal_states, w.out = b->dv, w.out_f = at(l.d);
  w.max_v = at(l.max_y), w.max_out = at(l.max_d), w.check = at(l.ds), w.max_check = at(l.max_ds);
  w.fin = b->dinitial_states;
  w.out_vec = s.P * esz % 16 == 0 && aligned(b->dv, 16);
  if ((e = launch_rwalk<T>(w, st)) != cudaSuccess) return e;
  GradArgs g = {};
  g.L = s.L, g.H = s.H, g.G = s.G, g.P = s.P, g.N = s.N, g.hpg = p.hpg;
  g.per_row = (int)((s.L + kCheck - 1) / kCheck), g.splits = l.splits, g.heads = l.heads, g.nslices = l.nslices;
  g.pg = l.pg, g.scale = s.scale, g.tokens = p.tokens, g.head = p.rev, g.dy = dy, g.pv = pv, g.pe = w.pe;
  g.e = at(l.e), g.d = at(l.d), g.s = at(l.s), g.ds = at(l.ds);
  g.max_y = at(l.max_y), g.max_e = at(l.max_e), g.max_d = at(l.max_d), g.max_s = at(l.max_s), g.max_ds = at(l.max_ds);
  g.slots = runs.slots, g.slots_n = s.slots, g.dq = b->dq, g.dk = b->dk;
  g.part = at(l.part), g.part_size = s.b * s.L * s.G * s.N;
  g.dg = l.nslices > 1 ? at(l.dg) : b->dg, g.dg_size = s.b * s.L * s.H, g.dbeta = b->dbeta;
  g.pair = s.N % 2 == 0 && aligned(b->dq, 2 * esz) && aligned(b->dk, 2 * esz);
  return launch_grads<T>(g, b->dg, st);
}

}  // namespace

extern "C" SSD_API size_t ssd_delta_bwd_workspace_size(const ssd_delta_bwd_args* b) {
  Shape s;
  if (!b || resolve(&b->fwd, &s) != SSD_OK) return 0;
  return layout(s, b).total;
}

extern "C" SSD_API ssd_status ssd_delta_bwd(const ssd_delta_bwd_args* b, void* stream) {
  Shape s;
  if (!b) return SSD_ERR_INVALID_ARG;
  const ssd_delta_args* a = &b->fwd;
  const ssd_status c = resolve(a, &s);
  if (c != SSD_OK) return c;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !b->dy || !b->dq || !b->dk || !b->dv || !b->dg || !b->dbeta)
    return SSD_ERR_INVALID_ARG;
  const size_t esz = s.bf16 ? 2 : 4;
  if (!inputs_aligned(a) || !aligned(b->dy, esz) || !aligned(b->dq, esz) || !aligned(b->dk, esz) || !aligned(b->dv, esz) ||
      !aligned(b->dg, 4) || !aligned(b->dbeta, 4) || !aligned(b->dfinal_states, 4) || !aligned(b->dinitial_states, 4))
    return SSD_ERR_INVALID_ARG;
  const Layout l = layout(s, b);
  if ((double)s.slots * s.G * l.nslices * l.splits >= 2147483647.0) return SSD_ERR_UNSUPPORTED;
  if (!b->workspace || b->workspace_bytes < l.total) return SSD_ERR_WORKSPACE;
  if (!aligned(b->workspace, kWsAlign)) return SSD_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.packed && (a->flags & SSD_FLAG_CHECK_SEQ)) {
    const ssd_status v = check_seq_device(a->seq_idx, s.b, s.L, s.num_seqs, st);
    if (v != SSD_OK) return v;
  }
  const RunList runs = runs_at(s, b->workspace);
  if (s.packed && launch_runs(s, a->seq_idx, runs, st) != cudaSuccess) return SSD_ERR_CUDA;
  const cudaError_t e =
      s.bf16 ? run_all<__nv_bfloat16>(b, s, l, runs, st) : run_all<float>(b, s, l, runs, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
