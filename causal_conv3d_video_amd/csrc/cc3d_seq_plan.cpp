// Host side of the sequence operators (include/cc3d_seq.h): plans, argument
// checks and C entry points of causal_conv1d, selective_scan and norm_join.
// No device calls but the launches.
#include "cc3d_seq_check.h"

namespace {

using cc3d::kScanLanes;

// Elements between two tokens of the scan: offsets inside a chunk of 64
// tokens are 32 bits.
constexpr int64_t kMaxRow = (int64_t(1) << 25) - 1;
// Channels of the scan: the last lane of a channel tile, up to 512 wide, counts
// in 32 bits too.
constexpr int32_t kMaxScanChannels = INT32_MAX - 511;

}  // namespace

// --------------------------------------------------------------------------
// causal_conv1d
// --------------------------------------------------------------------------

extern "C" cc3d_status_t causal_conv1d_plan(const cc3d_conv1d_desc_t* d, cc3d_conv1d_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  if (!d || d->n < 1 || d->t < 1 || d->c < 1 || d->k < 1 || !known_act(d->act) || !known_dtype(d->dtype))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->k > 8 || d->t > kMaxTokens) return refuse(CC3D_ERR_UNSUPPORTED);
  // Tokens per thread: long runs read less of the window twice, short ones
  // fill the card; 2^18 threads are four waves on every SIMD.
  const int64_t vecs = ceildiv(d->c, 8);
  int64_t seg = std::max<int64_t>(ceildiv(int64_t(d->n) * d->t, ceildiv(int64_t(1) << 18, vecs)), 1);
  seg = std::min<int64_t>(std::max<int64_t>(seg, 8), 64);
  seg = std::min<int64_t>(seg, d->t);
  if (int64_t(d->n) * ceildiv(d->t, seg) > (cc3d::kMaxThreads - 255) / vecs) return refuse(CC3D_ERR_UNSUPPORTED);
  auto* p = make_plan<cc3d_conv1d_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->seg = int32_t(seg);
  // Backward: two waves a SIMD (what registers allow at three to five taps; one
  // from six on, five in fp32, which makes it two turns), so 512 workgroups are
  // one turn of the card: runs are as long as that turn needs, up to 64
  // tokens, and a workgroup whose tiles are done takes further runs.  (964
  // workgroups of 17 tokens took 66 us where 500 of 33 take 54.)
  const int64_t lines = 256 / cc3d::conv1d_lanes(d->c), tiles = ceildiv(vecs, cc3d::conv1d_lanes(d->c));
  const int64_t rows = std::max<int64_t>(1, 2 * kUnits / tiles), slots = rows * lines;
  const int64_t turns = ceildiv(int64_t(d->n) * d->t, slots * 64);
  const int64_t runs = std::max<int64_t>(1, slots * turns / d->n);
  p->bwd_seg = int32_t(std::min<int64_t>(std::max<int64_t>(ceildiv(d->t, runs), 8), std::min(d->t, 64)));
  // partial sums of dw and db: one row for each workgroup along the tokens
  p->bwd_rows = std::min<int64_t>(ceildiv(int64_t(d->n) * ceildiv(d->t, p->bwd_seg), lines), rows);
  p->info.backward_workspace_bytes = p->bwd_rows * (d->k + 1) * int64_t(d->c) * 4;
  p->info.chunks = int32_t(ceildiv(d->t, p->seg));
  p->info.backward_chunks = int32_t(ceildiv(d->t, p->bwd_seg));
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t causal_conv1d_plan_info(cc3d_conv1d_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void causal_conv1d_plan_destroy(cc3d_conv1d_plan_t p) { delete p; }

extern "C" cc3d_status_t causal_conv1d_forward(cc3d_conv1d_plan_t p, const cc3d_conv1d_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  const int64_t e = elem_of(d.dtype), cache = int64_t(d.n) * (d.k - 1) * d.c * e;
  Check c(e);
  c.view(a->x, d.n, d.t, d.c, false, true);
  c.view(a->y, d.n, d.t, d.c, true, true);
  c.dense(a->w, int64_t(d.k) * d.c * e, e, false, true);
  c.dense(a->b, int64_t(d.c) * e, e, false, false);
  c.dense(a->cache_in, cache, e, false, false);
  c.dense(a->cache_out, cache, e, true, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_conv1d_forward(*p, *a, stream));
}

extern "C" cc3d_status_t causal_conv1d_backward(cc3d_conv1d_plan_t p, const cc3d_conv1d_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  const int64_t e = elem_of(d.dtype), cache = int64_t(d.n) * (d.k - 1) * d.c * e;
  Check c(e);
  c.view(a->x, d.n, d.t, d.c, false, true);
  c.view(a->dy, d.n, d.t, d.c, false, true);
  c.view(a->dx, d.n, d.t, d.c, true, false);
  c.dense(a->w, int64_t(d.k) * d.c * e, e, false, true);
  c.dense(a->b, int64_t(d.c) * e, e, false, false);
  c.dense(a->cache_in, cache, e, false, false);
  c.dense(a->dcache_out, cache, e, false, false);
  c.dense(a->dcache_in, cache, e, true, false);
  c.dense(a->dw, int64_t(d.k) * d.c * 4, 4, true, false);
  c.dense(a->db, int64_t(d.c) * 4, 4, true, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
  c.workspace(a->workspace, a->workspace_bytes, p->info.backward_workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  if (!sums_fit({{a->dw, int64_t(d.k) * d.c}, {a->db, d.c}})) return refuse(CC3D_ERR_UNSUPPORTED);
  return launched(cc3d::launch_conv1d_backward(*p, *a, stream));
}

// --------------------------------------------------------------------------
// selective_scan
// --------------------------------------------------------------------------

extern "C" cc3d_status_t selective_scan_plan(const cc3d_scan_desc_t* d, cc3d_scan_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  if (!d || d->n < 1 || d->t < 1 || d->d < 1 || d->states < 1 || d->groups < 1 || d->d % d->groups ||
      (d->softplus != 0 && d->softplus != 1) || !known_dtype(d->dtype))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->states > cc3d::kScanMaxStates || d->t > kMaxTokens || d->d > kMaxScanChannels) return refuse(CC3D_ERR_UNSUPPORTED);
  // (an output of more elements than a view may span would be refused by every call)
  if (int64_t(d->n) * d->t > kMaxSpan / d->d) return refuse(CC3D_ERR_UNSUPPORTED);
  const int64_t tiles = int64_t(d->groups) * cc3d::scan_tiles_per_group(*d), nc = int64_t(d->n);
  const int threads = 64 * cc3d::scan_fwd_waves(*d);
  if (d->t == 1 ? !cc3d::fits(nc * ceildiv(int64_t(d->d) * cc3d::scan_step_lanes(d->states), 256), 256)
                : !cc3d::fits(nc * tiles, threads))
    return refuse(CC3D_ERR_UNSUPPORTED);
  // Forward: split the time axis when the channels alone leave SIMDs idle, into
  // four waves a SIMD: 8192 tokens of 2048 channels in 125 us, two a SIMD 142 (a
  // join 1 us slower among them).  From one wave a SIMD on the second walk over the
  // tokens costs more than what it fills: 64 sequences of 1024 such tokens (two
  // waves a SIMD) 590 us whole and 881 split; right at the border, 32 of 2048, still
  // 919 whole and 868 split.
  const int64_t base = nc * tiles * cc3d::scan_fwd_waves(*d);
  int64_t chunk = ceildiv(d->t, 4) * 4;
  if (base < kSimds && d->t > 64) {
    const int64_t pieces = std::min<int64_t>(ceildiv(4 * kSimds, base), ceildiv(d->t, 32));
    chunk = ceildiv(ceildiv(d->t, pieces), 4) * 4;
  }
  const int64_t chunks = ceildiv(d->t, chunk);
  const cc3d::ScanBwdShape bw = cc3d::scan_bwd_shape(*d);
  const int64_t bwd_chunks = ceildiv(d->t, bw.chunk);
  const int64_t bwd_tiles = int64_t(d->groups) * bw.tiles_per_group;
  auto* p = make_plan<cc3d_scan_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->chunk = int32_t(chunk);
  p->info.chunks = int32_t(chunks);
  p->info.backward_chunks = int32_t(bwd_chunks);
  // carries [n][chunk][S][C] and the chunks' sums of delta [n][chunk][C]
  const int64_t state = int64_t(d->states) * d->d;
  if (chunks > 1) p->info.workspace_bytes = nc * chunks * (state + d->d) * 4;
  // backward: two waves a SIMD, each workgroup taking every bwd_workers-th chunk
  // (with 9 to 16 states; the LDS of other counts' workgroups of four waves lets a
  // compute unit hold one, and half of the workers are a second turn)
  p->bwd_workers = int32_t(std::min<int64_t>(nc * bwd_chunks, ceildiv(2 * kSimds, bwd_tiles * bw.waves * bw.wc)));
  // (groups * states stays below 2^30 with it: what follows them counts in 32 bits)
  p->bwd_fits = cc3d::fits(bwd_tiles * p->bwd_workers, 64 * bw.waves * bw.wc) &&
                (bwd_chunks == 1 || cc3d::fits(nc * tiles * bwd_chunks, threads));
  // partial sums: dA [worker][C][S], dD and ddt_bias [worker * waves][C], dB and dC [tile][n][t][waves][2][4 sg]
  int64_t ws = 0;
  if (bwd_chunks > 1) ws += nc * bwd_chunks * (2 * state + d->d);
  ws += int64_t(p->bwd_workers) * (state + 2 * bw.waves * int64_t(d->d));
  ws += bwd_tiles * nc * d->t * bw.waves * 8 * bw.sg;
  p->info.backward_workspace_bytes = ws * 4;
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t selective_scan_plan_info(cc3d_scan_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void selective_scan_plan_destroy(cc3d_scan_plan_t p) { delete p; }

namespace {
void scan_inputs(Check& c, const cc3d_scan_desc_t& d, const cc3d_scan_args_t* a) {
  const int64_t gs = int64_t(d.groups) * d.states;
  c.view(a->u, d.n, d.t, d.d, false, true);
  c.view(a->dt, d.n, d.t, d.d, false, true);
  c.view(a->b, d.n, d.t, gs, false, true);
  c.view(a->c, d.n, d.t, gs, false, true);
  c.view(a->z, d.n, d.t, d.d, false, false);
  c.dense(a->a, int64_t(d.d) * d.states * 4, 4, false, true);
  c.dense(a->d, int64_t(d.d) * 4, 4, false, false);
  c.dense(a->dt_bias, int64_t(d.d) * 4, 4, false, false);
  c.dense(a->h_in, int64_t(d.n) * d.d * d.states * 4, 4, false, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
}

bool far_rows(const cc3d_scan_desc_t& d, std::initializer_list<const cc3d_rows_t*> views) {
  for (const cc3d_rows_t* v : views)
    if (d.t > 1 && v->p && v->row > kMaxRow) return true;
  return false;
}
}  // namespace

extern "C" cc3d_status_t selective_scan_forward(cc3d_scan_plan_t p, const cc3d_scan_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  scan_inputs(c, d, a);
  c.view(a->y, d.n, d.t, d.d, true, true);
  c.dense(a->h_out, int64_t(d.n) * d.d * d.states * 4, 4, true, false);
  c.same_allowed(a->h_in, a->h_out);
  c.workspace(a->workspace, a->workspace_bytes, p->info.workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  if (far_rows(d, {&a->u, &a->dt, &a->b, &a->c, &a->z, &a->y})) return refuse(CC3D_ERR_UNSUPPORTED);
  return launched(cc3d::launch_scan_forward(*p, *a, stream));
}

extern "C" cc3d_status_t selective_scan_backward(cc3d_scan_plan_t p, const cc3d_scan_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  const int64_t gs = int64_t(d.groups) * d.states, state = int64_t(d.n) * d.d * d.states * 4;
  Check c(elem_of(d.dtype));
  scan_inputs(c, d, a);
  c.view(a->dy, d.n, d.t, d.d, false, true);
  c.dense(a->dh_out, state, 4, false, false);
  c.view(a->du, d.n, d.t, d.d, true, false);
  c.view(a->ddt, d.n, d.t, d.d, true, false);
  c.view(a->dz, d.n, d.t, d.d, true, false);
  c.view(a->db, d.n, d.t, gs, true, false);
  c.view(a->dc, d.n, d.t, gs, true, false);
  c.dense(a->dh_in, state, 4, true, false);
  c.dense(a->da, int64_t(d.d) * d.states * 4, 4, true, false);
  c.dense(a->dd, int64_t(d.d) * 4, 4, true, false);
  c.dense(a->ddt_bias, int64_t(d.d) * 4, 4, true, false);
  c.require(!a->dz.p || a->z.p);
  c.require(!a->dd || a->d);
  c.require(!a->ddt_bias || a->dt_bias);
  c.workspace(a->workspace, a->workspace_bytes, p->info.backward_workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  if (!p->bwd_fits || far_rows(d, {&a->u, &a->dt, &a->b, &a->c, &a->z, &a->dy, &a->du, &a->ddt, &a->dz}) ||
      !sums_fit({{a->da, int64_t(d.d) * d.states}, {a->dd, d.d}, {a->ddt_bias, d.d}}))
    return refuse(CC3D_ERR_UNSUPPORTED);
  return launched(cc3d::launch_scan_backward(*p, *a, stream));
}

// --------------------------------------------------------------------------
// norm_join
// --------------------------------------------------------------------------

extern "C" cc3d_status_t norm_join_plan(const cc3d_join_desc_t* d, cc3d_join_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  if (!d || d->rows < 1 || d->gate_rows < 1 || d->c < 1 || !known_norm(d->post) || !known_norm(d->pre) ||
      !known_act(d->act) || !known_act(d->gate_act) || !known_dtype(d->dtype) || !(d->eps > 0.f) ||
      !std::isfinite(d->eps) || (d->pre == CC3D_NORM_NONE && d->act != CC3D_ACT_NONE))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->c > 8192 || d->rows > (int64_t(1) << 36)) return refuse(CC3D_ERR_UNSUPPORTED);
  auto* p = make_plan<cc3d_join_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->d.gate_rows = std::min(d->gate_rows, d->rows);
  d = &p->d;
  p->info.chunks = p->info.backward_chunks = 1;
  // Backward: at most two waves a SIMD, each workgroup with a row of partial sums
  // of the five parameter gradients.  Where a gate row serves several rows a
  // workgroup takes whole gate rows, or, where there are few of them, a part of one,
  // whose partial sums of the gate's gradient follow.  Whole rows from half of the
  // workgroups on: 100 rows of 768 bf16 channels a gate row in 87 us either way at
  // 256 gate rows, 112 at 300, 162 at 500; 192 fp32 channels at 260 in 38.5 us, and
  // 40.7 where only twice as many gate rows are taken whole.
  const int lanes = cc3d::join_lanes(d->c), threads = cc3d::join_threads(lanes);
  const int64_t at_once = threads / lanes;
  const int64_t limit = 2 * kSimds * 64 / threads;
  const int64_t gates = ceildiv(d->rows, d->gate_rows);
  if (d->gate_rows == 1) {
    p->bwd_parts = std::min(limit, ceildiv(d->rows, at_once));
  } else if (gates >= limit / 2) {
    p->bwd_parts = std::min(limit, gates);
  } else {
    // (rounded down: one workgroup over the limit would be a second turn of the card)
    const int64_t each = std::min(limit / gates, ceildiv(d->gate_rows, at_once));
    p->gate_parts = each;
    p->bwd_parts = gates * each;
  }
  p->info.backward_workspace_bytes = p->bwd_parts * (p->gate_parts ? 6 : 5) * int64_t(d->c) * 4;
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t norm_join_plan_info(cc3d_join_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void norm_join_plan_destroy(cc3d_join_plan_t p) { delete p; }

namespace {
void join_inputs(Check& c, const cc3d_join_desc_t& d, const cc3d_join_args_t* a) {
  const int64_t e = elem_of(d.dtype), w = int64_t(d.c) * e;
  c.require(a->y.p || a->residual.p);
  c.require(a->y.p || (!a->gate.p && !a->scale && !a->post_w && !a->post_b && d.post == CC3D_NORM_NONE));
  c.require(d.post != CC3D_NORM_NONE || (!a->post_w && !a->post_b));
  c.require(d.pre != CC3D_NORM_NONE || (!a->pre_w && !a->pre_b));
  c.view(a->y, 1, d.rows, d.c, false, false);
  c.view(a->residual, 1, d.rows, d.c, false, false);
  c.view(a->gate, 1, ceildiv(d.rows, d.gate_rows), d.c, false, false);
  for (const void* q : {a->scale, a->post_w, a->post_b, a->pre_w, a->pre_b}) c.dense(q, w, e, false, false);
}
}  // namespace

extern "C" cc3d_status_t norm_join_forward(cc3d_join_plan_t p, const cc3d_join_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  join_inputs(c, d, a);
  c.require((d.pre != CC3D_NORM_NONE) == (a->h_out.p != nullptr));
  c.require(a->x_out.p || a->h_out.p);
  c.view(a->x_out, 1, d.rows, d.c, true, false);
  c.view(a->h_out, 1, d.rows, d.c, true, false);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_join_forward(*p, *a, stream));
}

extern "C" cc3d_status_t norm_join_backward(cc3d_join_plan_t p, const cc3d_join_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  join_inputs(c, d, a);
  c.require(a->dx_out.p || a->dh.p);
  c.require(d.pre != CC3D_NORM_NONE || !a->dh.p);
  c.view(a->dx_out, 1, d.rows, d.c, false, false);
  c.view(a->dh, 1, d.rows, d.c, false, false);
  c.view(a->dy, 1, d.rows, d.c, true, false);
  c.view(a->dresidual, 1, d.rows, d.c, true, false);
  c.view(a->dgate, 1, ceildiv(d.rows, d.gate_rows), d.c, true, false);
  c.require(!a->dy.p || a->y.p);
  c.require(!a->dresidual.p || a->residual.p);
  c.require(!a->dgate.p || a->gate.p);
  const void* params[5] = {a->scale, a->post_w, a->post_b, a->pre_w, a->pre_b};
  float* grads[5] = {a->dscale, a->dpost_w, a->dpost_b, a->dpre_w, a->dpre_b};
  for (int i = 0; i < 5; ++i) {
    c.require(!grads[i] || params[i]);
    c.dense(grads[i], int64_t(d.c) * 4, 4, true, false);
  }
  c.workspace(a->workspace, a->workspace_bytes, p->info.backward_workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_join_backward(*p, *a, stream));
}
