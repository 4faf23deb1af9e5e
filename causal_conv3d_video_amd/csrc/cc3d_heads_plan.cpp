// Host side of the operators on heads and groups (include/cc3d_heads.h): plans,
// argument checks and C entry points of linear_attention, rotary and
// group_norm.  No device calls but the launches.
#include "cc3d_heads_internal.h"
#include "cc3d_seq_check.h"

namespace {

// Whether a product of sizes >= 1 stays within the addresses a view may span.
bool within_span(std::initializer_list<int64_t> sizes) {
  int64_t left = kMaxSpan;
  for (int64_t s : sizes) {
    left /= s;
    if (left == 0) return false;
  }
  return true;
}

// Elements between two tokens of linear attention: places inside 64 tokens are
// 32 bits of bytes.
constexpr int64_t kMaxHeadRow = (int64_t(1) << 24) - 1;

constexpr double kTwoPi = 6.283185307179586476925286766559;
// No position is as far: offsets are 32 bits, tokens of a call up to 2^30.
constexpr double kFarthest = 4294967296.0;

}  // namespace

// --------------------------------------------------------------------------
// linear_attention
// --------------------------------------------------------------------------

namespace {

// Segments of the time axis, whole blocks of 64 tokens, where `units` workgroups
// alone leave compute units idle: as many as make one workgroup of four waves or two
// of two (64 columns of a state and fewer) a compute unit, rounded down.  8192 tokens
// of 16 heads of 128 in 70 to 75 us at 16 segments, 77 at 32 and 109 at 8; of 64 in 41 at
// 32, 43 at 16.  Two segments cost their second walk over the tokens and gain little: 192
// heads of 128, 1024 tokens, 69 us whole and 99 in two, 256 heads of 64 of 2048 tokens
// 75 and 91; 128 of 128, 2048 tokens, 126 and 132, in four 123.  512 tokens of 4 heads
// in 16 us block by block and 25 in two.
void split_time(int32_t t, int64_t units, int cols, int32_t* seg, int32_t* segs) {
  const int64_t blocks = ceildiv(t, cc3d::kLinTokens), want = cols == 64 ? 2 * kUnits : kUnits;
  int64_t pieces = std::min(want / units, blocks);
  if (pieces < 3) pieces = 1;
  const int64_t each = ceildiv(blocks, pieces);
  *seg = int32_t(each * cc3d::kLinTokens);
  *segs = int32_t(ceildiv(blocks, each));
}

// Forward calls that take their tokens one after another, in fp32 throughout, instead of as a
// block.  Both ways, in this order, us:
//   bf16, up to two, where the states' bytes are most of it: 1560 sequences of 6 heads of 64, 84 and 80 for 2
//   tokens; 128 of 16 of 128, 72 and 63; 512 of 4 of 256, 283 and 327.  Up to eight where the states are so
//   few that only latency counts: 64 of 12 of 64, 8.5 and 10.8 for 2 and 9.8 and 11.1 for 8; 16 of 4 of 256,
//   15 and 17 for 8.
//   fp32, whose matrix products are no faster than its vector ones: up to 20 tokens, 161 and 162 for 20 and
//   205 and 174 for 32 of 1560 by 6 heads of 64; 573 and 614, and 727 and 639, of 512 by 16 of 128; 59 and 61, and
//   76 and 64, of 300 by 6 of 50 by 100.  Of wider q and k, whose rows take twice the registers, up to 12:
//   20 and 25 for 12 tokens and 34 and 25 for 32 of 16 by 4 of 256; 506 and 473, and 977 and 486, of 512 by 4.
bool linear_steps(const cc3d_linear_desc_t& d, int64_t workgroups) {
  if (d.dtype != CC3D_BF16) return d.t <= (d.dk <= 128 ? 20 : 12);
  return d.t <= 2 || (d.t <= 8 && workgroups <= 4 * kUnits);
}

}  // namespace

extern "C" cc3d_status_t linear_attention_plan(const cc3d_linear_desc_t* d, cc3d_linear_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  if (!d || d->n < 1 || d->t < 1 || d->heads < 1 || d->q_heads < 1 || d->k_heads < 1 || d->v_heads < 1 || d->dk < 1 ||
      d->dv < 1 || d->heads % d->q_heads || d->heads % d->k_heads || d->heads % d->v_heads || !std::isfinite(d->scale) ||
      !known_dtype(d->dtype))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->t > kMaxTokens || d->dk > 256 || d->dv > 256) return refuse(CC3D_ERR_UNSUPPORTED);
  const int64_t widest = std::max(d->dk, d->dv);
  if (!within_span({d->n, d->t, d->heads, widest}) || !within_span({d->n, d->heads, d->dk, d->dv}))
    return refuse(CC3D_ERR_UNSUPPORTED);
  const int64_t nh = int64_t(d->n) * d->heads;
  const int64_t blocks = cc3d::linear_blocks(d->dv, cc3d::linear_cols(d->dv)), units = nh * blocks;
  const int64_t short_units = nh * cc3d::linear_blocks(d->dv, 64);
  // (heads are rounded up to eight, one for each die)
  if (!cc3d::fits(units + 7 * blocks, cc3d::kLinThreads) || !cc3d::fits(short_units, cc3d::kLinThreads)) return refuse(CC3D_ERR_UNSUPPORTED);
  auto* p = make_plan<cc3d_linear_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->steps = linear_steps(*d, short_units);
  if (!p->steps) split_time(d->t, units, cc3d::linear_cols(d->dv), &p->seg, &p->segs);
  const int cols = cc3d::linear_cols(int(widest));
  // Backward: by dq's recurrence, which is a launch by itself where the decay's gradient is asked for (2 by 2049
  // tokens, 16 heads, 64 by 128: 129 us at 11 segments, 131 at 7, 152 at 17).
  const int64_t of_k = cc3d::linear_blocks(d->dk, cols), of_v = cc3d::linear_blocks(d->dv, cols);
  split_time(d->t, nh * of_k, cc3d::linear_cols(d->dk), &p->bwd_seg, &p->bwd_segs);
  p->bwd_fits = cc3d::fits((nh + 7) * (2 * of_k + of_v), cc3d::kLinThreads);  // (where it is split it is far below)
  p->info.chunks = p->segs;
  p->info.backward_chunks = p->bwd_segs;
  // (states between segments, and a copy of h_in for calls in place)
  p->info.workspace_bytes = p->segs > 1 ? nh * p->segs * d->dk * d->dv * 4 : 0;
  p->info.backward_workspace_bytes = cc3d::linear_bwd_space(*p).total * 4;
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t linear_attention_plan_info(cc3d_linear_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void linear_attention_plan_destroy(cc3d_linear_plan_t p) { delete p; }

namespace {
void linear_inputs(Check& c, const cc3d_linear_desc_t& d, const cc3d_linear_args_t* a) {
  c.view(a->q, d.n, d.t, int64_t(d.q_heads) * d.dk, false, true);
  c.view(a->k, d.n, d.t, int64_t(d.k_heads) * d.dk, false, true);
  c.view(a->v, d.n, d.t, int64_t(d.v_heads) * d.dv, false, true);
  c.dense(a->log_decay, int64_t(d.heads) * 4, 4, false, false);
  c.dense(a->h_in, int64_t(d.n) * d.heads * d.dk * d.dv * 4, 4, false, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
}
}  // namespace

namespace {
bool far_heads(const cc3d_linear_desc_t& d, std::initializer_list<const cc3d_rows_t*> views) {
  for (const cc3d_rows_t* v : views)
    if (d.t > 1 && v->p && v->row > kMaxHeadRow) return true;
  return false;
}
}  // namespace

extern "C" cc3d_status_t linear_attention_forward(cc3d_linear_plan_t p, const cc3d_linear_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  linear_inputs(c, d, a);
  c.view(a->o, d.n, d.t, int64_t(d.heads) * d.dv, true, true);
  c.dense(a->h_out, int64_t(d.n) * d.heads * d.dk * d.dv * 4, 4, true, false);
  c.same_allowed(a->h_in, a->h_out);
  c.workspace(a->workspace, a->workspace_bytes, p->info.workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  if (far_heads(d, {&a->q, &a->k, &a->v, &a->o})) return refuse(CC3D_ERR_UNSUPPORTED);
  return launched(cc3d::launch_linear_forward(*p, *a, stream));
}

extern "C" cc3d_status_t linear_attention_backward(cc3d_linear_plan_t p, const cc3d_linear_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  const int64_t state = int64_t(d.n) * d.heads * d.dk * d.dv * 4;
  Check c(elem_of(d.dtype));
  linear_inputs(c, d, a);
  c.view(a->grad_o, d.n, d.t, int64_t(d.heads) * d.dv, false, true);
  c.view(a->dq, d.n, d.t, int64_t(d.q_heads) * d.dk, true, false);
  c.view(a->dk, d.n, d.t, int64_t(d.k_heads) * d.dk, true, false);
  c.view(a->dv, d.n, d.t, int64_t(d.v_heads) * d.dv, true, false);
  c.dense(a->dh_out, state, 4, false, false);
  c.dense(a->dh_in, state, 4, true, false);
  c.dense(a->dlog_decay, int64_t(d.heads) * 4, 4, true, false);
  c.require(!a->dlog_decay || a->log_decay);
  c.workspace(a->workspace, a->workspace_bytes, p->info.backward_workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  if (!p->bwd_fits || far_heads(d, {&a->q, &a->k, &a->v, &a->grad_o, &a->dq, &a->dk, &a->dv}))
    return refuse(CC3D_ERR_UNSUPPORTED);
  return launched(cc3d::launch_linear_backward(*p, *a, stream));
}

// --------------------------------------------------------------------------
// rotary
// --------------------------------------------------------------------------

extern "C" cc3d_status_t rotary_plan(const cc3d_rotary_desc_t* d, cc3d_rotary_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  auto positive = [](double v) { return std::isfinite(v) && v > 0.0; };
  if (!d || d->n < 1 || d->t < 1 || d->q_heads < 1 || d->k_heads < 0 || d->d < 1 || d->rot < 2 || d->rot % 2 ||
      d->first < 0 || d->first > d->d - d->rot ||
      (d->layout != CC3D_ROTARY_HALF && d->layout != CC3D_ROTARY_INTERLEAVED) || d->scaling < CC3D_ROTARY_UNSCALED ||
      d->scaling > CC3D_ROTARY_PARTS || !known_dtype(d->dtype) || !positive(d->theta) || !std::isfinite(float(d->amplitude)) ||
      (d->scaling != CC3D_ROTARY_UNSCALED && !positive(d->factor)) || (d->scaling == CC3D_ROTARY_BASE && d->rot < 4) ||
      (d->scaling == CC3D_ROTARY_PARTS &&
       !(positive(d->original) && std::isfinite(d->fast) && d->slow >= 0.0 && d->fast > d->slow)))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->t > kMaxTokens || d->d > 1024 || d->rot > 256) return refuse(CC3D_ERR_UNSUPPORTED);
  const int64_t heads = int64_t(d->q_heads) + d->k_heads;
  // (a token's pieces are counted in 32 bits)
  if (heads > (int64_t(1) << 30) / d->d || !within_span({d->n, d->t, heads, d->d})) return refuse(CC3D_ERR_UNSUPPORTED);
  const int64_t all = int64_t(d->n) * d->t, each = heads * ceildiv(d->d, 8);
  // Four pieces of eight channels a thread, and 1024 workgroups where the tokens allow.
  const int64_t tokens =
      std::max<int64_t>(1, std::min<int64_t>({ceildiv(4 * cc3d::kRotaryThreads, each), all / (4 * kUnits), 16}));
  if (!cc3d::fits(ceildiv(all, tokens), cc3d::kRotaryThreads)) return refuse(CC3D_ERR_UNSUPPORTED);
  double each_turns[128];
  double theta = d->theta;
  if (d->scaling == CC3D_ROTARY_BASE) theta *= std::pow(d->factor, double(d->rot) / (d->rot - 2));
  for (int j = 0; j < d->rot / 2; ++j) {
    double f = std::pow(theta, -2.0 * j / d->rot);
    if (d->scaling == CC3D_ROTARY_LINEAR) f /= d->factor;
    if (d->scaling == CC3D_ROTARY_PARTS) {
      const double turns = d->original * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - d->slow) / (d->fast - d->slow)));
      f = f * keep + f / d->factor * (1.0 - keep);
    }
    each_turns[j] = f / kTwoPi;
    if (!std::isfinite(each_turns[j] * kFarthest)) return refuse(CC3D_ERR_INVALID_ARG);
  }
  auto* p = make_plan<cc3d_rotary_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->tokens = int32_t(tokens);
  p->info.chunks = p->info.backward_chunks = 1;
  std::copy(each_turns, each_turns + d->rot / 2, p->turns);
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t rotary_plan_info(cc3d_rotary_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void rotary_plan_destroy(cc3d_rotary_plan_t p) { delete p; }

namespace {
cc3d_status_t rotary_call(cc3d_rotary_plan_t p, const cc3d_rotary_args_t* a, bool backward, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  c.view(a->q, d.n, d.t, int64_t(d.q_heads) * d.d, false, true);
  c.view(a->q_out, d.n, d.t, int64_t(d.q_heads) * d.d, true, true);
  c.require(d.k_heads > 0 || (!a->k.p && !a->k_out.p));
  if (d.k_heads > 0) {
    c.view(a->k, d.n, d.t, int64_t(d.k_heads) * d.d, false, true);
    c.view(a->k_out, d.n, d.t, int64_t(d.k_heads) * d.d, true, true);
  }
  c.same_allowed(a->q.p, a->q_out.p);
  c.same_allowed(a->k.p, a->k_out.p);
  c.dense(a->positions, int64_t(d.n) * d.t * 4, 4, false, false);
  c.dense(a->offsets, int64_t(d.n) * 4, 4, false, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
  c.require(!a->positions || !a->offsets);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_rotary(*p, *a, backward, stream));
}
}  // namespace

extern "C" cc3d_status_t rotary_forward(cc3d_rotary_plan_t p, const cc3d_rotary_args_t* a, void* stream) {
  return rotary_call(p, a, false, stream);
}

extern "C" cc3d_status_t rotary_backward(cc3d_rotary_plan_t p, const cc3d_rotary_args_t* a, void* stream) {
  return rotary_call(p, a, true, stream);
}

// --------------------------------------------------------------------------
// group_norm
// --------------------------------------------------------------------------

extern "C" cc3d_status_t group_norm_plan(const cc3d_group_desc_t* d, cc3d_group_plan_t* out) {
  if (!out) return refuse(CC3D_ERR_INVALID_ARG);
  *out = nullptr;
  if (!d || d->n < 1 || d->p < 1 || d->c < 1 || d->groups < 1 || d->c % d->groups || !known_act(d->act) ||
      !known_dtype(d->dtype) || !(d->eps > 0.f) || !std::isfinite(d->eps))
    return refuse(CC3D_ERR_INVALID_ARG);
  if (d->c > 8192 || d->p > kMaxTokens || !within_span({d->n, d->p, d->c})) return refuse(CC3D_ERR_UNSUPPORTED);
  const int lanes = cc3d::group_lanes(d->c), threads = cc3d::group_threads(d->c), lines = threads / lanes;
  int64_t splits = 0, rows = 0, bwd_splits = 0, bwd_rows = 0, workers = 0;
  if (d->p <= lines * cc3d::kGroupRows) {
    int64_t line_n = 1;
    while (line_n * cc3d::kGroupRows < d->p) line_n *= 2;
    // (every workgroup of the backward call leaves a row of partial sums)
    workers = std::min<int64_t>(ceildiv(d->n, lines / line_n), 8 * kUnits);
  } else {
    // Runs of rows: eight workgroups of 256 threads a compute unit, in the backward call, whose threads hold more,
    // four (17 samples of 1560 positions, 515 fp32 channels, 48 us and 52 with eight; three of 57600, 384 channels of
    // bf16, 150 both; four of 230400, 192 channels, forward, 219 and with four 231), at least two steps of a thread each.
    auto cut = [&](int each, int64_t* runs, int64_t* of) {
      *runs = std::max<int64_t>(1, std::min<int64_t>(ceildiv(each * kUnits * 256 / threads, d->n),
                                                     d->p / (2 * lines * cc3d::kGroupRows)));
      *of = ceildiv(ceildiv(d->p, *runs), lines) * lines;
      *runs = ceildiv(d->p, *of);
    };
    cut(8, &splits, &rows);
    cut(4, &bwd_splits, &bwd_rows);
    const int64_t others = std::max<int64_t>(ceildiv(int64_t(d->n) * d->groups, 4) * 256,
                                             int64_t(d->n) * ceildiv(2 * d->c, 64) * 1024);
    if (!cc3d::fits(int64_t(d->n) * splits, threads) || others > cc3d::kMaxThreads) return refuse(CC3D_ERR_UNSUPPORTED);
  }
  auto* p = make_plan<cc3d_group_plan>(d);
  if (!p) return CC3D_ERR_NO_MEMORY;
  p->splits = int32_t(splits);
  p->rows = int32_t(rows);
  p->bwd_splits = int32_t(bwd_splits);
  p->bwd_rows = int32_t(bwd_rows);
  p->workers = workers;
  p->info.chunks = int32_t(std::max<int64_t>(splits, 1));
  p->info.backward_chunks = int32_t(std::max<int64_t>(bwd_splits, 1));
  const int64_t stats = int64_t(d->n) * d->groups * 2;
  if (splits) {
    p->info.workspace_bytes = (stats * splits + stats) * 4;
    // (the forward runs' moments lie where the sums come to be)
    p->bwd_stats = std::max((bwd_splits + 1) * d->n * 2 * d->c, splits * stats);
    p->info.backward_workspace_bytes = (p->bwd_stats + stats) * 4;
  } else {
    p->info.backward_workspace_bytes = workers * 2 * d->c * 4;
  }
  *out = p;
  return CC3D_OK;
}

extern "C" cc3d_status_t group_norm_plan_info(cc3d_group_plan_t p, cc3d_seq_info_t* info) {
  if (!p || !info) return refuse(CC3D_ERR_INVALID_ARG);
  *info = p->info;
  return CC3D_OK;
}

extern "C" void group_norm_plan_destroy(cc3d_group_plan_t p) { delete p; }

namespace {
void group_inputs(Check& c, const cc3d_group_desc_t& d, const cc3d_group_args_t* a, bool backward) {
  const int64_t e = elem_of(d.dtype);
  c.view(a->x, d.n, d.p, d.c, false, true);
  c.dense(a->w, d.c * e, e, false, false);
  c.dense(a->b, d.c * e, e, false, false);
  c.dense(a->stats, int64_t(d.n) * d.groups * 8, 8, !backward, false);
  c.dense(a->lengths, int64_t(d.n) * 4, 4, false, false);
}
}  // namespace

extern "C" cc3d_status_t group_norm_forward(cc3d_group_plan_t p, const cc3d_group_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  group_inputs(c, d, a, false);
  c.view(a->y, d.n, d.p, d.c, true, true);
  c.workspace(a->workspace, a->workspace_bytes, p->info.workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_group_forward(*p, *a, stream));
}

extern "C" cc3d_status_t group_norm_backward(cc3d_group_plan_t p, const cc3d_group_args_t* a, void* stream) {
  if (!p || !a) return refuse(CC3D_ERR_INVALID_ARG);
  const auto& d = p->d;
  Check c(elem_of(d.dtype));
  group_inputs(c, d, a, true);
  c.view(a->dy, d.n, d.p, d.c, false, true);
  c.view(a->dx, d.n, d.p, d.c, true, false);
  c.dense(a->dw, int64_t(d.c) * 4, 4, true, false);
  c.dense(a->db, int64_t(d.c) * 4, 4, true, false);
  c.require(!a->dw || a->w);
  c.require(!a->db || a->b);
  c.workspace(a->workspace, a->workspace_bytes, p->info.backward_workspace_bytes);
  if (!c.ok()) return refuse(CC3D_ERR_INVALID_ARG);
  return launched(cc3d::launch_group_backward(*p, *a, stream));
}
