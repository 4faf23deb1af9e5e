// Group norm, forward.
#include "cc3d_heads_group.h"

namespace {

// ---- whole samples in registers: mean, then the squares about it, then the results.
// ROWS: of a thread; THREADS: at most.  The next samples' rows load while some are worked on.
template <class T, int KIND, bool WHOLE, int ROWS, int THREADS>
__global__ __launch_bounds__(THREADS) void group_whole(GroupArgs a) {
  constexpr int kTerms = Lane<T, KIND, WHOLE>::kTerms;
  extern __shared__ __attribute__((aligned(16))) float box[];
  const Lane<T, KIND, WHOLE> l(a);
  const int samples = l.lines / a.line_n, row0 = l.line % a.line_n;
  const Raw8<T> rw = l.cols.param(a.w, 1.f), rb = l.cols.param(a.b, 0.f);
  const int64_t step = int64_t(gridDim.x) * samples;
  Rows8<T, KIND, ROWS> next;
  int64_t n = int64_t(blockIdx.x) * samples + l.line / a.line_n;
  int next_len = n < a.n ? valid_rows(a, n) : 0;
  next.load(l.cols, a.x, n * a.xb, a.xr, row0, a.line_n, next_len);
  // (every thread of the workgroup takes part in the barriers of every turn)
  for (int64_t n0 = int64_t(blockIdx.x) * samples; n0 < a.n; n0 += step, n += step) {
    const Rows8<T, KIND, ROWS> x = next;
    const int len = next_len;
    next_len = n + step < a.n ? valid_rows(a, n + step) : 0;
    next.load(l.cols, a.x, (n + step) * a.xb, a.xr, row0, a.line_n, next_len);
    float sum[1][kTerms] = {};
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0][WHOLE ? 0 : j] += get8(x.v[r], j);
    sample_sums(a, l, box, sum);
    const float inv = len > 0 ? 1.f / (float(len) * float(a.cg)) : 0.f;
    float mean[kTerms], sq[1][kTerms] = {};
#pragma unroll
    for (int j = 0; j < kTerms; ++j) mean[j] = sum[0][j] * inv;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const bool there = row0 + r * a.line_n < len;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = there ? get8(x.v[r], j) - mean[WHOLE ? 0 : j] : 0.f;
        sq[0][WHOLE ? 0 : j] = fmaf(d, d, sq[0][WHOLE ? 0 : j]);
      }
    }
    sample_sums(a, l, box, sq);
    float rs[kTerms];
#pragma unroll
    for (int j = 0; j < kTerms; ++j) rs[j] = len > 0 ? 1.f / sqrtf(fmaf(sq[0][j], inv, a.eps)) : 0.f;
    if (n >= a.n) continue;
    if (a.stats && row0 == 0 && l.cols.any)
      l.groups(a, [&](int j, int g) {
        // the lane of a group's first channel says what it is
        if (WHOLE ? l.cols.c0 == g * a.cg : l.cols.on(j) && l.cols.c0 + j == g * a.cg)
          reinterpret_cast<float2*>(a.stats)[n * a.groups + g] = float2{mean[j], rs[j]};
      });
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int row = row0 + r * a.line_n;
      if (row >= a.p) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = fmaf((get8(x.v[r], j) - mean[WHOLE ? 0 : j]) * rs[WHOLE ? 0 : j], get8(rw, j), get8(rb, j));
        o[j] = row < len ? (a.act == CC3D_ACT_SILU ? u * sigmoid_f32(u) : u) : 0.f;
      }
      l.cols.store(a.y, n * a.yb + row * a.yr + l.cols.c0, o);
    }
  }
}

// ---- split samples: each run's mean and sum of squares about it

// (count, mean, m2) joined with another
struct Moments {
  float mean, m2;
};
__device__ __forceinline__ Moments join(Moments a, float na, Moments b, float nb, float inv) {  // inv = 1 / (na + nb), or 0
  const float d = b.mean - a.mean;
  return {fmaf(d, nb * inv, a.mean), a.m2 + b.m2 + d * d * (na * nb * inv)};
}

template <class T, int KIND, bool WHOLE>
__global__ __launch_bounds__(1024) void group_stats(GroupArgs a) {
  constexpr int kRows = 4, kTerms = Lane<T, KIND, WHOLE>::kTerms, kEach = WHOLE ? 8 : 1;
  extern __shared__ __attribute__((aligned(16))) float box[];
  const Lane<T, KIND, WHOLE> l(a);
  const int64_t n = blockIdx.x / a.splits;
  const int split = int(blockIdx.x - n * a.splits), len = valid_rows(a, n);
  const int begin = split * a.rows, end = min(begin + a.rows, len);
  // A thread's sums are about its first row (WHOLE: its first element), near the mean for the variance's
  // subtraction to lose little; where that row is far off, so is the thread's own sum of squares.
  const float rows = float(begin + l.line < end ? (end - begin - l.line - 1) / l.lines + 1 : 0);
  float pivot[kTerms], sum[kTerms] = {}, sq[kTerms] = {}, count = rows * kEach;
  Rows8<T, KIND, kRows> next;
  next.load(l.cols, a.x, n * a.xb, a.xr, begin + l.line, l.lines, end);
#pragma unroll
  for (int j = 0; j < kTerms; ++j) pivot[j] = get8(next.v[0], j);
  for (int r0 = begin + l.line; r0 < end; r0 += l.lines * kRows) {
    const Rows8<T, KIND, kRows> x = next;
    next.load(l.cols, a.x, n * a.xb, a.xr, r0 + l.lines * kRows, l.lines, end);
    auto add = [&](int r) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = get8(x.v[r], j) - pivot[WHOLE ? 0 : j];
        sum[WHOLE ? 0 : j] += d;
        sq[WHOLE ? 0 : j] = fmaf(d, d, sq[WHOLE ? 0 : j]);
      }
    };
    if (r0 + (kRows - 1) * l.lines < end) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) add(r);
    } else {
#pragma unroll
      for (int r = 0; r < kRows - 1; ++r)
        if (r0 + r * l.lines < end) add(r);
    }
  }
  Moments have[kTerms];
  const float inv = count > 0.f ? 1.f / count : 0.f;
#pragma unroll
  for (int j = 0; j < kTerms; ++j) {
    const float m2 = fmaf(-sum[j] * inv, sum[j], sq[j]);
    have[j] = {fmaf(sum[j], inv, pivot[j]), m2 < 0.f ? 0.f : m2};
  }
  // across the lines: each second half into the first
  const int half_threads = blockDim.x / 2;
  for (int half = l.lines / 2; half > 0; half /= 2) {
    float* mine = box + threadIdx.x;  // [2 terms + 1][half the threads]
    if (l.line >= half && l.line < 2 * half) {
      mine -= half * a.lanes;
#pragma unroll
      for (int j = 0; j < kTerms; ++j) {
        mine[2 * j * half_threads] = have[j].mean;
        mine[(2 * j + 1) * half_threads] = have[j].m2;
      }
      mine[2 * kTerms * half_threads] = count;
    }
    __syncthreads();
    if (l.line < half) {
      const float now = mine[2 * kTerms * half_threads], inv = count + now > 0.f ? 1.f / (count + now) : 0.f;
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
        have[j] = join(have[j], count, {mine[2 * j * half_threads], mine[(2 * j + 1) * half_threads]}, now, inv);
      count += now;
    }
    __syncthreads();
  }
  // across a group's terms, all of the same count
  const int wide = WHOLE ? a.lanes : a.c, unit = WHOLE ? a.cg / 8 : a.cg;
  float *means = box, *m2s = box + wide;
  if (l.line == 0) {
#pragma unroll
    for (int j = 0; j < kTerms; ++j) {
      if (!(WHOLE ? l.cols.any : l.cols.on(j))) continue;
      const int at = WHOLE ? l.lane : l.cols.c0 + j;
      means[at] = have[j].mean;
      m2s[at] = have[j].m2;
    }
  }
  __syncthreads();
  const float each = float(max(end - begin, 0)) * kEach;
  const int team = team_width(a.groups, unit), teams = blockDim.x / team;
  for (int g0 = 0; g0 < a.groups; g0 += teams) {
    const int g = g0 + int(threadIdx.x) / team, first = threadIdx.x % team;
    const bool in = g < a.groups;
    float s = 0.f, q = 0.f;
    if (in)
      for (int x = first; x < unit; x += team) s += means[g * unit + x];
    const float mean = team_sum(s, team) / float(unit);
    if (in)
      for (int x = first; x < unit; x += team) {
        const float d = means[g * unit + x] - mean;
        q += fmaf(each * d, d, m2s[g * unit + x]);
      }
    q = team_sum(q, team);
    if (in && first == 0)
      reinterpret_cast<float2*>(a.part)[(n * a.splits + split) * a.groups + g] = float2{mean, q};
  }
}

// ---- runs joined: a wave a group.  Its lanes join every 64th run in turn, then each other.
__global__ __launch_bounds__(256) void group_join(GroupArgs a) {
  const int64_t item = int64_t(blockIdx.x) * 4 + threadIdx.x / 64, all = int64_t(a.n) * a.groups;
  const int lane = threadIdx.x % 64;
  if (item >= all) return;
  const int64_t n = item / a.groups;
  const int g = int(item - n * a.groups), len = valid_rows(a, n);
  const float2* part = reinterpret_cast<const float2*>(a.part) + n * a.splits * a.groups + g;
  Moments have = {0.f, 0.f};
  float count = 0.f;
  for (int s0 = lane; s0 < a.splits; s0 += 512) {
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[int64_t(min(s0 + 64 * i, a.splits - 1)) * a.groups];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + 64 * i;
      const float now = s < a.splits ? float(min(max(len - s * a.rows, 0), a.rows)) * float(a.cg) : 0.f;
      const float inv = count + now > 0.f ? 1.f / (count + now) : 0.f;
      if (now > 0.f) have = join(have, count, {v[i].x, v[i].y}, now, inv);
      count += now;
    }
  }
  for (int d = 32; d > 0; d /= 2) {
    const Moments other = {__shfl_down(have.mean, d), __shfl_down(have.m2, d)};
    const float now = __shfl_down(count, d);
    if (now > 0.f) have = join(have, count, other, now, 1.f / (count + now));
    count += now;
  }
  if (lane == 0)
    reinterpret_cast<float2*>(a.stats)[item] =
        count > 0.f ? float2{have.mean, 1.f / sqrtf(have.m2 / count + a.eps)} : float2{0.f, 0.f};
}

// ---- split samples: the results
template <class T, int KIND, bool WHOLE>
__global__ __launch_bounds__(1024) void group_apply(GroupArgs a) {
  constexpr int kTerms = Lane<T, KIND, WHOLE>::kTerms, kRows = 4;
  const Lane<T, KIND, WHOLE> l(a);
  // (from the last run to the first: those are in the last-level cache from the sums)
  const unsigned run = gridDim.x - 1 - blockIdx.x;
  const int64_t n = run / a.splits;
  const int split = int(run - n * a.splits), len = valid_rows(a, n);
  const int begin = split * a.rows, end = min(begin + a.rows, a.p);
  float mean[kTerms], f[8], b[8];
  const Raw8<T> rw = l.cols.param(a.w, 1.f), rb = l.cols.param(a.b, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = get8(rw, j);
    b[j] = get8(rb, j);
  }
  l.groups(a, [&](int j, int g) {
    const float2 s = reinterpret_cast<const float2*>(a.stats)[n * a.groups + g];
    mean[j] = s.x;
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s.y;
    } else {
      f[j] *= s.y;
    }
  });
  Rows8<T, KIND, kRows> next;
  next.load(l.cols, a.x, n * a.xb, a.xr, begin + l.line, l.lines, min(end, len));
  for (int r0 = begin + l.line; r0 < end; r0 += l.lines * kRows) {
    const Rows8<T, KIND, kRows> x = next;
    next.load(l.cols, a.x, n * a.xb, a.xr, r0 + l.lines * kRows, l.lines, min(end, len));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = r0 + r * l.lines;
      if (row >= end) break;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = fmaf(get8(x.v[r], j) - mean[WHOLE ? 0 : j], f[j], b[j]);
        o[j] = row < len ? (a.act == CC3D_ACT_SILU ? u * sigmoid_f32(u) : u) : 0.f;
      }
      l.cols.store(a.y, n * a.yb + row * a.yr + l.cols.c0, o);
    }
  }
}

template <class T, int KIND, bool WHOLE>
struct RunWhole {
  static int run(const cc3d_group_plan& p, const GroupArgs& a, hipStream_t s) {
    const int threads = cc3d::group_threads(a.c);
    auto go = [&](auto* kernel) { return launch_lds(kernel, p.workers, threads, sample_lds(a, WHOLE, 1, threads), s, a); };
    if (a.p == 1) return threads == 256 ? go(&group_whole<T, KIND, WHOLE, 1, 256>) : go(&group_whole<T, KIND, WHOLE, 1, 1024>);
    return threads == 256 ? go(&group_whole<T, KIND, WHOLE, cc3d::kGroupRows, 256>)
                          : go(&group_whole<T, KIND, WHOLE, cc3d::kGroupRows, 1024>);
  }
};

template <class T, int KIND, bool WHOLE>
struct RunStats {
  static int run(const GroupArgs& a, hipStream_t s) {
    const int threads = cc3d::group_threads(a.c), terms = WHOLE ? 1 : 8;
    const int lines = threads > a.lanes ? (2 * terms + 1) * threads / 2 * 4 : 0, groups = 8 * (WHOLE ? a.lanes : a.c);
    return launch_lds(&group_stats<T, KIND, WHOLE>, a.blocks, threads, std::max(lines, groups), s, a);
  }
};

template <class T, int KIND, bool WHOLE>
struct RunApply {
  static int run(const GroupArgs& a, hipStream_t s) {
    return launch(group_apply<T, KIND, WHOLE>, a.blocks, cc3d::group_threads(a.c), 0, s, a);
  }
};

}  // namespace

namespace cc3d {

int launch_group_stats(const cc3d_group_plan& p, const cc3d_group_args_t& c, float* part, float* stats, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  GroupArgs a = group_args(p, c);
  a.part = part;
  a.stats = stats;
  const int e = pick_group<RunStats>(p.d, a, s);
  if (e) return e;
  return launch(group_join, (int64_t(a.n) * a.groups + 3) / 4, 256, 0, s, a);
}

int launch_group_forward(const cc3d_group_plan& p, const cc3d_group_args_t& c, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  GroupArgs a = group_args(p, c);
  a.y = c.y.p;
  a.yb = c.y.batch;
  a.yr = c.y.row;
  a.stats = c.stats;
  if (!p.splits) return pick_group<RunWhole>(p.d, p, a, s);
  float* part = static_cast<float*>(c.workspace);
  if (!a.stats) a.stats = part + a.blocks * a.groups * 2;
  const int e = launch_group_stats(p, c, part, a.stats, stream);
  return e ? e : pick_group<RunApply>(p.d, a, s);
}

}  // namespace cc3d
