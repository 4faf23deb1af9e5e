// Group norm, backward.
//
//   g = dy act'(u);  dw = sum g xn;  db = sum g;  dx = rstd (g w - mean of g w - xn mean of g w xn)
#include "cc3d_heads_group.h"

namespace {

// The eight elements of a row: xn and g.
template <class T, int TERMS>
__device__ __forceinline__ void slope(const Raw8<T>& x, const Raw8<T>& dy, const float (&mean)[TERMS], const float (&rs)[TERMS],
                                      const float (&w)[8], const float (&b)[8], int act, float (&xn)[8], float (&g)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    xn[j] = (get8(x, j) - mean[TERMS == 1 ? 0 : j]) * rs[TERMS == 1 ? 0 : j];
    g[j] = get8(dy, j);
    if (act == CC3D_ACT_SILU) g[j] *= silu_slope(fmaf(xn[j], w[j], b[j]));
  }
}

template <class T, int KIND>
__device__ __forceinline__ void params(const GroupArgs& a, const Cols<T, KIND>& cols, float (&w)[8], float (&b)[8]) {
  const Raw8<T> rw = cols.param(a.w, 1.f), rb = cols.param(a.b, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = get8(rw, j);
    b[j] = get8(rb, j);
  }
}

// dw and db of a workgroup: its lines' sums in order, into a row of [2][C].
template <class T, int KIND, bool WHOLE>
__device__ __forceinline__ void fold_lines(const GroupArgs& a, const Lane<T, KIND, WHOLE>& l, float* box, const float (&dw)[8],
                                           const float (&db)[8], float* out) {
  const int per = l.lines * a.c;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (l.cols.on(j)) {
      box[l.line * a.c + l.cols.c0 + j] = dw[j];
      box[per + l.line * a.c + l.cols.c0 + j] = db[j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.c; i += blockDim.x) {
    const int k = i >= a.c, c = i - k * a.c;
    float s = 0.f;
    for (int x = 0; x < l.lines; ++x) s += box[k * per + x * a.c + c];
    out[i] = s;
  }
}

// ---- whole samples in registers.  ROWS: of a thread; THREADS: at most (registers spill at 1024, of more than 2048
// channels, and at four rows)
template <class T, int KIND, bool WHOLE, int ROWS, int THREADS>
__global__ __launch_bounds__(THREADS) void group_whole_bwd(GroupArgs a) {
  constexpr int kRows = ROWS, kTerms = Lane<T, KIND, WHOLE>::kTerms;
  extern __shared__ __attribute__((aligned(16))) float box[];
  const Lane<T, KIND, WHOLE> l(a);
  const int samples = l.lines / a.line_n, row0 = l.line % a.line_n;
  float w[8], b[8], dw[8] = {}, db[8] = {};
  params(a, l.cols, w, b);
  for (int64_t n0 = int64_t(blockIdx.x) * samples; n0 < a.n; n0 += int64_t(gridDim.x) * samples) {
    const int64_t n = n0 + l.line / a.line_n;
    const bool in = n < a.n;
    const int len = in ? valid_rows(a, n) : 0;
    const float inv = len > 0 ? 1.f / (float(len) * float(a.cg)) : 0.f;
    Raw8<T> x[kRows], dy[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row0 + r * a.line_n;
      x[r] = row < len ? l.cols.load(a.x, n * a.xb + row * a.xr + l.cols.c0) : zero8<T>();
      dy[r] = row < len ? l.cols.load(a.dy, n * a.dyb + row * a.dyr + l.cols.c0) : zero8<T>();
    }
    float mean[kTerms], rs[kTerms];
    if (a.stats_in) {
      l.groups(a, [&](int j, int g) {
        const float2 s = in ? reinterpret_cast<const float2*>(a.stats_in)[n * a.groups + g] : float2{0.f, 0.f};
        mean[j] = s.x;
        rs[j] = s.y;
      });
    } else {
      float sum[1][kTerms] = {}, sq[1][kTerms] = {};
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0][WHOLE ? 0 : j] += get8(x[r], j);
      sample_sums(a, l, box, sum);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) mean[j] = sum[0][j] * inv;
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (row0 + r * a.line_n < len)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = get8(x[r], j) - mean[WHOLE ? 0 : j];
            sq[0][WHOLE ? 0 : j] = fmaf(d, d, sq[0][WHOLE ? 0 : j]);
          }
      sample_sums(a, l, box, sq);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) rs[j] = len > 0 ? 1.f / sqrtf(fmaf(sq[0][j], inv, a.eps)) : 0.f;
    }
    float m[2][kTerms] = {};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row0 + r * a.line_n >= len) continue;
      float xn[8], g[8];
      slope(x[r], dy[r], mean, rs, w, b, a.act, xn, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[j] = fmaf(g[j], xn[j], dw[j]);
        db[j] += g[j];
        const float gw = g[j] * w[j];
        m[0][WHOLE ? 0 : j] += gw;
        m[1][WHOLE ? 0 : j] = fmaf(gw, xn[j], m[1][WHOLE ? 0 : j]);
      }
    }
    if (!a.dx) continue;  // (the same for all threads)
    sample_sums(a, l, box, m);
    if (!in) continue;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row0 + r * a.line_n;
      if (row >= a.p) continue;
      float xn[8], g[8], o[8];
      slope(x[r], dy[r], mean, rs, w, b, a.act, xn, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        constexpr bool one = WHOLE;
        const float d = fmaf(-xn[j], m[1][one ? 0 : j] * inv, fmaf(g[j], w[j], -m[0][one ? 0 : j] * inv)) * rs[one ? 0 : j];
        o[j] = row < len ? d : 0.f;
      }
      l.cols.store(a.dx, n * a.dxb + row * a.dxr + l.cols.c0, o);
    }
  }
  if (a.want_dw || a.want_db) fold_lines(a, l, box, dw, db, a.part + int64_t(blockIdx.x) * 2 * a.c);
}

// ---- split samples: each run's sums of g xn and g, by channel
template <class T, int KIND, bool WHOLE>
__global__ __launch_bounds__(1024) void group_sums_bwd(GroupArgs a) {
  constexpr int kTerms = Lane<T, KIND, WHOLE>::kTerms, kRows = 2;
  extern __shared__ __attribute__((aligned(16))) float box[];
  const Lane<T, KIND, WHOLE> l(a);
  const int64_t n = blockIdx.x / a.splits;
  const int split = int(blockIdx.x - n * a.splits), len = valid_rows(a, n);
  const int begin = split * a.rows, end = min(begin + a.rows, len);
  float w[8], b[8], dw[8] = {}, db[8] = {}, mean[kTerms], rs[kTerms];
  params(a, l.cols, w, b);
  l.groups(a, [&](int j, int g) {
    const float2 s = reinterpret_cast<const float2*>(a.stats_in)[n * a.groups + g];
    mean[j] = s.x;
    rs[j] = s.y;
  });
  Rows8<T, KIND, kRows> nx, ny;
  auto fetch = [&](int r0) {
    nx.load(l.cols, a.x, n * a.xb, a.xr, r0, l.lines, end);
    ny.load(l.cols, a.dy, n * a.dyb, a.dyr, r0, l.lines, end);
  };
  // (the next rows load ahead; in fp32 the registers are worth more: 19 us so, 17 without)
  constexpr bool kAhead = sizeof(T) == 2;
  if (kAhead) fetch(begin + l.line);
  for (int r0 = begin + l.line; r0 < end; r0 += l.lines * kRows) {
    if (!kAhead) fetch(r0);
    const Rows8<T, KIND, kRows> x = nx, dy = ny;
    if (kAhead) fetch(r0 + l.lines * kRows);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r0 + r * l.lines >= end) break;
      float xn[8], g[8];
      slope(x.v[r], dy.v[r], mean, rs, w, b, a.act, xn, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[j] = fmaf(g[j], xn[j], dw[j]);
        db[j] += g[j];
      }
    }
  }
  fold_lines(a, l, box, dw, db, a.part + int64_t(blockIdx.x) * 2 * a.c);
}

// ---- a sample's runs added, 64 of its 2 C columns a workgroup: each of 16 waves takes every 16th run
__global__ __launch_bounds__(1024) void group_fold(GroupArgs a, int tiles) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x % 64, line = threadIdx.x / 64;
  const int64_t n = blockIdx.x / tiles;
  const int col = int(blockIdx.x - n * tiles) * 64 + lane, wide = 2 * a.c;
  const float* src = a.part + n * a.splits * wide + (col < wide ? col : 0);
  float s = 0.f;
  for (int r0 = line; r0 < a.splits; r0 += 128) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r0 + 16 * i < a.splits ? src[int64_t(r0 + 16 * i) * wide] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  red[line][lane] = s;
  __syncthreads();
  if (line == 0 && col < wide) {
#pragma unroll
    for (int x = 1; x < 16; ++x) s += red[x][lane];
    a.chan[n * wide + col] = s;
  }
}

// ---- split samples: the groups' means from the channels' sums, then dx
template <class T, int KIND, bool WHOLE>
__global__ __launch_bounds__(1024) void group_apply_bwd(GroupArgs a) {
  constexpr int kTerms = Lane<T, KIND, WHOLE>::kTerms, kRows = 2;
  extern __shared__ __attribute__((aligned(16))) float box[];  // [groups][2]
  const Lane<T, KIND, WHOLE> l(a);
  // (from the last run to the first: those are in the last-level cache from the sums)
  const unsigned run = gridDim.x - 1 - blockIdx.x;
  const int64_t n = run / a.splits;
  const int split = int(run - n * a.splits), len = valid_rows(a, n);
  const int begin = split * a.rows, end = min(begin + a.rows, a.p);
  const float inv = len > 0 ? 1.f / (float(len) * float(a.cg)) : 0.f;
  const float* chan = a.chan + n * 2 * a.c;
  const T* weight = static_cast<const T*>(a.w);
  const int team = team_width(a.groups, a.cg), teams = blockDim.x / team;
  for (int g0 = 0; g0 < a.groups; g0 += teams) {
    const int g = g0 + int(threadIdx.x) / team;
    float s = 0.f, q = 0.f;
    if (g < a.groups)
      for (int x = threadIdx.x % team; x < a.cg; x += team) {
        const int c = g * a.cg + x;
        const float f = weight ? to_f32(weight[c]) : 1.f;
        q = fmaf(chan[c], f, q);
        s = fmaf(chan[a.c + c], f, s);
      }
    s = team_sum(s, team);
    q = team_sum(q, team);
    if (g < a.groups && threadIdx.x % team == 0) {
      box[2 * g] = s * inv;
      box[2 * g + 1] = q * inv;
    }
  }
  __syncthreads();
  float w[8], b[8], mean[kTerms], rs[kTerms], m[2][kTerms];
  params(a, l.cols, w, b);
  l.groups(a, [&](int j, int g) {
    const float2 s = reinterpret_cast<const float2*>(a.stats_in)[n * a.groups + g];
    mean[j] = s.x;
    rs[j] = s.y;
    m[0][j] = box[2 * g];
    m[1][j] = box[2 * g + 1];
  });
  for (int r0 = begin + l.line; r0 < end; r0 += l.lines * kRows) {
    Rows8<T, KIND, kRows> x, dy;
    x.load(l.cols, a.x, n * a.xb, a.xr, r0, l.lines, min(end, len));
    dy.load(l.cols, a.dy, n * a.dyb, a.dyr, r0, l.lines, min(end, len));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = r0 + r * l.lines;
      if (row >= end) break;
      float xn[8], g[8], o[8];
      slope(x.v[r], dy.v[r], mean, rs, w, b, a.act, xn, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        constexpr bool one = WHOLE;
        const float d = fmaf(-xn[j], m[1][one ? 0 : j], fmaf(g[j], w[j], -m[0][one ? 0 : j])) * rs[one ? 0 : j];
        o[j] = row < len ? d : 0.f;
      }
      l.cols.store(a.dx, n * a.dxb + row * a.dxr + l.cols.c0, o);
    }
  }
}

template <class T, int KIND, bool WHOLE>
struct RunWhole {
  static int run(const cc3d_group_plan& p, const GroupArgs& a, hipStream_t s) {
    const int threads = cc3d::group_threads(a.c);
    const int lds = std::max(sample_lds(a, WHOLE, 2, threads), 8 * threads / a.lanes * a.c);
    auto go = [&](auto* kernel) { return launch_lds(kernel, p.workers, threads, lds, s, a); };
    if (a.p == 1) return threads == 256 ? go(&group_whole_bwd<T, KIND, WHOLE, 1, 256>) : go(&group_whole_bwd<T, KIND, WHOLE, 1, 1024>);
    return threads == 256 ? go(&group_whole_bwd<T, KIND, WHOLE, cc3d::kGroupRows, 256>)
                          : go(&group_whole_bwd<T, KIND, WHOLE, cc3d::kGroupRows, 1024>);
  }
};
template <class T, int KIND, bool WHOLE>
struct RunSums {
  static int run(const GroupArgs& a, hipStream_t s) {
    const int threads = cc3d::group_threads(a.c);
    return launch_lds(&group_sums_bwd<T, KIND, WHOLE>, a.blocks, threads, 8 * threads / a.lanes * a.c, s, a);
  }
};
template <class T, int KIND, bool WHOLE>
struct RunApply {
  static int run(const GroupArgs& a, hipStream_t s) {
    return launch_lds(&group_apply_bwd<T, KIND, WHOLE>, a.blocks, cc3d::group_threads(a.c), 8 * a.groups, s, a);
  }
};

}  // namespace

namespace cc3d {

int launch_group_backward(const cc3d_group_plan& p, const cc3d_group_args_t& c, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  GroupArgs a = group_args(p, c);
  a.dy = c.dy.p;
  a.dyb = c.dy.batch;
  a.dyr = c.dy.row;
  a.dx = c.dx.p;
  a.dxb = c.dx.batch;
  a.dxr = c.dx.row;
  a.stats_in = c.stats;
  a.want_dw = c.dw != nullptr;
  a.want_db = c.db != nullptr;
  float* w = static_cast<float*>(c.workspace);
  int e;
  if (!p.splits) {
    a.part = w;
    if ((e = pick_group<RunWhole>(p.d, p, a, s))) return e;
    const SumJob jobs[] = {{a.part, c.dw, p.workers, a.c, 2 * a.c}, {a.part + a.c, c.db, p.workers, a.c, 2 * a.c}};
    return launch_sums(jobs, 2, stream);
  }
  if (!a.stats_in) {
    float* stats = w + p.bwd_stats;
    if ((e = launch_group_stats(p, c, w, stats, stream))) return e;
    a.stats_in = stats;
  }
  a.rows = p.bwd_rows;
  a.splits = p.bwd_splits;
  a.blocks = int64_t(a.n) * a.splits;
  a.part = w;
  a.chan = w + a.blocks * 2 * a.c;
  if ((e = pick_group<RunSums>(p.d, a, s))) return e;
  const int tiles = (2 * a.c + 63) / 64;
  if ((e = launch(group_fold, int64_t(a.n) * tiles, 1024, 0, s, a, tiles))) return e;
  const SumJob jobs[] = {{a.chan, c.dw, a.n, a.c, 2 * a.c}, {a.chan + a.c, c.db, a.n, a.c, 2 * a.c}};
  if ((e = launch_sums(jobs, 2, stream))) return e;
  return a.dx ? pick_group<RunApply>(p.d, a, s) : 0;
}

}  // namespace cc3d
