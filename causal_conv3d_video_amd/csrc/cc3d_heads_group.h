// Group norm, channels last: shared by its forward and backward kernel files.
//
//   mean, rstd of each group of channels of a sample over all its positions
//   y = act((x - mean) rstd w + b)
//   g = dy act'(u);  dx = rstd (g w - mean of g w - xn mean of g w xn)
//
// Some 7 operations an element forward and 14 backward beside the activation's:
// bound by memory.  A thread takes eight neighbouring channels of a row (as the
// block join does, Cols), `lanes` threads side by side cover a row and a
// workgroup's `lines` take rows below each other.  Two forms:
//   whole  a sample's rows fit the registers of its lines, four a thread: each
//          element is read once (8192 tokens of 2048 channels, bf16, 67 MB, in 17 us);
//   split  larger samples are cut into runs of rows, a workgroup each: one launch
//          for the runs' sums, one that joins them, one that reads everything again
//          and writes the result.  The second reading meets a part of the sample in
//          the last-level cache (four frames of 230400 positions, 192 channels, 354
//          MB read in 90 us, read and written again in 127).
// A group's borders need not be a lane's: sums go by channel into LDS and are
// added there by a team of threads a group.  Where groups are whole lanes (a
// multiple of eight channels) a lane's eight are one term, and where they are
// moreover a power of two of lanes the sum is taken across lanes without LDS.
#pragma once
#include "cc3d_heads_internal.h"
#include "cc3d_seq_join.h"

namespace {

struct GroupArgs {
  const void *x, *dy, *w, *b;
  void *y, *dx;
  int64_t xb, xr, yb, yr, dyb, dyr, dxb, dxr;
  const float* stats_in;
  float* stats;        // [N][G][2]
  float* part;         // split: [N][splits][G][2] or [N][splits][2][C]; whole, backward: [workgroups][2][C]
  float* chan;         // split, backward: [N][2][C]
  const int* lengths;
  int64_t blocks;      // of rows over all samples (split)
  int n, p, c, groups, cg;  // cg: channels of a group
  int lanes, act, rows, splits;
  int line_n;          // whole: lines of a sample, a power of two
  int want_dw, want_db;
  float eps;
};

// A lane's channels and its groups.  WHOLE: all eight are of one group.
template <class T, int KIND, bool WHOLE>
struct Lane {
  static constexpr int kTerms = WHOLE ? 1 : 8;
  Cols<T, KIND> cols;
  int line, lane, lines;
  __device__ __forceinline__ Lane(const GroupArgs& a)
      : cols(int(threadIdx.x % a.lanes) * 8, a.c), line(threadIdx.x / a.lanes), lane(threadIdx.x % a.lanes),
        lines(blockDim.x / a.lanes) {}
  // f(j, group of channel j)
  template <class F>
  __device__ __forceinline__ void groups(const GroupArgs& a, F&& f) const {
    if constexpr (WHOLE) {
      f(0, cols.c0 / a.cg);
    } else {
      int g = cols.c0 / a.cg, in = cols.c0 - g * a.cg;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f(j, min(g, a.groups - 1));
        if (++in == a.cg) {
          in = 0;
          ++g;
        }
      }
    }
  }
};

// v of another lane of each 16.
template <int CTRL>
__device__ __forceinline__ float other_lane(float v) {
  return __uint_as_float(unsigned(__builtin_amdgcn_mov_dpp(int(__float_as_uint(v)), CTRL, 0xf, 0xf, true)));
}

// Sum over aligned teams of `width` lanes, a power of two up to 64, in all of them.  (Within 16 lanes by the vector
// unit's own paths: 8192 rows of 16 groups of 128 in 17.1 us, by way of LDS 19.5.)
__device__ __forceinline__ float team_sum(float v, int width) {
  if (width > 1) v += other_lane<0xb1>(v);   // the neighbour
  if (width > 2) v += other_lane<0x4e>(v);   // two on
  if (width > 4) v += other_lane<0x141>(v);  // the other end of eight
  if (width > 8) v += other_lane<0x140>(v);  // of sixteen
  if (width > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (width > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Threads that add one group's terms: a power of two up to a wave, as many as
// there are for `items` sums of `terms`.
__device__ __forceinline__ int team_width(int items, int terms) {
  int w = 1;
  while (w < 64 && w * 2 <= terms && 2 * w * items <= int(blockDim.x)) w *= 2;
  return w;
}

__device__ __forceinline__ int valid_rows(const GroupArgs& a, int64_t n) {
  return a.lengths ? min(max(a.lengths[n], 0), a.p) : a.p;
}

// A thread's rows of a sample, or of a run of rows: row0, row0 + step, ... below end.
template <class T, int KIND, int ROWS>
struct Rows8 {
  Raw8<T> v[ROWS];
  __device__ __forceinline__ void load(const Cols<T, KIND>& cols, const void* p, int64_t at, int64_t stride, int row0, int step,
                                       int end) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int row = row0 + r * step;
      v[r] = row < end ? cols.load(p, at + row * stride + cols.c0) : zero8<T>();
    }
  }
};

// The sums of groups over the lines of each sample of a workgroup: V sums at
// once, a term a lane (WHOLE) or a channel.  LDS: box [V][lines][terms of a row],
// then sum [V][samples of the workgroup][groups].
template <class T, int KIND, bool WHOLE, int V>
__device__ __forceinline__ void sample_sums(const GroupArgs& a, const Lane<T, KIND, WHOLE>& l, float* box,
                                            float (&v)[V][Lane<T, KIND, WHOLE>::kTerms]) {
  constexpr int kTerms = Lane<T, KIND, WHOLE>::kTerms;
  const int wide = WHOLE ? a.lanes : a.c, unit = WHOLE ? a.cg / 8 : a.cg;
  if constexpr (WHOLE) {
    if (a.line_n == 1 && unit <= 64 && (unit & (unit - 1)) == 0) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[k][0] = team_sum(v[k][0], unit);
      return;
    }
  }
  const int samples = l.lines / a.line_n, items = samples * a.groups;
  float* sum = box + V * l.lines * wide;
  __syncthreads();  // (the sums of the call before have been read)
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int j = 0; j < kTerms; ++j) {
      if constexpr (WHOLE) box[(k * l.lines + l.line) * wide + l.lane] = l.cols.any ? v[k][0] : 0.f;
      else if (l.cols.on(j)) box[(k * l.lines + l.line) * wide + l.cols.c0 + j] = v[k][j];
    }
  __syncthreads();
  const int team = team_width(items, a.line_n * unit), teams = blockDim.x / team;
  for (int i0 = 0; i0 < items; i0 += teams) {  // (all threads: the lanes of a team meet)
    const int i = i0 + int(threadIdx.x) / team;
    const int sample = i / a.groups, g = i - sample * a.groups;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float s = 0.f;
      if (i < items)
        for (int x = threadIdx.x % team; x < a.line_n * unit; x += team) {
          const int row = x / unit;
          s += box[(k * l.lines + sample * a.line_n + row) * wide + g * unit + x - row * unit];
        }
      s = team_sum(s, team);
      if (i < items && threadIdx.x % team == 0) sum[k * items + i] = s;
    }
  }
  __syncthreads();
  const int sample = l.line / a.line_n;
  l.groups(a, [&](int j, int g) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k][j] = sum[k * items + sample * a.groups + g];
  });
}

// bytes of sample_sums' LDS
inline int sample_lds(const GroupArgs& a, bool whole, int v, int threads) {
  const int lines = threads / a.lanes;
  return 4 * v * (lines * (whole ? a.lanes : a.c) + lines / a.line_n * a.groups);
}

// Calls run<T, KIND, WHOLE> for a plan's channels.
template <template <class, int, bool> class Run, class... A>
int pick_group(const cc3d_group_desc_t& d, A&&... args) {
  const int cg = d.c / d.groups;
  auto go = [&](auto t) {
    using T = decltype(t);
    if (d.c < 8) return Run<T, kFew, false>::run(args...);
    if (d.c % 8) return Run<T, kTail, false>::run(args...);
    return cg % 8 == 0 ? Run<T, kEven, true>::run(args...) : Run<T, kEven, false>::run(args...);
  };
  return d.dtype == CC3D_BF16 ? go(bf16_s()) : go(float());
}

// A launch whose LDS may be over 64 KB.
template <class K>
int launch_lds(K kernel, int64_t workgroups, int threads, int lds, hipStream_t s, const GroupArgs& a) {
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return int(e);
    }
  }
  return launch(kernel, workgroups, threads, lds, s, a);
}

inline GroupArgs group_args(const cc3d_group_plan& p, const cc3d_group_args_t& c) {
  GroupArgs a{};
  a.x = c.x.p;
  a.xb = c.x.batch;
  a.xr = c.x.row;
  a.w = c.w;
  a.b = c.b;
  a.lengths = c.lengths;
  a.n = p.d.n;
  a.p = p.d.p;
  a.c = p.d.c;
  a.groups = p.d.groups;
  a.cg = p.d.c / p.d.groups;
  a.lanes = cc3d::group_lanes(p.d.c);
  a.act = p.d.act;
  a.rows = p.rows;
  a.splits = p.splits;
  a.blocks = int64_t(p.d.n) * p.splits;
  a.line_n = 1;
  while (a.line_n * cc3d::kGroupRows < p.d.p && a.line_n < cc3d::group_threads(p.d.c) / a.lanes) a.line_n *= 2;
  a.eps = p.d.eps;
  return a;
}

}  // namespace

namespace cc3d {
// Split samples: mean and rstd of every group into a.stats, by way of a.part (cc3d_heads_group.hip).
int launch_group_stats(const cc3d_group_plan& p, const cc3d_group_args_t& c, float* part, float* stats, void* stream);
}  // namespace cc3d
