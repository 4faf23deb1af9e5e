// Shared by the block join's forward and backward kernel files: the norm after
// a block, its gate, the residual scale and sum, and the norm and activation
// before the next block.
//
//   n1 = norm(y) * post_w + post_b;  x = residual + scale * ga(gate) * n1
//   h = act(norm(x) * pre_w + pre_b)
//
// About 16 operations an element against at least two elements read and two
// written: bound by memory.  A row lives in the registers of LPR lanes (eight
// consecutive channels each, a power of two of lanes, so four rows of 96
// channels share a wave and a row of 8192 takes a workgroup): everything is
// read once, both norms' sums are taken over registers (the mean first where
// there is one, then the squares about it), and both results are written from
// the same pass.  The next row's inputs load while a row is worked on.
#pragma once
#include "cc3d_seq_device.h"

#include <algorithm>

namespace {

struct JoinArgs {
  const void *y, *res, *gate, *dxo, *dh;
  void *xo, *ho, *dy, *dres, *dgate;
  int64_t yr, rr, gr, xr, hr, dxr, dhr, dyr, drr, dgr;  // row strides
  const void *scale, *w1, *b1, *w2, *b2;
  float* part;  // backward: [workgroup][5 or 6][C]
  int64_t rows, gate_rows, gates;
  int64_t gate_parts;  // workgroups per gate row, 0: whole gate rows per workgroup
  int c, post, pre, act, gate_act;
  int shared_gate;  // gate_rows > 1 and a gate is there
  float eps, inv_c;
};

// The eight channels of a lane.  KIND says how rows divide into eights:
//   kEven  C is a multiple of eight;
//   kTail  it is not: the last lane takes the row's last eight, of which the
//          first `skip` are the lane's before it too.  Both compute (and store)
//          the same values there, and only the sums over the row leave them out;
//   kFew   C is less than eight: the first lane's, element by element.
// Lanes past the row hold its last eight, and count nowhere.
enum { kEven, kTail, kFew };

template <class T, int KIND>
struct Cols {
  int c0, skip, c;
  bool any;  // this lane has channels of its own
  __device__ __forceinline__ Cols(int first, int channels)
      : c0(KIND == kFew ? 0 : min(first, channels - 8)), skip(first - c0), c(channels), any(first < channels) {}
  __device__ __forceinline__ bool on(int j) const {
    return KIND == kEven ? any : KIND == kTail ? j >= skip : any && j < c;
  }
  __device__ __forceinline__ Raw8<T> load(const void* p, int64_t off) const {
    const T* q = static_cast<const T*>(p) + off;
    if constexpr (KIND == kFew) return load_some(q, c);
    else return load8(q);
  }
  // a parameter's elements, or `none` in the place of each
  __device__ __forceinline__ Raw8<T> param(const void* p, float none) const {
    if (p) return load(p, c0);
    Raw8<T> r = zero8<T>();
#pragma unroll
    for (int j = 0; j < 8; ++j) set8(r, j, from_f32<T>(none));
    return r;
  }
  __device__ __forceinline__ void store(void* p, int64_t off, const float* v) const {
    if (!any) return;
    T* q = static_cast<T*>(p) + off;
    if constexpr (KIND == kFew) store_some(q, c, v);
    else store8(q, v);
  }
};

// Sums over a row's LPR lanes.  Rows wider than a wave pass through LDS, in
// two slots used in turn, so one barrier a sum is enough.
template <int LPR>
struct RowSum {
  static constexpr int kThreads = cc3d::join_threads(LPR);
  float (*box)[2][kThreads / 64];
  int turn = 0;
  __device__ __forceinline__ void two(float& a, float& b) {
    if constexpr (LPR <= 64) {
      a = group_sum<LPR>(a);
      b = group_sum<LPR>(b);
    } else {
      a = group_sum<64>(a);
      b = group_sum<64>(b);
      const int wave = threadIdx.x / 64, first = threadIdx.x / LPR * (LPR / 64);
      if (threadIdx.x % 64 == 0) {
        box[turn][0][wave] = a;
        box[turn][1][wave] = b;
      }
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < LPR / 64; ++i) {
        a += box[turn][0][first + i];
        b += box[turn][1][first + i];
      }
      turn ^= 1;
    }
  }
  __device__ __forceinline__ float one(float a) {
    float b = 0.f;
    two(a, b);
    return a;
  }
};

// The norm of a row: v becomes the normalised row; returns the reciprocal root.
template <class T, int LPR, int KIND>
__device__ __forceinline__ float normalise(float (&v)[8], int kind, const Cols<T, KIND>& cols, const JoinArgs& a, RowSum<LPR>& sum) {
  if (kind == CC3D_NORM_NONE) return 1.f;
  if (kind == CC3D_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += cols.on(j) ? v[j] : 0.f;
    const float mean = sum.one(s) * a.inv_c;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = cols.on(j) ? v[j] : 0.f;
    q = fmaf(x, x, q);
  }
  const float rs = rsqrtf(fmaf(sum.one(q), a.inv_c, a.eps));
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= rs;
  return rs;
}

// The parameters of a lane's channels, in fp32 (they serve every row): ones
// and zeros where there are none.
template <class T, int KIND>
struct Params {
  float scale[8], w1[8], b1[8], w2[8], b2[8];
  __device__ __forceinline__ Params(const JoinArgs& a, const Cols<T, KIND>& cols) {
    auto get = [&](const void* p, float none, float (&v)[8]) {
      const Raw8<T> r = cols.param(p, none);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = get8(r, j);
    };
    get(a.scale, 1.f, scale);
    get(a.w1, 1.f, w1);
    get(a.b1, 0.f, b1);
    get(a.w2, 1.f, w2);
    get(a.b2, 0.f, b2);
  }
};

__device__ __forceinline__ float gate_of(float g, bool silu) { return silu ? g * sigmoid_f32(g) : g; }
__device__ __forceinline__ float silu_slope(float v) {
  const float s = sigmoid_f32(v);
  return s * (1.f + v * (1.f - s));
}

// One stream of rows: the workgroup's address of the first of its rows of one
// step, moved on by whole steps, and this lane's place behind it.
template <class T>
struct RowStream {
  T* p;
  int64_t row, at;
  __device__ __forceinline__ RowStream(const void* base, int64_t row, int64_t first, int line, int c0)
      : p(base ? const_cast<T*>(static_cast<const T*>(base)) + first * row : nullptr), row(row), at(line * row + c0) {}
  __device__ __forceinline__ void move(int64_t rows) { p += rows * row; }
};

// Calls run<T, LPR, KIND> for a plan's rows.
template <template <class, int, int> class Run, class T, class... A>
int pick_join(int c, A&&... args) {
  if (c < 8) return Run<T, 8, kFew>::run(args...);
  const bool even = c % 8 == 0;
  switch (cc3d::join_lanes(c)) {
    case 8: return even ? Run<T, 8, kEven>::run(args...) : Run<T, 8, kTail>::run(args...);
    case 16: return even ? Run<T, 16, kEven>::run(args...) : Run<T, 16, kTail>::run(args...);
    case 32: return even ? Run<T, 32, kEven>::run(args...) : Run<T, 32, kTail>::run(args...);
    case 64: return even ? Run<T, 64, kEven>::run(args...) : Run<T, 64, kTail>::run(args...);
    case 128: return even ? Run<T, 128, kEven>::run(args...) : Run<T, 128, kTail>::run(args...);
    case 256: return even ? Run<T, 256, kEven>::run(args...) : Run<T, 256, kTail>::run(args...);
    case 512: return even ? Run<T, 512, kEven>::run(args...) : Run<T, 512, kTail>::run(args...);
    default: return even ? Run<T, 1024, kEven>::run(args...) : Run<T, 1024, kTail>::run(args...);
  }
}

inline JoinArgs join_args(const cc3d_join_plan& p, const cc3d_join_args_t& c) {
  JoinArgs a{};
  a.y = c.y.p;
  a.res = c.residual.p;
  a.gate = c.gate.p;
  a.yr = c.y.row;
  a.rr = c.residual.row;
  a.gr = c.gate.row;
  a.scale = c.scale;
  a.w1 = c.post_w;
  a.b1 = c.post_b;
  a.w2 = c.pre_w;
  a.b2 = c.pre_b;
  a.rows = p.d.rows;
  a.gate_rows = p.d.gate_rows;
  a.gates = (p.d.rows + p.d.gate_rows - 1) / p.d.gate_rows;
  a.gate_parts = p.gate_parts;
  a.shared_gate = c.gate.p && p.d.gate_rows > 1;
  a.c = p.d.c;
  a.post = p.d.post;
  a.pre = p.d.pre;
  a.act = p.d.act;
  a.gate_act = c.gate.p ? p.d.gate_act : int(CC3D_ACT_NONE);  // without a gate its factor is one
  a.eps = p.d.eps;
  a.inv_c = 1.f / float(p.d.c);
  return a;
}

}  // namespace
