// Block join: the norm after a block, its gate, the residual scale and sum,
// and the norm and activation before the next block, forward and backward.
//
//   n1 = norm(y) * post_w + post_b;  x = residual + scale * ga(gate) * n1
//   h = act(norm(x) * pre_w + pre_b)
//
// About 16 operations an element against at least two elements read and two
// written: bound by memory.  A row lives in the registers of LPR lanes (eight
// channels each, a power of two of lanes, so four rows of 96 channels share a
// wave and a row of 8192 takes a workgroup): everything is read once, both
// norms' sums are taken over registers (the mean first where there is one, then
// the squares about it), and both results are written from the same pass.
// Where a pointer or a stride does not allow 16-byte accesses the lanes take
// every LPR-th channel instead.
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

// Eight channels of a lane: consecutive ones, or every LPR-th.
template <class T, int LPR, bool VEC>
struct Cols {
  int lane, c;
  __device__ __forceinline__ int at(int j) const { return VEC ? lane * 8 + j : j * LPR + lane; }
  __device__ __forceinline__ bool on(int j) const { return VEC ? lane * 8 < c : j * LPR + lane < c; }
  // zeros outside the row, and everywhere when there is no row or no pointer
  __device__ __forceinline__ void load(const void* p, int64_t off, bool there, Raw8<T>& r) const {
    r = zero8<T>();
    if (!p || !there) return;
    const T* q = static_cast<const T*>(p) + off;
    if constexpr (VEC) {
      if (lane * 8 < c) r = load8(q + lane * 8);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (on(j)) set(r, j, q[at(j)]);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t off, const float* v) const {
    T* q = static_cast<T*>(p) + off;
    if constexpr (VEC) {
      if (lane * 8 < c) store8(q + lane * 8, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (on(j)) q[at(j)] = from_f32<T>(v[j]);
    }
  }
  static __device__ __forceinline__ void set(Raw8<T>& r, int j, T v) {
    if constexpr (sizeof(T) == 4) r.q[j / 4][j % 4] = __float_as_uint(v);
    else r.q[0][j / 2] |= unsigned(v) << (16 * (j & 1));
  }
};

// Sums over a row's LPR lanes.  Rows wider than a wave pass through LDS, in
// two slots used in turn, so one barrier a sum is enough.
template <int LPR>
struct RowSum {
  static constexpr int kThreads = LPR > cc3d::kJoinThreads ? LPR : cc3d::kJoinThreads;
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

// The norm of a row: v becomes the normalised row (zero outside it); returns
// the reciprocal root.
template <int LPR, class C>
__device__ __forceinline__ float normalise(float (&v)[8], int kind, const C& cols, const JoinArgs& a, RowSum<LPR>& sum) {
  if (kind == CC3D_NORM_NONE) return 1.f;
  if (kind == CC3D_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[j];
    const float mean = sum.one(s) * a.inv_c;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = cols.on(j) ? v[j] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
  const float rs = rsqrtf(fmaf(sum.one(q), a.inv_c, a.eps));
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= rs;
  return rs;
}

__device__ __forceinline__ int64_t gate_row(const JoinArgs& a, int64_t row) {
  if (a.gate_rows == 1) return row;
  if (a.rows < (int64_t(1) << 31)) return a.gate_rows > row ? 0 : unsigned(row) / unsigned(a.gate_rows);
  return row / a.gate_rows;
}

// The parameters of a lane's channels: ones and zeros where there are none.
template <class T, int LPR, bool VEC>
struct Params {
  Raw8<T> scale, w1, b1, w2, b2;
  __device__ __forceinline__ void load(const JoinArgs& a, const Cols<T, LPR, VEC>& cols) {
    cols.load(a.scale, 0, true, scale);
    cols.load(a.w1, 0, true, w1);
    cols.load(a.b1, 0, true, b1);
    cols.load(a.w2, 0, true, w2);
    cols.load(a.b2, 0, true, b2);
  }
};

template <class T, int LPR, bool VEC>
__global__ __launch_bounds__(RowSum<LPR>::kThreads) void join_fwd(JoinArgs a) {
  constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
  __shared__ float box[2][2][kThreads / 64];
  RowSum<LPR> sum{box};
  const Cols<T, LPR, VEC> cols{int(threadIdx.x % LPR), a.c};
  Params<T, LPR, VEC> p;
  p.load(a, cols);
  // every thread of the workgroup takes part in every row's barriers
  for (int64_t base = int64_t(blockIdx.x) * kAtOnce; base < a.rows; base += int64_t(gridDim.x) * kAtOnce) {
    const int64_t row = base + threadIdx.x / LPR;
    const bool there = row < a.rows;
    Raw8<T> ry, rr, rg;
    cols.load(a.y, row * a.yr, there, ry);
    cols.load(a.res, row * a.rr, there, rr);
    if (a.gate) cols.load(a.gate, gate_row(a, row) * a.gr, there, rg);
    float v[8], x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = get8(ry, j);
      x[j] = get8(rr, j);
    }
    if (a.y) {
      normalise(v, a.post, cols, a, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (a.w1) v[j] *= get8(p.w1, j);
        if (a.b1) v[j] += get8(p.b1, j);
        float f = a.scale ? get8(p.scale, j) : 1.f;
        if (a.gate) {
          const float g = get8(rg, j);
          f *= a.gate_act == CC3D_ACT_SILU ? g * sigmoid_f32(g) : g;
        }
        x[j] = fmaf(f, v[j], x[j]);
      }
    }
    if (a.xo && there) cols.store(a.xo, row * a.xr, x);
    if (a.ho) {
      normalise(x, a.pre, cols, a, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (a.w2) x[j] *= get8(p.w2, j);
        if (a.b2) x[j] += get8(p.b2, j);
        if (a.act == CC3D_ACT_SILU) x[j] *= sigmoid_f32(x[j]);
      }
      if (there) cols.store(a.ho, row * a.hr, x);
    }
  }
}

// Backward.  The row is computed again; then, with d the gradient of a
// norm's output times its weight and xn its normalised row,
//   gradient of its input = (d - xn * mean(d * xn) - [centred] mean(d)) / root.
// The parameters' gradients are sums over rows: kept in registers over every
// row that a workgroup takes, added over its lines of lanes in LDS and
// written as one row of partial sums a workgroup.
template <class T, int LPR, bool VEC>
__global__ __launch_bounds__(RowSum<LPR>::kThreads) void join_bwd(JoinArgs a) {
  constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
  __shared__ float box[2][2][kThreads / 64];
  __shared__ float red[kThreads * 8];
  RowSum<LPR> sum{box};
  const Cols<T, LPR, VEC> cols{int(threadIdx.x % LPR), a.c};
  Params<T, LPR, VEC> p;
  p.load(a, cols);
  float acc[6][8] = {};  // dscale, dw1, db1, dw2, db2 and a shared gate's gradient

  // acc[i] over the workgroup's lines of lanes, in the first line's lanes
  auto over_lines = [&](float (&v)[8]) {
    if constexpr (kAtOnce > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = v[j];
      __syncthreads();
      if (threadIdx.x < LPR) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float s = 0.f;
          for (int l = 0; l < kAtOnce; ++l) s += red[(l * LPR + threadIdx.x) * 8 + j];
          v[j] = s;
        }
      }
    }
  };

  auto one_row = [&](int64_t row, bool there) {
    Raw8<T> ry, rr, rg, rdx, rdh;
    cols.load(a.y, row * a.yr, there, ry);
    cols.load(a.res, row * a.rr, there, rr);
    if (a.gate) cols.load(a.gate, gate_row(a, row) * a.gr, there, rg);
    cols.load(a.dxo, row * a.dxr, there, rdx);
    cols.load(a.dh, row * a.dhr, there, rdh);
    float xn1[8], x[8], dx[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xn1[j] = get8(ry, j);
      x[j] = get8(rr, j);
      dx[j] = get8(rdx, j);
    }
    const float rs1 = a.y ? normalise(xn1, a.post, cols, a, sum) : 1.f;
    auto factor = [&](int j, float& ga, float& slope) {
      ga = 1.f;
      slope = 0.f;
      if (a.gate) {
        const float g = get8(rg, j);
        if (a.gate_act == CC3D_ACT_SILU) {
          const float s = sigmoid_f32(g);
          ga = g * s;
          slope = s * (1.f + g * (1.f - s));
        } else {
          ga = g;
          slope = 1.f;
        }
      }
      return a.scale ? get8(p.scale, j) : 1.f;
    };
    auto after = [&](int j) {  // n1
      float v = xn1[j];
      if (a.w1) v *= get8(p.w1, j);
      if (a.b1) v += get8(p.b1, j);
      return v;
    };
    if (a.dh) {
      if (a.y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float ga, slope;
          const float s = factor(j, ga, slope);
          x[j] = fmaf(s * ga, after(j), x[j]);
        }
      }
      const float rs2 = normalise(x, a.pre, cols, a, sum);
      float d[8], m = 0.f, md = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float g = get8(rdh, j);
        const float w = a.w2 ? get8(p.w2, j) : 1.f;
        if (a.act == CC3D_ACT_SILU) {
          float h = x[j] * w;
          if (a.b2) h += get8(p.b2, j);
          const float s = sigmoid_f32(h);
          g *= s * (1.f + h * (1.f - s));
        }
        acc[3][j] = fmaf(g, x[j], acc[3][j]);
        acc[4][j] += g;
        d[j] = g * w;
        m = fmaf(d[j], x[j], m);
        md += d[j];
      }
      sum.two(m, md);
      m *= a.inv_c;
      md = a.pre == CC3D_NORM_LAYER ? md * a.inv_c : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dx[j] = fmaf(rs2, d[j] - fmaf(x[j], m, md), dx[j]);
    }
    if (a.dres && there) cols.store(a.dres, row * a.drr, dx);
    if (!a.y) return;
    float dn[8], dg[8], m = 0.f, md = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float ga, slope;
      const float s = factor(j, ga, slope);
      const float along = dx[j] * after(j);
      acc[0][j] = fmaf(along, ga, acc[0][j]);
      dg[j] = along * s;
      if (a.shared_gate) acc[5][j] += dg[j];
      else dg[j] *= slope;
      dn[j] = dx[j] * s * ga;
      acc[1][j] = fmaf(dn[j], xn1[j], acc[1][j]);
      acc[2][j] += dn[j];
      if (a.w1) dn[j] *= get8(p.w1, j);
      m = fmaf(dn[j], xn1[j], m);
      md += dn[j];
    }
    if (a.dgate && !a.shared_gate && there) cols.store(a.dgate, row * a.dgr, dg);
    if (!a.dy) return;
    if (a.post != CC3D_NORM_NONE) {
      sum.two(m, md);
      m *= a.inv_c;
      md = a.post == CC3D_NORM_LAYER ? md * a.inv_c : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dn[j] = rs1 * (dn[j] - fmaf(xn1[j], m, md));
    }
    if (there) cols.store(a.dy, row * a.dyr, dn);
  };

  const int line = threadIdx.x / LPR;
  if (!a.shared_gate) {
    for (int64_t base = int64_t(blockIdx.x) * kAtOnce; base < a.rows; base += int64_t(gridDim.x) * kAtOnce)
      one_row(base + line, base + line < a.rows);
  } else if (a.gate_parts == 0) {  // whole gate rows
    for (int64_t g = blockIdx.x; g < a.gates; g += gridDim.x) {
      const int64_t lo = g * a.gate_rows, hi = min(lo + a.gate_rows, a.rows);
      for (int64_t base = lo; base < hi; base += kAtOnce) one_row(base + line, base + line < hi);
      over_lines(acc[5]);
      if (a.dgate && threadIdx.x < LPR) {
        Raw8<T> rg;
        cols.load(a.gate, g * a.gr, true, rg);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gt = get8(rg, j), s = sigmoid_f32(gt);
          v[j] = acc[5][j] * (a.gate_act == CC3D_ACT_SILU ? s * (1.f + gt * (1.f - s)) : 1.f);
        }
        cols.store(a.dgate, g * a.dgr, v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[5][j] = 0.f;
    }
  } else {  // a part of one gate row
    const int64_t g = blockIdx.x / a.gate_parts, q = blockIdx.x - g * a.gate_parts;
    const int64_t lo = g * a.gate_rows, hi = min(lo + a.gate_rows, a.rows), n = hi - lo;
    const int64_t from = lo + n * q / a.gate_parts, to = lo + n * (q + 1) / a.gate_parts;
    for (int64_t base = from; base < to; base += kAtOnce) one_row(base + line, base + line < to);
  }

  const int kinds = a.gate_parts ? 6 : 5;
  float* part = a.part + int64_t(blockIdx.x) * kinds * a.c;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    if (i < kinds) {
      over_lines(acc[i]);
      if (threadIdx.x < LPR) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (cols.on(j)) part[int64_t(i) * a.c + cols.at(j)] = acc[i][j];
      }
    }
  }
}

// The gradient of a gate row from the partial sums of its workgroups.
template <class T>
__global__ __launch_bounds__(256) void gate_sum(JoinArgs a) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t g = id / a.c;
  if (g >= a.gates) return;
  const int c = int(id - g * a.c);
  float s = 0.f;
  for (int64_t q = 0; q < a.gate_parts; ++q) s += a.part[((g * a.gate_parts + q) * 6 + 5) * a.c + c];
  if (a.gate_act == CC3D_ACT_SILU) {
    const float gt = to_f32(static_cast<const T*>(a.gate)[g * a.gr + c]), sg = sigmoid_f32(gt);
    s *= sg * (1.f + gt * (1.f - sg));
  }
  static_cast<T*>(a.dgate)[g * a.dgr + c] = from_f32<T>(s);
}

template <class T, int LPR>
void run_lanes(const JoinArgs& a, bool vec, int64_t parts, hipStream_t s) {
  constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
  if (parts) {
    if (vec) join_bwd<T, LPR, true><<<unsigned(parts), kThreads, 0, s>>>(a);
    else join_bwd<T, LPR, false><<<unsigned(parts), kThreads, 0, s>>>(a);
  } else {
    const unsigned blocks = unsigned(std::min<int64_t>((a.rows + kAtOnce - 1) / kAtOnce, 2048));
    if (vec) join_fwd<T, LPR, true><<<blocks, kThreads, 0, s>>>(a);
    else join_fwd<T, LPR, false><<<blocks, kThreads, 0, s>>>(a);
  }
}

template <class T>
void run_join(const JoinArgs& a, bool vec, int64_t parts, hipStream_t s) {
  switch (cc3d::join_lanes(a.c)) {
    case 8: return run_lanes<T, 8>(a, vec, parts, s);
    case 16: return run_lanes<T, 16>(a, vec, parts, s);
    case 32: return run_lanes<T, 32>(a, vec, parts, s);
    case 64: return run_lanes<T, 64>(a, vec, parts, s);
    case 128: return run_lanes<T, 128>(a, vec, parts, s);
    case 256: return run_lanes<T, 256>(a, vec, parts, s);
    case 512: return run_lanes<T, 512>(a, vec, parts, s);
    default: return run_lanes<T, 1024>(a, vec, parts, s);
  }
}

bool vec_ok(const cc3d_rows_t& v) {
  return !v.p || (reinterpret_cast<uintptr_t>(v.p) % 16 == 0 && v.row % 8 == 0);
}

JoinArgs base_args(const cc3d_join_plan& p, const cc3d_join_args_t& c, bool& vec) {
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
  a.gate_act = p.d.gate_act;
  a.eps = p.d.eps;
  a.inv_c = 1.f / float(p.d.c);
  vec = p.d.c % 8 == 0 && vec_ok(c.y) && vec_ok(c.residual) && vec_ok(c.gate);
  for (const void* q : {a.scale, a.w1, a.b1, a.w2, a.b2}) vec = vec && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  return a;
}

}  // namespace

namespace cc3d {

int launch_join_forward(const cc3d_join_plan& p, const cc3d_join_args_t& c, void* stream) {
  bool vec;
  JoinArgs a = base_args(p, c, vec);
  a.xo = c.x_out.p;
  a.ho = c.h_out.p;
  a.xr = c.x_out.row;
  a.hr = c.h_out.row;
  vec = vec && vec_ok(c.x_out) && vec_ok(c.h_out);
  if (p.d.dtype == CC3D_BF16) run_join<bf16_s>(a, vec, 0, static_cast<hipStream_t>(stream));
  else run_join<float>(a, vec, 0, static_cast<hipStream_t>(stream));
  return int(hipGetLastError());
}

int launch_join_backward(const cc3d_join_plan& p, const cc3d_join_args_t& c, void* stream) {
  bool vec;
  JoinArgs a = base_args(p, c, vec);
  a.dxo = c.dx_out.p;
  a.dh = c.dh.p;
  a.dy = c.dy.p;
  a.dres = c.dresidual.p;
  a.dgate = c.dgate.p;
  a.dxr = c.dx_out.row;
  a.dhr = c.dh.row;
  a.dyr = c.dy.row;
  a.drr = c.dresidual.row;
  a.dgr = c.dgate.row;
  a.part = static_cast<float*>(c.workspace);
  vec = vec && vec_ok(c.dx_out) && vec_ok(c.dh) && vec_ok(c.dy) && vec_ok(c.dresidual) && vec_ok(c.dgate);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p.d.dtype == CC3D_BF16) run_join<bf16_s>(a, vec, p.bwd_parts, s);
  else run_join<float>(a, vec, p.bwd_parts, s);
  int e = int(hipGetLastError());
  if (!e && a.gate_parts && a.shared_gate && a.dgate) {
    const unsigned blocks = unsigned((a.gates * a.c + 255) / 256);
    if (p.d.dtype == CC3D_BF16) gate_sum<bf16_s><<<blocks, 256, 0, s>>>(a);
    else gate_sum<float><<<blocks, 256, 0, s>>>(a);
    e = int(hipGetLastError());
  }
  const int64_t stride = int64_t(a.gate_parts ? 6 : 5) * a.c;
  float* out[5] = {c.dscale, c.dpost_w, c.dpost_b, c.dpre_w, c.dpre_b};
  for (int i = 0; i < 5 && !e; ++i)
    e = launch_sum_rows(a.part + int64_t(i) * a.c, p.bwd_parts, a.c, stride, out[i], stream);
  return e;
}

}  // namespace cc3d
