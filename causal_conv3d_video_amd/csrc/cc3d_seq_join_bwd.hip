// Block join, backward: one read of what the forward pass read and of the two
// gradients, one write of the inputs' gradients.
//
// Measured: 16386 rows of 2048 bf16 channels, every element gated, in 109 us with
// the sums, 4.9 TB/s against a large copy's 4.74; vector units busy 72%.  26520
// rows of 515 fp32 channels, 1560 rows a gate row, centred norms: 105 us, 3.1
// TB/s, vector units busy 65%, with the last 63 of a row's 128 lanes idle.
#include "cc3d_seq_join.h"

namespace {

// The row is computed again; then, with d the gradient of a norm's output
// times its weight and xn its normalised row,
//   gradient of its input = (d - xn * mean(d * xn) - [centred] mean(d)) / root.
// The parameters' gradients are sums over rows: kept in registers over every
// row that a workgroup takes, added over its lines of lanes in LDS and
// written as one row of partial sums a workgroup.
//
// A workgroup's rows are one stretch, walked in strides: every so many rows of
// all; or those of one gate row after another, when a gate row serves several
// rows and there are many; or a part of one gate row's.
template <class T, int LPR, int KIND>
__global__ __launch_bounds__(RowSum<LPR>::kThreads, LPR > 512 ? 4 : 2) void join_bwd(JoinArgs a) {
  constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
  constexpr bool kAhead = LPR < 1024;  // sixteen waves have 128 registers each: none for the next row
  __shared__ float box[2][2][kThreads / 64];
  __shared__ float red[kAtOnce > 1 ? kThreads * 8 : 1];
  RowSum<LPR> sum{box};
  const int line = threadIdx.x / LPR;
  const Cols<T, KIND> cols(int(threadIdx.x % LPR) * 8, a.c);
  const Params<T, KIND> p(a, cols);
  const bool gate_silu = a.gate_act == CC3D_ACT_SILU, act_silu = a.act == CC3D_ACT_SILU;
  const bool whole_gates = a.shared_gate && a.gate_parts == 0;
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

  Raw8<T> next_y = zero8<T>(), next_r = next_y, next_dx = next_y, next_dh = next_y, next_g = cols.param(nullptr, 1.f);
  int64_t span = blockIdx.x;  // the gate row, or the part of one
  do {
    int64_t lo = int64_t(blockIdx.x) * kAtOnce, hi = a.rows, step = int64_t(gridDim.x) * kAtOnce;
    if (a.shared_gate) {
      step = kAtOnce;
      const int64_t g = whole_gates ? span : span / a.gate_parts, q = whole_gates ? 0 : span - g * a.gate_parts;
      lo = g * a.gate_rows;
      hi = min(lo + a.gate_rows, a.rows);
      if (!whole_gates) {
        const int64_t n = hi - lo;
        hi = lo + n * (q + 1) / a.gate_parts;
        lo += n * q / a.gate_parts;
      }
    }
    RowStream<T> y(a.y, a.yr, lo, line, cols.c0), res(a.res, a.rr, lo, line, cols.c0),
        dxo(a.dxo, a.dxr, lo, line, cols.c0), dh(a.dh, a.dhr, lo, line, cols.c0);
    RowStream<T> dy(a.dy, a.dyr, lo, line, cols.c0), dres(a.dres, a.drr, lo, line, cols.c0);
    // a gate row of its own for every row, or one for the whole stretch
    RowStream<T> gate(a.gate, a.gr, a.shared_gate ? lo / a.gate_rows : lo, a.shared_gate ? 0 : line, cols.c0);
    RowStream<T> dgate(a.shared_gate ? nullptr : a.dgate, a.dgr, lo, line, cols.c0);
    if (a.gate && a.shared_gate) next_g = cols.load(gate.p, gate.at);
    auto fetch = [&](int64_t base) {
      if (base + line >= hi) {  // a row that is not there: zeros, whatever the one before held
        next_y = next_r = next_dx = next_dh = zero8<T>();
        return;
      }
      if (y.p) next_y = cols.load(y.p, y.at);
      if (res.p) next_r = cols.load(res.p, res.at);
      if (gate.p && !a.shared_gate) next_g = cols.load(gate.p, gate.at);
      if (dxo.p) next_dx = cols.load(dxo.p, dxo.at);
      if (dh.p) next_dh = cols.load(dh.p, dh.at);
      y.move(y.p ? step : 0);
      res.move(res.p ? step : 0);
      gate.move(gate.p && !a.shared_gate ? step : 0);
      dxo.move(dxo.p ? step : 0);
      dh.move(dh.p ? step : 0);
    };
    if (kAhead) fetch(lo);
    for (int64_t base = lo; base < hi; base += step) {
      const bool there = base + line < hi;
      if (!kAhead) fetch(base);
      const Raw8<T> ry = next_y, rr = next_r, rg = next_g, rdx = next_dx, rdh = next_dh;
      if (kAhead) fetch(base + step);
      float xn1[8], x[8], dx[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xn1[j] = get8(ry, j);
        x[j] = get8(rr, j);
        dx[j] = get8(rdx, j);
      }
      // the gate's factor and slope, once for both of their places
      float ga[8], slope[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) ga[j] = get8(rg, j);
      if (gate_silu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float g = ga[j], sg = sigmoid_f32(g);
          ga[j] = g * sg;
          slope[j] = sg * (1.f + g * (1.f - sg));
        }
      }
      const float rs1 = a.y ? normalise(xn1, a.post, cols, a, sum) : 1.f;
      if (a.dh) {
        // (a row that is not there stays zero: an infinite gate times it would reach every channel)
        if (a.y && (kAtOnce == 1 || there)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fmaf(p.scale[j] * ga[j], fmaf(xn1[j], p.w1[j], p.b1[j]), x[j]);
        }
        const float rs2 = normalise(x, a.pre, cols, a, sum);
        float d[8], m = 0.f, md = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float g = get8(rdh, j);
          if (act_silu) g *= silu_slope(fmaf(x[j], p.w2[j], p.b2[j]));
          acc[3][j] = fmaf(g, x[j], acc[3][j]);
          acc[4][j] += g;
          d[j] = g * p.w2[j];
          const float own = cols.on(j) ? d[j] : 0.f;
          m = fmaf(own, x[j], m);
          md += own;
        }
        sum.two(m, md);
        m *= a.inv_c;
        md = a.pre == CC3D_NORM_LAYER ? md * a.inv_c : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] = fmaf(rs2, d[j] - fmaf(x[j], m, md), dx[j]);
      }
      if (dres.p) {
        if (there) cols.store(dres.p, dres.at, dx);
        dres.move(step);
      }
      if (!a.y) continue;
      float dn[8], dg[8], m = 0.f, md = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = p.scale[j];
        const float along = dx[j] * fmaf(xn1[j], p.w1[j], p.b1[j]);
        acc[0][j] = fmaf(along, ga[j], acc[0][j]);
        dg[j] = along * s;
        acc[5][j] += dg[j];  // (left alone without a shared gate)
        if (gate_silu) dg[j] *= slope[j];
        dn[j] = dx[j] * s * ga[j];
        acc[1][j] = fmaf(dn[j], xn1[j], acc[1][j]);
        acc[2][j] += dn[j];
        dn[j] *= p.w1[j];
        const float own = cols.on(j) ? dn[j] : 0.f;
        m = fmaf(own, xn1[j], m);
        md += own;
      }
      if (dgate.p) {
        if (there) cols.store(dgate.p, dgate.at, dg);
        dgate.move(step);
      }
      if (!dy.p) continue;
      if (a.post != CC3D_NORM_NONE) {
        sum.two(m, md);
        m *= a.inv_c;
        md = a.post == CC3D_NORM_LAYER ? md * a.inv_c : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) dn[j] = rs1 * (dn[j] - fmaf(xn1[j], m, md));
      }
      if (there) cols.store(dy.p, dy.at, dn);
      dy.move(step);
    }
    if (!whole_gates) break;
    over_lines(acc[5]);
    if (a.dgate && threadIdx.x < LPR) {
      const Raw8<T> rg = cols.load(a.gate, span * a.gr + cols.c0);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[5][j] * (gate_silu ? silu_slope(get8(rg, j)) : 1.f);
      cols.store(a.dgate, span * a.dgr + cols.c0, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[5][j] = 0.f;
    span += gridDim.x;
  } while (span < a.gates);

  const int kinds = a.gate_parts ? 6 : 5;
  float* part = a.part + int64_t(blockIdx.x) * kinds * a.c;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    if (i < kinds) {
      over_lines(acc[i]);
      if (threadIdx.x < LPR) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (cols.on(j)) part[int64_t(i) * a.c + cols.c0 + j] = acc[i][j];
      }
    }
  }
}

// The gradient of a gate row from the partial sums of its workgroups: 64
// columns of one gate row a workgroup, as in sum_rows.
template <class T>
__global__ __launch_bounds__(256) void gate_sum(JoinArgs a) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x % 64, line = threadIdx.x / 64, tiles = (a.c + 63) / 64;
  const int64_t g = blockIdx.x / tiles;
  const int c = int(blockIdx.x - g * tiles) * 64 + lane;
  const float* src = a.part + (g * a.gate_parts * 6 + 5) * a.c + min(c, a.c - 1);
  float s = 0.f;
  for (int64_t q0 = line; q0 < a.gate_parts; q0 += 32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q0 + 4 * i < a.gate_parts ? src[(q0 + 4 * i) * 6 * a.c] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  red[line][lane] = s;
  __syncthreads();
  if (line != 0 || c >= a.c) return;
  s += red[1][lane] + red[2][lane] + red[3][lane];
  if (a.gate_act == CC3D_ACT_SILU) s *= silu_slope(to_f32(static_cast<const T*>(a.gate)[g * a.gr + c]));
  static_cast<T*>(a.dgate)[g * a.dgr + c] = from_f32<T>(s);
}

template <class T, int LPR, int KIND>
struct Backward {
  static int run(const JoinArgs& a, int64_t parts, hipStream_t s) {
    return launch(join_bwd<T, LPR, KIND>, parts, RowSum<LPR>::kThreads, 0, s, a);
  }
};

}  // namespace

namespace cc3d {

int launch_join_backward(const cc3d_join_plan& p, const cc3d_join_args_t& c, void* stream) {
  JoinArgs a = join_args(p, c);
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
  hipStream_t s = static_cast<hipStream_t>(stream);
  int e = p.d.dtype == CC3D_BF16 ? pick_join<Backward, bf16_s>(a.c, a, p.bwd_parts, s)
                                 : pick_join<Backward, float>(a.c, a, p.bwd_parts, s);
  if (!e && a.gate_parts && a.shared_gate && a.dgate) {
    e = launch(p.d.dtype == CC3D_BF16 ? gate_sum<bf16_s> : gate_sum<float>, a.gates * ((a.c + 63) / 64), 256, 0, s, a);
  }
  if (e) return e;
  const int64_t stride = int64_t(a.gate_parts ? 6 : 5) * a.c;
  float* out[5] = {c.dscale, c.dpost_w, c.dpost_b, c.dpre_w, c.dpre_b};
  SumJob jobs[5];
  for (int i = 0; i < 5; ++i) jobs[i] = {a.part + int64_t(i) * a.c, out[i], p.bwd_parts, a.c, stride};
  return launch_sums(jobs, 5, stream);
}

}  // namespace cc3d
