// Block join, forward: one read and one write of everything.
//
//   n1 = norm(y) * post_w + post_b;  x = residual + scale * ga(gate) * n1
//   h = act(norm(x) * pre_w + pre_b)
//
// Measured: 921600 rows of 192 bf16 channels, root-mean-square norms, scale and
// SiLU, in 290 us, 4.9 TB/s against a large copy's 4.74; the vector units are busy
// 94% of it, so either bound is near.  64 rows of 768: 4 us, the launch.
#include "cc3d_seq_join.h"

namespace {

template <class T, int LPR, int KIND>
__global__ __launch_bounds__(RowSum<LPR>::kThreads) void join_fwd(JoinArgs a) {
  constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
  __shared__ float box[2][2][kThreads / 64];
  RowSum<LPR> sum{box};
  const int line = threadIdx.x / LPR;
  const Cols<T, KIND> cols(int(threadIdx.x % LPR) * 8, a.c);
  const Params<T, KIND> p(a, cols);
  const bool gate_silu = a.gate_act == CC3D_ACT_SILU, act_silu = a.act == CC3D_ACT_SILU;
  const int64_t first = int64_t(blockIdx.x) * kAtOnce, step = int64_t(gridDim.x) * kAtOnce;
  RowStream<T> y(a.y, a.yr, first, line, cols.c0), res(a.res, a.rr, first, line, cols.c0),
      xo(a.xo, a.xr, first, line, cols.c0), ho(a.ho, a.hr, first, line, cols.c0);
  // the gate row of this lane's row, and how far that is into it
  int64_t g = 0, in_g = 0, g_step = 0, in_step = 0;
  if (a.gate) {
    g = (first + line) / a.gate_rows;
    in_g = first + line - g * a.gate_rows;
    g_step = step / a.gate_rows;
    in_step = step - g_step * a.gate_rows;
  }
  // (a row that is not there keeps what was in the registers: its results go nowhere)
  Raw8<T> next_y = zero8<T>(), next_r = zero8<T>(), next_g = cols.param(nullptr, 1.f);
  auto fetch = [&](int64_t base) {
    if (base + line >= a.rows) return;
    if (y.p) next_y = cols.load(y.p, y.at);
    if (res.p) next_r = cols.load(res.p, res.at);
    if (a.gate) next_g = cols.load(a.gate, g * a.gr + cols.c0);
  };
  fetch(first);
  // every thread of the workgroup takes part in every row's barriers
  for (int64_t base = first; base < a.rows; base += step) {
    const Raw8<T> ry = next_y, rr = next_r, rg = next_g;
    const bool there = base + line < a.rows;
    y.move(y.p ? step : 0);
    res.move(res.p ? step : 0);
    g += g_step;
    in_g += in_step;
    if (in_g >= a.gate_rows) {
      in_g -= a.gate_rows;
      ++g;
    }
    fetch(base + step);
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
        const float n1 = fmaf(v[j], p.w1[j], p.b1[j]);
        x[j] = fmaf(p.scale[j] * gate_of(get8(rg, j), gate_silu), n1, x[j]);
      }
    }
    if (xo.p) {
      if (there) cols.store(xo.p, xo.at, x);
      xo.move(step);
    }
    if (ho.p) {
      normalise(x, a.pre, cols, a, sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], p.w2[j], p.b2[j]);
      if (act_silu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= sigmoid_f32(x[j]);
      }
      if (there) cols.store(ho.p, ho.at, x);
      ho.move(step);
    }
  }
}

template <class T, int LPR, int KIND>
struct Forward {
  static int run(const JoinArgs& a, hipStream_t s) {
    constexpr int kThreads = RowSum<LPR>::kThreads, kAtOnce = kThreads / LPR;
    // two turns of the four waves a SIMD that its registers allow: one turn is 2 to 3%
    // slower (921600 rows of 192 bf16 channels 302 us for 296, 400000 of 96 64.8 for 63.0)
    return launch(join_fwd<T, LPR, KIND>, std::min<int64_t>((a.rows + kAtOnce - 1) / kAtOnce, 8192 * 64 / kThreads), kThreads, 0,
                  s, a);
  }
};

}  // namespace

namespace cc3d {

int launch_join_forward(const cc3d_join_plan& p, const cc3d_join_args_t& c, void* stream) {
  JoinArgs a = join_args(p, c);
  a.xo = c.x_out.p;
  a.ho = c.h_out.p;
  a.xr = c.x_out.row;
  a.hr = c.h_out.row;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p.d.dtype == CC3D_BF16 ? pick_join<Forward, bf16_s>(a.c, a, s) : pick_join<Forward, float>(a.c, a, s);
}

}  // namespace cc3d
