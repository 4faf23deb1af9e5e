// Linear attention with a decay for each head: the kernels beside the
// recurrence (cc3d_heads_linear.h), and the launches.
#include "cc3d_heads_linear.h"

#include <algorithm>

namespace {

struct StepArgs {
  const void *q, *k, *v;
  void* o;
  int64_t qb, kb, vb, ob;
  int qper, kper, vper;
  int heads, dk, dv, lanes;  // lanes side by side along Dv, four columns each, a power of two
  float scale;
  const float *log_decay, *h_in;
  float* h_out;
  const int* lengths;
};

// One token: S = f S + k^T v, o = scale q S, in fp32.  Reads and writes each
// state once and does little besides: bound by memory.  A workgroup has one
// head; its threads are rows of `lanes` lanes with four columns of the state
// each, eight rows in flight before any is used; q S is summed over a thread's
// rows, across the lanes of a wave and across the waves.
template <class T>
__global__ __launch_bounds__(256) void linear_step(StepArgs a) {
  __shared__ float box[4][256];
  const int tid = threadIdx.x, line = tid / a.lanes, lines = 256 / a.lanes, e = tid % a.lanes * 4;
  const int64_t nh = blockIdx.x, n = nh / a.heads;
  const int h = int(nh - n * a.heads), width = a.dv - e;
  const bool on = valid_tokens(a.lengths, int(n), 1) > 0;
  const T* q = static_cast<const T*>(a.q) + n * a.qb + int64_t(h / a.qper) * a.dk;
  const T* k = static_cast<const T*>(a.k) + n * a.kb + int64_t(h / a.kper) * a.dk;
  const T* v = static_cast<const T*>(a.v) + n * a.vb + int64_t(h / a.vper) * a.dv;
  const int64_t base = nh * a.dk * a.dv + e;
  const float f = a.log_decay ? __builtin_amdgcn_exp2f(a.log_decay[h] * kLog2e) : 1.f;
  float vv[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) vv[i] = on && i < width ? to_f32(v[e + i]) : 0.f;
  constexpr int kAhead = 8;
  for (int c0 = line; c0 < a.dk; c0 += lines * kAhead) {
    f32x4_s s[kAhead];
    float kk[kAhead], qq[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int c = c0 + x * lines;
      s[x] = zero4();
      kk[x] = qq[x] = 0.f;
      if (c < a.dk && width > 0) {
        if (on) {
          kk[x] = to_f32(k[c]);
          qq[x] = to_f32(q[c]);
        }
        if (a.h_in) {
          const float* p = a.h_in + base + int64_t(c) * a.dv;
          if (width >= 4) s[x] = __builtin_bit_cast(f32x4_s, *reinterpret_cast<const u32x4_by4*>(p));
          else
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (i < width) s[x][i] = p[i];
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int c = c0 + x * lines;
      if (c >= a.dk || width <= 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (on) s[x][i] = fmaf(f, s[x][i], kk[x] * vv[i]);
        o[i] = on ? fmaf(qq[x], s[x][i], o[i]) : 0.f;
      }
      if (a.h_out) {
        float* p = a.h_out + base + int64_t(c) * a.dv;
        if (width >= 4) *reinterpret_cast<u32x4_by4*>(p) = __builtin_bit_cast(u32x4_s, s[x]);
        else
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < width) p[i] = s[x][i];
      }
    }
  }
  for (int d = a.lanes; d < 64; d *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], d);
  if (tid % 64 < a.lanes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) box[tid / 64][e + i] = o[i];
  }
  __syncthreads();
  if (tid < a.dv) {
    const float sum = (box[0][tid] + box[1][tid]) + (box[2][tid] + box[3][tid]);
    static_cast<T*>(a.o)[n * a.ob + int64_t(h) * a.dv + tid] = from_f32<T>(sum * a.scale);
  }
}

struct JoinArgs {
  struct Way {
    const float* from;  // [N][H][size], or null
    float* segs;        // [N][H][segments - 1][size]: what a segment adds; becomes the state after it
    float* segs2;       // the derivative by the decay, or null
  } way[2];
  int64_t items, size;  // states of all heads, floats of one
  int heads, t, seg, segs;
  const float* log_decay;
  const int* lengths;
};

// States across segments: after[s] = f[tokens of s] before[s] + added[s], and
// of its derivative S2 by the decay f (S2 + tokens S) + added2.  Four segments'
// loads are in flight.
__global__ __launch_bounds__(256) void linear_join(JoinArgs a) {
  const JoinArgs::Way w = a.way[blockIdx.y];
  for (int64_t item = int64_t(blockIdx.x) * 256 + threadIdx.x; item < a.items; item += int64_t(gridDim.x) * 256) {
    const int64_t nh = item / a.size, off = item - nh * a.size, n = nh / a.heads;
    const float g = a.log_decay ? a.log_decay[nh - n * a.heads] : 0.f;
    const int len = valid_tokens(a.lengths, int(n), a.t);
    const float whole = fade_m1(g, a.seg);
    float* p = w.segs + nh * (a.segs - 1) * a.size + off;
    float* p2 = w.segs2 ? w.segs2 + nh * (a.segs - 1) * a.size + off : nullptr;
    float s = w.from ? w.from[item] : 0.f, s2 = 0.f;
    for (int x0 = 0; x0 < a.segs - 1; x0 += 4) {
      float u[4], u2[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool in = x0 + x < a.segs - 1;
        u[x] = in ? p[(x0 + x) * a.size] : 0.f;
        u2[x] = in && p2 ? p2[(x0 + x) * a.size] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x0 + x >= a.segs - 1) break;
        const int tokens = min(max(len - (x0 + x) * a.seg, 0), a.seg);
        const float m1 = tokens == a.seg ? whole : fade_m1(g, tokens);
        const float both = fmaf(float(tokens), s, s2);
        s2 = fmaf(both, m1, both) + u2[x];
        s = fmaf(s, m1, s) + u[x];
        p[(x0 + x) * a.size] = s;
        if (p2) p2[(x0 + x) * a.size] = s2;
      }
    }
  }
}

struct HeadSum {
  const float* part;  // [N][T][heads][D]
  void* out;
  int64_t batch, row, el;  // el: N T (heads / per) D
  int per, d, t, heads;    // heads: of the result
};
struct HeadSums {
  HeadSum job[3];
};

// Gradients of shared heads: sums over the heads that share one, in order.
template <class T>
__global__ __launch_bounds__(256) void linear_heads(HeadSums a) {
  const HeadSum j = a.job[blockIdx.y];
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < j.el; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / j.d, d = i - row * j.d;       // (n, t, head) and column
    const int64_t tok = row / j.heads, head = row - tok * j.heads, n = tok / j.t;
    const float* p = j.part + row * j.per * j.d + d;
    float s = 0.f;
    for (int x = 0; x < j.per; ++x) s += p[int64_t(x) * j.d];
    static_cast<T*>(j.out)[n * j.batch + (tok - n * j.t) * j.row + head * j.d + d] = from_f32<T>(s);
  }
}

// dlog_decay: a workgroup's partial sums of one head, each thread's in order, then a tree.
__global__ __launch_bounds__(256) void linear_decay(const double* part, float* out, int n, int heads, int each) {
  __shared__ double box[256];
  const int h = blockIdx.x, tid = threadIdx.x;
  double s = 0.0;
  for (int64_t i = tid; i < int64_t(n) * each; i += 256) {
    const int64_t b = i / each;
    s += part[(b * heads + h) * each + (i - b * each)];
  }
  box[tid] = s;
  __syncthreads();
  for (int half = 128; half > 0; half /= 2) {
    if (tid < half) box[tid] += box[tid + half];
    __syncthreads();
  }
  if (tid == 0) out[h] = float(box[0]);
}

constexpr int64_t kGrid = 1 << 16;  // workgroups of the kernels that walk their work in turns

int run(cc3d::LinArgs& a, const cc3d_linear_desc_t& d, int pad, bool out, bool dec, hipStream_t s) {
  static cc3d::LinStart* const of[2][3] = {
      {cc3d::linear_f32_eights, cc3d::linear_f32_rest, cc3d::linear_f32_less},
      {cc3d::linear_bf16_eights, cc3d::linear_bf16_rest, cc3d::linear_bf16_less}};
  const int kind = std::min(d.dk, d.dv) < 8 ? kLess : d.dk % 8 || d.dv % 8 ? kRest : kEights;
  return of[d.dtype == CC3D_BF16][kind](a, pad, out, dec, s);
}

cc3d::LinArgs common(const cc3d_linear_plan& p, const cc3d_linear_args_t& c, int seg, int segs) {
  cc3d::LinArgs a{};
  a.n = p.d.n;
  a.heads = p.d.heads;
  a.t = p.d.t;
  a.seg = seg;
  a.segs = segs;
  a.log_decay = c.log_decay;
  a.lengths = c.lengths;
  return a;
}

JoinArgs join_of(const cc3d::LinArgs& a, int64_t size) {
  JoinArgs j{};
  j.size = size;
  j.items = int64_t(a.n) * a.heads * size;
  j.heads = a.heads;
  j.t = a.t;
  j.seg = a.seg;
  j.segs = a.segs;
  j.log_decay = a.log_decay;
  j.lengths = a.lengths;
  return j;
}

int start_join(const JoinArgs& j, int ways, hipStream_t s) {
  void* at[] = {const_cast<JoinArgs*>(&j)};
  const int64_t blocks = std::min((j.items + 255) / 256, kGrid);
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&linear_join), dim3(unsigned(blocks), unsigned(ways)),
                                       dim3(256), at, 0, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return int(e);
}

}  // namespace

namespace cc3d {

int launch_linear_forward(const cc3d_linear_plan& p, const cc3d_linear_args_t& c, void* stream) {
  const auto& d = p.d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (d.t == 1) {
    StepArgs a{c.q.p, c.k.p, c.v.p, c.o.p, c.q.batch, c.k.batch, c.v.batch, c.o.batch, d.heads / d.q_heads,
               d.heads / d.k_heads, d.heads / d.v_heads, d.heads, d.dk, d.dv, 1, d.scale, c.log_decay, c.h_in, c.h_out,
               c.lengths};
    while (a.lanes * 4 < d.dv) a.lanes *= 2;
    const int64_t workgroups = int64_t(d.n) * d.heads;
    return d.dtype == CC3D_BF16 ? launch(linear_step<bf16_s>, workgroups, 256, 0, s, a)
                                : launch(linear_step<float>, workgroups, 256, 0, s, a);
  }
  LinArgs a = common(p, c, p.seg, p.segs);
  a.runs = 1;
  a.run[0] = LinRun{c.q.p, c.k.p, c.v.p, c.o.p, c.q.batch, c.q.row, c.k.batch, c.k.row, c.v.batch, c.v.row, c.o.batch,
                    c.o.row, d.heads / d.q_heads, d.heads / d.k_heads, d.heads / d.v_heads, d.dk, d.dv, d.dv, 1, 0, 0, 1,
                    0, d.scale, d.scale, 1.f, c.h_in, c.h_out, static_cast<float*>(c.workspace), 0};
  const int pad = linear_pad(d.dk);
  if (a.segs > 1) {
    int e = run(a, d, pad, false, false, s);
    if (e) return e;
    JoinArgs j = join_of(a, int64_t(d.dk) * d.dv);
    j.way[0] = {c.h_in, a.run[0].segs, nullptr};
    if ((e = start_join(j, 1, s))) return e;
  }
  return run(a, d, pad, true, false, s);
}

int launch_linear_backward(const cc3d_linear_plan& p, const cc3d_linear_args_t& c, void* stream) {
  const auto& d = p.d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LinearSpace space = linear_bwd_space(p);
  float* w = static_cast<float*>(c.workspace);
  float* states = w;
  float* states2 = states + space.state;
  float* grads = states2 + space.state;
  float* part_q = grads + space.state;
  float* part_k = part_q + space.dq;
  float* part_v = part_k + space.dk;
  double* decay = reinterpret_cast<double*>(part_v + space.dv);
  const int qper = d.heads / d.q_heads, kper = d.heads / d.k_heads, vper = d.heads / d.v_heads;
  const int pad = linear_pad(std::max(d.dk, d.dv));
  // results go to the caller's view, or where heads are shared to partial sums [N][T][heads][D]
  auto out = [&](LinRun r, const cc3d_rows_t& v, int per, float* part) {
    r.o = per == 1 ? v.p : part;
    r.o_f32 = per > 1;
    r.ob = per == 1 ? v.batch : int64_t(d.t) * d.heads * r.e;
    r.orow = per == 1 ? v.row : int64_t(d.heads) * r.e;
    return r;
  };
  // dq: the recurrence of (do, v, k) over the transposed state; dk and dv: of (v, do, q) and (k, q, do), reversed
  const LinRun rq = out(LinRun{c.grad_o.p, c.v.p, c.k.p, nullptr, c.grad_o.batch, c.grad_o.row, c.v.batch, c.v.row,
                               c.k.batch, c.k.row, 0, 0, 1, vper, kper, d.dv, d.dk, 1, d.dv, 0, 0, 1, 0, d.scale, d.scale,
                               1.f, c.h_in, nullptr, states, 0}, c.dq, qper, part_q);
  const LinRun rk = out(LinRun{c.v.p, c.grad_o.p, c.q.p, nullptr, c.v.batch, c.v.row, c.grad_o.batch, c.grad_o.row,
                               c.q.batch, c.q.row, 0, 0, vper, 1, qper, d.dv, d.dk, 1, d.dv, 0, 1, 0, 0, d.scale, 1.f,
                               d.scale, c.dh_out, nullptr, grads, 0}, c.dk, kper, part_k);
  const LinRun rv = out(LinRun{c.k.p, c.q.p, c.grad_o.p, nullptr, c.k.batch, c.k.row, c.q.batch, c.q.row, c.grad_o.batch,
                               c.grad_o.row, 0, 0, kper, qper, 1, d.dk, d.dv, d.dv, 1, 0, 1, 0, 0, d.scale, 1.f, d.scale,
                               c.dh_out, c.dh_in, grads, 0}, c.dv, vper, part_v);
  LinArgs a = common(p, c, p.bwd_seg, p.bwd_segs);
  a.segs2 = states2;
  a.x = c.q.p;
  a.xb = c.q.batch;
  a.xr = c.q.row;
  a.xper = qper;
  a.dto = c.dh_out;
  a.part = decay;
  const bool dec = c.dlog_decay, back = c.dk.p || c.dv.p || c.dh_in;
  int e = 0;
  if (a.segs > 1) {
    JoinArgs j = join_of(a, int64_t(d.dk) * d.dv);
    int ways = 0;
    if (dec || c.dq.p) {
      a.runs = 1;
      a.run[0] = rq;
      if ((e = run(a, d, pad, false, dec, s))) return e;
      j.way[ways++] = {c.h_in, states, dec ? states2 : nullptr};
    }
    if (back) {
      a.runs = 1;
      a.run[0] = rv;
      if ((e = run(a, d, pad, false, false, s))) return e;
      j.way[ways++] = {c.dh_out, grads, nullptr};
    }
    if (ways && (e = start_join(j, ways, s))) return e;
  }
  if (dec) {
    a.runs = 1;
    a.run[0] = rq;
    if ((e = run(a, d, pad, true, true, s))) return e;
    e = launch(linear_decay, d.heads, 256, 0, s, decay, c.dlog_decay, d.n, d.heads, a.segs * a.run[0].blocks);
    if (e) return e;
  }
  a.runs = 0;
  if (c.dq.p) a.run[a.runs++] = rq;
  if (c.dk.p) a.run[a.runs++] = rk;
  if (c.dv.p || c.dh_in) a.run[a.runs++] = rv;
  if (a.runs && (e = run(a, d, pad, true, false, s))) return e;
  HeadSums sums{};
  int jobs = 0;
  int64_t most = 0;
  auto add = [&](const cc3d_rows_t& v, int per, const float* part, int heads, int width) {
    if (!v.p || per == 1) return;
    const int64_t el = int64_t(d.n) * d.t * heads * width;
    sums.job[jobs++] = HeadSum{part, v.p, v.batch, v.row, el, per, width, d.t, heads};
    most = std::max(most, el);
  };
  add(c.dq, qper, part_q, d.q_heads, d.dk);
  add(c.dk, kper, part_k, d.k_heads, d.dk);
  add(c.dv, vper, part_v, d.v_heads, d.dv);
  if (jobs) {
    void* at[] = {&sums};
    const void* kernel = d.dtype == CC3D_BF16 ? reinterpret_cast<const void*>(&linear_heads<bf16_s>)
                                              : reinterpret_cast<const void*>(&linear_heads<float>);
    const hipError_t err = hipLaunchKernel(kernel, dim3(unsigned(std::min((most + 255) / 256, kGrid)), unsigned(jobs)),
                                           dim3(256), at, 0, s);
    if (err != hipSuccess) (void)hipGetLastError();
    return int(err);
  }
  return 0;
}

}  // namespace cc3d
