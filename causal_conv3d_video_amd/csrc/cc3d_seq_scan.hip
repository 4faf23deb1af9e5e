// Selective state space scan, forward.
//
//   delta = softplus(dt + dt_bias);  h = exp(delta A) h + delta u B
//   y = (sum_s C_s h_s + D u) silu(z)
//
// One exponential and four multiply-adds a channel, token and state against
// four elements moved a channel and token: with 16 states the vector units
// bound it, not memory.  A lane owns one channel with 16 of its states in
// registers (more states: more waves, whose sums over states meet in LDS), so
// the sum over states needs no exchange between lanes, and B and C, shared by
// the channels of a group, are read back from LDS as broadcasts.  Tokens are
// taken four at a time, the next four loading meanwhile.  Where the channels
// alone leave SIMDs idle the time axis is split into chunks: a first pass
// finds what each chunk adds to the state and its decay, exp(A sum delta), a
// small one joins them, and the main pass starts each chunk from its state.
//
// Measured, bf16, 16 states: 8192 tokens of 2048 channels in 126 us (in a kernel
// trace, whose durations add up to more than the pass: 54 for the chunks' sums, 9
// for the join, 73 for the main pass).  The vector units are busy 83% of the main
// pass, with 123 instructions a channel and token; the bytes alone would take 28
// at a large copy's 4.74 TB/s.  1560 ragged sequences of up to 17 tokens of 768
// channels take one pass, 83 us, vector units busy 65%; the nominal bytes, 67.
#include "cc3d_seq_scan.h"

namespace {

template <class T, int NS, bool MULTI>
__global__ __launch_bounds__(MULTI ? 64 * (cc3d::kScanMaxStates / NS) : 64) void scan_fwd(ScanArgs a) {
  constexpr int kWaves = MULTI ? cc3d::kScanMaxStates / NS : 1;
  __shared__ __attribute__((aligned(16))) float box_all[kWaves][StateBox<NS>::kSize];
  __shared__ float part[MULTI ? 2 : 1][kWaves][MULTI ? 4 : 1][64];
  const Place at(a);
  float* box = box_all[at.wave];
  const int n = int(at.item / a.chunks), ch = int(at.item - int64_t(n) * a.chunks);
  const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
  const int s0 = at.wave * NS, states = min(a.s - s0, NS);
  const int channels = a.groups * a.wide;
  const float bias = a.bias ? a.bias[at.chan] : 0.f, skip = a.d ? a.d[at.chan] : 0.f;
  const int64_t state_at = (int64_t(n) * channels + at.first) * a.s + s0;

  Stream<T> dt(a.dt, n, t0, at.chan), u(a.u, n, t0, at.chan), z(a.z, n, t0, at.chan), y(a.y, n, t0, at.chan);
  Stream<T> bs(a.b, n, t0, 0), cs(a.c, n, t0, 0);
  bs.p += at.group * a.s + s0;
  cs.p += at.group * a.s + s0;
  Feed<T, NS, 2> next;
  if (t0 < te) feed(next, te - t0, dt, u, z, bs, cs, states, at.lane);

  float h[NS] = {}, a2[NS];
  load_states<NS>(a.a + int64_t(at.first) * a.s + s0, a.s, states, at.live, at.lane, box, a2);
#pragma unroll
  for (int i = 0; i < NS; ++i) a2[i] = rate_of(a2[i]);
  if (a.chunks > 1) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < states) h[i] = a.carry[(at.item * a.s + s0 + i) * channels + at.chan];
  } else if (a.h_in) {
    load_states<NS>(a.h_in + state_at, a.s, states, at.live, at.lane, box, h);
  }

  int turn = 0;
  for (int tb = t0; tb < te; tb += 4) {
    wave_fence();
    spread_rows(next, box, tb, te, states, at.lane);
    float delta[4], uu[4];
    T zz[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      delta[j] = tb + j < te ? delta_of(a, to_f32(next.dt[j]) + bias) : 0.f;
      uu[j] = tb + j < te ? to_f32(next.x[j]) : 0.f;
      zz[j] = next.z[j];
    }
    wave_fence();
    if (tb + 4 < te) {
      dt.move(1);
      u.move(1);
      z.move(z.p ? 1 : 0);
      bs.move(1);
      cs.move(1);
      feed(next, te - tb - 4, dt, u, z, bs, cs, states, at.lane);
    }
    float sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float du = delta[j] * uu[j];
      sum[j] = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float decay = __builtin_amdgcn_exp2f(delta[j] * a2[i]);
        h[i] = fmaf(decay, h[i], du * box[j * NS + i]);
        sum[j] = fmaf(h[i], box[(4 + j) * NS + i], sum[j]);
      }
    }
    if (MULTI) {
#pragma unroll
      for (int j = 0; j < 4; ++j) part[turn][at.wave][j][at.lane] = sum[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[j] = 0.f;
        if (j % a.waves == at.wave)
          for (int w = 0; w < a.waves; ++w) sum[j] += part[turn][w][j][at.lane];
      }
      turn ^= 1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fmaf(skip, uu[j], sum[j]);
    if (z.p) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = to_f32(zz[j]);
        sum[j] *= g * sigmoid_f32(g);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tb + j < te && (!MULTI || j % a.waves == at.wave)) y.p[y.off[j]] = from_f32<T>(sum[j]);
    y.move(1);
  }
  if (at.wave == 0) {
    T* out = out_rows<T>(a.y, n) + at.chan;
    for (int t = max(t0, te); t < t1; ++t) out[int64_t(t) * a.y.row] = from_f32<T>(0.f);
  }
  if (a.h_out && ch == a.chunks - 1) store_states<NS>(a.h_out + state_at, a.s, states, at.live, at.lane, box, h);
}

// One token: the states are read and written once and little else is moved.
// A lane holds four states of one channel, so a channel's states are one
// stretch of memory across LP lanes, and its sum over states LP lanes wide.
// VEC: states and rows of B and C are aligned to four.
// 256 streams of 768 channels, 16 states: 7.7 us, 3.5 TB/s of states and inputs,
// vector units busy 17%.  As one more token of scan_fwd the call took 35 us, with
// this kernel 10 (of which the host is a part).
template <class T, int LP, bool VEC>
__global__ __launch_bounds__(256) void scan_step(ScanArgs a, unsigned per_sequence) {
  const unsigned n = blockIdx.x / per_sequence;
  const int at = int((blockIdx.x - n * per_sequence) * (256 / LP) + threadIdx.x / LP);
  const int part = threadIdx.x % LP;
  const int channels = a.groups * a.wide;
  const bool on = at < channels;  // the same for a channel's LP lanes; all take part in the sum
  const int chan = on ? at : channels - 1;
  const int s0 = part * 4, left = a.s - s0;  // may be negative
  const int64_t state_at = (int64_t(n) * channels + chan) * a.s + s0;
  const int group = a.groups == 1 ? 0 : chan / a.wide;
  float h[4] = {}, sum = 0.f, uu = 0.f;
  const bool valid = valid_tokens(a, int(n)) > 0;
  if (left > 0) {
    // (a row of B or C may hold more than 2^31 elements here; with more tokens the plan's limits keep it below)
    const int64_t bc_at = int64_t(group) * a.s + s0;
    const T *b = rows<T>(a.b, int(n)) + bc_at, *c = rows<T>(a.c, int(n)) + bc_at;
    const float* aa = a.a + int64_t(chan) * a.s + s0;
    float a4[4] = {}, b4[4] = {}, c4[4] = {};
    if constexpr (VEC) {
      using U = std::conditional_t<sizeof(T) == 4, f32x4_s, unsigned long long>;
      const f32x4_s va = *reinterpret_cast<const f32x4_s*>(aa);
      f32x4_s vh{0.f, 0.f, 0.f, 0.f};
      if (a.h_in) vh = *reinterpret_cast<const f32x4_s*>(a.h_in + state_at);
      U vb{}, vc{};
      if (valid) {
        vb = *reinterpret_cast<const U*>(b);
        vc = *reinterpret_cast<const U*>(c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = vh[i];
        a4[i] = va[i];
        if constexpr (sizeof(T) == 4) {
          b4[i] = vb[i];
          c4[i] = vc[i];
        } else {
          b4[i] = to_f32(bf16_s(vb >> (16 * i)));
          c4[i] = to_f32(bf16_s(vc >> (16 * i)));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) {
          if (a.h_in) h[i] = a.h_in[state_at + i];
          a4[i] = aa[i];
          b4[i] = valid ? to_f32(b[i]) : 0.f;
          c4[i] = valid ? to_f32(c[i]) : 0.f;
        }
    }
    if (valid) {
      const float delta = delta_of(a, to_f32(rows<T>(a.dt, int(n))[chan]) + (a.bias ? a.bias[chan] : 0.f));
      uu = to_f32(rows<T>(a.u, int(n))[chan]);
      const float du = delta * uu;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (VEC || i < left) {
          h[i] = fmaf(__builtin_amdgcn_exp2f(delta * (a4[i] * kLog2e)), h[i], du * b4[i]);
          sum = fmaf(h[i], c4[i], sum);
        }
    }
  }
  sum = group_sum<LP>(sum);
  if (!on) return;
  if (a.h_out && left > 0) {
    if constexpr (VEC) {
      *reinterpret_cast<f32x4_s*>(a.h_out + state_at) = f32x4_s{h[0], h[1], h[2], h[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) a.h_out[state_at + i] = h[i];
    }
  }
  if (part == 0) {
    float v = 0.f;
    if (valid) {
      v = a.d ? fmaf(a.d[chan], uu, sum) : sum;
      if (a.z.p) {
        const float g = to_f32(rows<T>(a.z, int(n))[chan]);
        v *= g * sigmoid_f32(g);
      }
    }
    out_rows<T>(a.y, int(n))[chan] = from_f32<T>(v);
  }
}

template <class T, int LP>
int run_step(const ScanArgs& a, hipStream_t s) {
  const unsigned per_sequence = unsigned((int64_t(a.groups) * a.wide * LP + 255) / 256);
  bool vec = a.s % 4 == 0;
  for (const void* p : {static_cast<const void*>(a.a), static_cast<const void*>(a.h_in), static_cast<const void*>(a.h_out)})
    vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  for (const ScanRows* v : {&a.b, &a.c})
    vec = vec && reinterpret_cast<uintptr_t>(v->p) % (4 * sizeof(T)) == 0 && (a.n == 1 || v->batch % 4 == 0);
  return launch(vec ? scan_step<T, LP, true> : scan_step<T, LP, false>, int64_t(per_sequence) * a.n, 256, 0, s, a, per_sequence);
}

template <class T>
int pick_step(const ScanArgs& a, hipStream_t s) {
  if (a.s <= 4) return run_step<T, 1>(a, s);
  if (a.s <= 8) return run_step<T, 2>(a, s);
  if (a.s <= 16) return run_step<T, 4>(a, s);
  if (a.s <= 32) return run_step<T, 8>(a, s);
  return run_step<T, 16>(a, s);
}

template <class T, int NS>
int run_scan(const cc3d_scan_plan& p, ScanArgs& a, hipStream_t s) {
  a.waves = cc3d::scan_fwd_waves(p.d);
  const int64_t tiles = int64_t(a.groups) * a.tiles_per_group;
  if (a.chunks > 1) {
    int e = run_carry<T, NS, false>(a, s);
    if (e) return e;
    e = run_join(a, false, s);
    if (e) return e;
  }
  const int64_t blocks = tiles * a.n * a.chunks;
  if constexpr (NS == cc3d::kScanFwdStates)  // (fewer a wave: all of them in one)
    if (a.waves > 1) return launch(scan_fwd<T, NS, true>, blocks, 64 * a.waves, 0, s, a);
  return launch(scan_fwd<T, NS, false>, blocks, 64, 0, s, a);
}

template <class T>
int pick_states(const cc3d_scan_plan& p, ScanArgs& a, hipStream_t s) {
  if (a.t == 1) return pick_step<T>(a, s);
  switch (cc3d::scan_fwd_ns(p.d)) {
    case 4: return run_scan<T, 4>(p, a, s);
    case 8: return run_scan<T, 8>(p, a, s);
    default: return run_scan<T, 16>(p, a, s);
  }
}

}  // namespace

namespace cc3d {

int launch_scan_forward(const cc3d_scan_plan& p, const cc3d_scan_args_t& c, void* stream) {
  ScanArgs a = scan_args(p, c);
  a.y = view_of(c.y);
  a.h_out = c.h_out;
  a.chunk = p.chunk;
  a.chunks = p.info.chunks;
  const int64_t state = int64_t(p.d.n) * a.chunks * p.d.states * p.d.d;
  a.carry = static_cast<float*>(c.workspace);
  a.sums = a.carry + state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p.d.dtype == CC3D_BF16 ? pick_states<bf16_s>(p, a, s) : pick_states<float>(p, a, s);
}

}  // namespace cc3d
