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
#include "cc3d_seq_scan.h"

namespace {

template <class T, int NS, bool MULTI>
__global__ __launch_bounds__(MULTI ? 64 * (cc3d::kScanMaxStates / NS) : 64) void scan_fwd(ScanArgs a) {
  constexpr int kWaves = MULTI ? cc3d::kScanMaxStates / NS : 1;
  __shared__ __attribute__((aligned(16))) float box_all[kWaves][2 * 4 * NS];
  __shared__ float part[MULTI ? 2 : 1][kWaves][MULTI ? 4 : 1][64];
  const Place at(a);
  float* box = box_all[at.wave];
  const int n = int(at.item / a.chunks), ch = int(at.item - int64_t(n) * a.chunks);
  const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
  const int s0 = at.wave * NS, states = min(a.s - s0, NS);
  const int channels = a.groups * a.wide;
  const T *bp = rows<T>(a.b, n) + at.group * a.s + s0, *cp = rows<T>(a.c, n) + at.group * a.s + s0;
  const T *dt = rows<T>(a.dt, n), *u = rows<T>(a.u, n), *z = a.z.p ? rows<T>(a.z, n) : nullptr;
  T* y = out_rows<T>(a.y, n);
  const float bias = a.bias ? a.bias[at.chan] : 0.f, skip = a.d ? a.d[at.chan] : 0.f;
  const int64_t state_at = (int64_t(n) * channels + at.chan) * a.s + s0;

  float h[NS], a2[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    a2[i] = i < states ? a.a[int64_t(at.chan) * a.s + s0 + i] * kLog2e : 0.f;
    h[i] = 0.f;
    if (i < states) {
      if (a.chunks > 1) h[i] = a.carry[(at.item * a.s + s0 + i) * channels + at.chan];
      else if (a.h_in) h[i] = a.h_in[state_at + i];
    }
  }

  Feed<T, NS, 2> next;
  auto fetch = [&](int tb) {
    feed(next, tb, te, dt, a.dt.row, u, a.u.row, z, a.z.row, bp, a.b.row, cp, a.c.row, states, at.lane, at.chan);
  };
  if (t0 < te) fetch(t0);
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
    if (tb + 4 < te) fetch(tb + 4);
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
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (MULTI && j % a.waves != at.wave) continue;
      if (MULTI) {
        sum[j] = 0.f;
        for (int w = 0; w < a.waves; ++w) sum[j] += part[turn][w][j][at.lane];
      }
      const int t = tb + j;
      if (t < te && at.on) {
        float v = fmaf(skip, uu[j], sum[j]);
        if (z) {
          const float g = to_f32(zz[j]);
          v *= g * sigmoid_f32(g);
        }
        (y + int64_t(t) * a.y.row)[at.chan] = from_f32<T>(v);
      }
    }
    turn ^= 1;
  }
  if (!at.on) return;
  if (at.wave == 0)
    for (int t = max(t0, te); t < t1; ++t) (y + int64_t(t) * a.y.row)[at.chan] = from_f32<T>(0.f);
  if (a.h_out && ch == a.chunks - 1) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < states) a.h_out[state_at + i] = h[i];
  }
}

// One token: the states are read and written once and little else is moved.
// A lane holds four states of one channel, so a channel's states are one
// stretch of memory across LP lanes, and its sum over states LP lanes wide.
template <class T, int LP, bool VEC>
__global__ __launch_bounds__(256) void scan_step(ScanArgs a) {
  const int64_t id = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LP;
  const int part = threadIdx.x % LP;
  const int channels = a.groups * a.wide;
  const bool on = id < int64_t(a.n) * channels;  // the same for a channel's LP lanes; all take part in the sum
  const int n = on ? int(id / channels) : 0, chan = on ? int(id - int64_t(n) * channels) : 0;
  const int s0 = part * 4, left = a.s - s0;  // may be negative
  const int64_t state_at = (int64_t(n) * channels + chan) * a.s + s0;
  const int group = chan / a.wide;
  const bool valid = valid_tokens(a, n) > 0;
  float h[4] = {}, sum = 0.f, uu = 0.f;
  if (a.h_in && left > 0) {
    if constexpr (VEC) {
      const f32x4_s v = *reinterpret_cast<const f32x4_s*>(a.h_in + state_at);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) h[i] = a.h_in[state_at + i];
    }
  }
  if (valid) {
    const float bias = a.bias ? a.bias[chan] : 0.f;
    const float delta = delta_of(a, to_f32(rows<T>(a.dt, n)[chan]) + bias);
    uu = to_f32(rows<T>(a.u, n)[chan]);
    const float du = delta * uu;
    const T *b = rows<T>(a.b, n) + group * a.s + s0, *c = rows<T>(a.c, n) + group * a.s + s0;
    const float* aa = a.a + int64_t(chan) * a.s + s0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        h[i] = fmaf(__builtin_amdgcn_exp2f(delta * (aa[i] * kLog2e)), h[i], du * to_f32(b[i]));
        sum = fmaf(h[i], to_f32(c[i]), sum);
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
        const float g = to_f32(rows<T>(a.z, n)[chan]);
        v *= g * sigmoid_f32(g);
      }
    }
    out_rows<T>(a.y, n)[chan] = from_f32<T>(v);
  }
}

template <class T, int LP>
int run_step(const ScanArgs& a, hipStream_t s) {
  const int64_t threads = int64_t(a.n) * a.groups * a.wide * LP;
  const unsigned blocks = unsigned((threads + 255) / 256);
  if (a.s % 4 == 0 && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0 && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0)
    scan_step<T, LP, true><<<blocks, 256, 0, s>>>(a);
  else
    scan_step<T, LP, false><<<blocks, 256, 0, s>>>(a);
  return int(hipGetLastError());
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
  const unsigned blocks = unsigned(tiles * a.n * a.chunks);
  if (a.chunks > 1) {
    scan_carry<T, NS, false><<<blocks, 64 * a.waves, 0, s>>>(a);
    int e = int(hipGetLastError());
    if (e) return e;
    scan_join<false><<<join_blocks(p.d), 256, 0, s>>>(a);
    e = int(hipGetLastError());
    if (e) return e;
  }
  if (a.waves > 1) scan_fwd<T, NS, true><<<blocks, 64 * a.waves, 0, s>>>(a);
  else scan_fwd<T, NS, false><<<blocks, 64, 0, s>>>(a);
  return int(hipGetLastError());
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
