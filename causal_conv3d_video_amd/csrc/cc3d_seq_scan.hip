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
  __shared__ __attribute__((aligned(16))) float box[kWaves][2][4 * NS];
  __shared__ float part[MULTI ? 2 : 1][kWaves][MULTI ? 4 : 1][64];
  const Place at(a);
  const int n = int(at.item / a.chunks), ch = int(at.item - int64_t(n) * a.chunks);
  const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
  const int s0 = at.wave * NS;
  const int channels = a.groups * a.wide;
  const T* bp = rows<T>(a.b, n) + at.group * a.s;
  const T* cp = rows<T>(a.c, n) + at.group * a.s;
  const T* dt = rows<T>(a.dt, n) + at.chan;
  const T* u = rows<T>(a.u, n) + at.chan;
  const T* z = a.z.p ? rows<T>(a.z, n) + at.chan : nullptr;
  T* y = out_rows<T>(a.y, n) + at.chan;
  const float bias = a.bias ? a.bias[at.chan] : 0.f, skip = a.d ? a.d[at.chan] : 0.f;
  const int64_t state_at = (int64_t(n) * channels + at.chan) * a.s + s0;

  float h[NS], a2[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const bool in = s0 + i < a.s;
    a2[i] = in ? a.a[int64_t(at.chan) * a.s + s0 + i] * kLog2e : 0.f;
    h[i] = 0.f;
    if (in) {
      if (a.chunks > 1) h[i] = a.carry[(at.item * a.s + s0 + i) * channels + at.chan];
      else if (a.h_in) h[i] = a.h_in[state_at + i];
    }
  }

  int turn = 0;
  for (int tb = t0; tb < te; tb += 4) {
    wave_fence();
    for (int i = at.lane; i < 4 * NS; i += 64) {
      const int t = tb + i / NS, s = s0 + i % NS;
      const bool in = t < te && s < a.s;
      box[at.wave][0][i] = in ? to_f32(bp[int64_t(t) * a.b.row + s]) : 0.f;
      box[at.wave][1][i] = in ? to_f32(cp[int64_t(t) * a.c.row + s]) : 0.f;
    }
    float delta[4], du[4], uu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = tb + j;
      delta[j] = uu[j] = 0.f;
      if (t < te) {
        delta[j] = delta_of(a, to_f32(dt[int64_t(t) * a.dt.row]) + bias);
        uu[j] = to_f32(u[int64_t(t) * a.u.row]);
      }
      du[j] = delta[j] * uu[j];
    }
    wave_fence();
    float sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[j] = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float decay = __builtin_amdgcn_exp2f(delta[j] * a2[i]);
        h[i] = fmaf(decay, h[i], du[j] * box[at.wave][0][j * NS + i]);
        sum[j] = fmaf(h[i], box[at.wave][1][j * NS + i], sum[j]);
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
          const float zz = to_f32(z[int64_t(t) * a.z.row]);
          v *= zz * sigmoid_f32(zz);
        }
        y[int64_t(t) * a.y.row] = from_f32<T>(v);
      }
    }
    turn ^= 1;
  }
  if (!at.on) return;
  if (at.wave == 0)
    for (int t = max(t0, te); t < t1; ++t) y[int64_t(t) * a.y.row] = from_f32<T>(0.f);
  if (a.h_out && ch == a.chunks - 1) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (s0 + i < a.s) a.h_out[state_at + i] = h[i];
  }
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
