// Shared by the scan's forward and backward kernel files: the kernel
// argument block, the workgroup's place, and the passes that carry the state
// across chunks of the time axis.
#pragma once
#include "cc3d_seq_device.h"

namespace {

struct ScanRows {
  void* p;
  int64_t batch, row;
};

struct ScanArgs {
  ScanRows u, dt, b, c, z, y, dy, du, ddt, dz;
  const float *a, *d, *bias, *h_in, *dh_out;
  float *h_out, *dh_in;
  const int* lengths;
  float* carry;    // [n][chunk][S][C]: the state that a chunk adds, then the state that enters it
  float* gcarry;   // the same of the gradient, which enters from the right
  float* sums;     // [n][chunk][C]: sum of delta over the chunk
  float* part_a;   // backward partial sums: [worker][C][S]
  float* part_d;   // [worker * waves][C]
  float* part_bias;
  float* part_bc;  // [tile][n][t][waves][2][states of a wave]
  int n, t, ch, s, groups, wide;  // wide: channels of a group
  int tiles_per_group, chunk, chunks, waves, workers;
  int softplus;
};

// A wave holds 64 channels of one group; blockIdx.x = tile + tiles * item.
struct Place {
  int lane, wave, tile, group, chan;
  bool on;
  int64_t item;
  __device__ __forceinline__ Place(const ScanArgs& a) {
    lane = threadIdx.x % 64;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tiles = a.tiles_per_group * a.groups;
    tile = blockIdx.x % tiles;
    item = blockIdx.x / tiles;
    group = tile / a.tiles_per_group;
    const int in_group = (tile - group * a.tiles_per_group) * 64 + lane;
    on = in_group < a.wide;
    chan = group * a.wide + (on ? in_group : 0);
  }
};

__device__ __forceinline__ int valid_tokens(const ScanArgs& a, int n) {
  return a.lengths ? min(max(a.lengths[n], 0), a.t) : a.t;
}

template <class T>
__device__ __forceinline__ const T* rows(const ScanRows& v, int n) {
  return static_cast<const T*>(v.p) + int64_t(n) * v.batch;
}

template <class T>
__device__ __forceinline__ T* out_rows(const ScanRows& v, int n) {
  return static_cast<T*>(v.p) + int64_t(n) * v.batch;
}

__device__ __forceinline__ float delta_of(const ScanArgs& a, float raw) {
  return a.softplus ? softplus_f32(raw) : raw;
}

// Orders a wave's own LDS writes before its lanes' reads of each other's.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a chunk adds to the state, starting from zero: the forward recurrence
//   h = exp(delta A) h + delta u B
// or, REV, the gradient's from the chunk's last token back,
//   g = exp(delta A) (g + gy C),  gy = dy silu(z),
// and the chunk's sum of delta, whose exponential is the whole chunk's decay.
template <class T, int NS, bool REV>
__global__ __launch_bounds__(64 * (cc3d::kScanMaxStates / NS)) void scan_carry(ScanArgs a) {
  __shared__ __attribute__((aligned(16))) float box[cc3d::kScanMaxStates / NS][4 * NS];
  const Place at(a);
  const int n = int(at.item / a.chunks), ch = int(at.item - int64_t(n) * a.chunks);
  const int t0 = ch * a.chunk, te = min(min(t0 + a.chunk, a.t), valid_tokens(a, n));
  const int s0 = at.wave * NS;
  const ScanRows& coef = REV ? a.c : a.b;
  const T* cf = rows<T>(coef, n) + at.group * a.s;
  const T* dt = rows<T>(a.dt, n) + at.chan;
  const T* xin = rows<T>(REV ? a.dy : a.u, n) + at.chan;
  const T* zin = REV && a.z.p ? rows<T>(a.z, n) + at.chan : nullptr;
  const float bias = a.bias ? a.bias[at.chan] : 0.f;
  float h[NS], a2[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    h[i] = 0.f;
    a2[i] = s0 + i < a.s ? a.a[int64_t(at.chan) * a.s + s0 + i] * kLog2e : 0.f;
  }
  float total = 0.f;
  const int groups = te > t0 ? (te - t0 + 3) / 4 : 0;
  for (int q = 0; q < groups; ++q) {
    const int tb = t0 + 4 * (REV ? groups - 1 - q : q);
    wave_fence();
    for (int i = at.lane; i < 4 * NS; i += 64) {
      const int t = tb + i / NS, s = s0 + i % NS;
      box[at.wave][i] = t < te && s < a.s ? to_f32(cf[int64_t(t) * coef.row + s]) : 0.f;
    }
    float delta[4], x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = tb + j;
      delta[j] = x[j] = 0.f;
      if (t < te) {
        delta[j] = delta_of(a, to_f32(dt[int64_t(t) * a.dt.row]) + bias);
        x[j] = to_f32(xin[int64_t(t) * (REV ? a.dy.row : a.u.row)]);
        if (!REV) x[j] *= delta[j];
        if (REV && zin) {
          const float z = to_f32(zin[int64_t(t) * a.z.row]);
          x[j] *= z * sigmoid_f32(z);
        }
      }
      total += delta[j];
    }
    wave_fence();
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = REV ? 3 - jj : jj;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float decay = __builtin_amdgcn_exp2f(delta[j] * a2[i]), add = x[j] * box[at.wave][j * NS + i];
        h[i] = REV ? decay * (h[i] + add) : fmaf(decay, h[i], add);
      }
    }
  }
  if (!at.on) return;
  const int channels = a.groups * a.wide;
  float* out = (REV ? a.gcarry : a.carry) + (at.item * a.s + s0) * channels + at.chan;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (s0 + i < a.s) out[int64_t(i) * channels] = h[i];
  if (!REV && at.wave == 0) a.sums[at.item * channels + at.chan] = total;
}

// Turns what every chunk adds into the state that enters it, from the
// sequence's first state on (REV: the gradient that enters it from the right).
template <bool REV>
__global__ __launch_bounds__(256) void scan_join(ScanArgs a) {
  const int channels = a.groups * a.wide;
  const int tiles = (channels + 63) / 64;
  // blockIdx.x = (n * ceil(S / 4) + states / 4) * tiles + tile
  const int tile = blockIdx.x % tiles;
  const int per = (a.s + 3) / 4;
  const int64_t rest = blockIdx.x / tiles;
  const int n = int(rest / per), s = int(rest - int64_t(n) * per) * 4 + threadIdx.x / 64;
  const int chan = tile * 64 + threadIdx.x % 64;
  if (chan >= channels || s >= a.s) return;
  const float a2 = a.a[int64_t(chan) * a.s + s] * kLog2e;
  const float* first = REV ? a.dh_out : a.h_in;
  float h = first ? first[(int64_t(n) * channels + chan) * a.s + s] : 0.f;
  float* carry = (REV ? a.gcarry : a.carry) + (int64_t(n) * a.chunks * a.s + s) * channels + chan;
  const float* sums = a.sums + int64_t(n) * a.chunks * channels + chan;
  const int64_t step = int64_t(a.s) * channels;
  for (int c0 = 0; c0 < a.chunks; c0 += 8) {
    float add[8], sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = REV ? a.chunks - 1 - (c0 + i) : c0 + i;
      const bool in = c0 + i < a.chunks;
      add[i] = in ? carry[c * step] : 0.f;
      sum[i] = in ? sums[int64_t(c) * channels] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = REV ? a.chunks - 1 - (c0 + i) : c0 + i;
      if (c0 + i < a.chunks) carry[c * step] = h;
      h = fmaf(__builtin_amdgcn_exp2f(sum[i] * a2), h, add[i]);
    }
  }
}

inline ScanRows view_of(const cc3d_rows_t& v) { return {v.p, v.batch, v.row}; }

inline ScanArgs scan_args(const cc3d_scan_plan& p, const cc3d_scan_args_t& c) {
  ScanArgs a{};
  a.u = view_of(c.u);
  a.dt = view_of(c.dt);
  a.b = view_of(c.b);
  a.c = view_of(c.c);
  a.z = view_of(c.z);
  a.a = c.a;
  a.d = c.d;
  a.bias = c.dt_bias;
  a.h_in = c.h_in;
  a.lengths = c.lengths;
  a.n = p.d.n;
  a.t = p.d.t;
  a.s = p.d.states;
  a.groups = p.d.groups;
  a.wide = p.d.d / p.d.groups;
  a.tiles_per_group = cc3d::scan_tiles_per_group(p.d);
  a.softplus = p.d.softplus;
  return a;
}

inline unsigned join_blocks(const cc3d_scan_desc_t& d) {
  return unsigned(int64_t(d.n) * ((d.states + 3) / 4) * ((d.d + 63) / 64));
}

}  // namespace
