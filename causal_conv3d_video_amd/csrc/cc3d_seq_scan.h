// Shared by the scan's forward and backward kernel files: the kernel
// argument block, the workgroup's place, and the passes that carry the state
// across chunks of the time axis.
#pragma once
#include "cc3d_seq_device.h"

#include <algorithm>
#include <cfloat>

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
  int first, live;  // the wave's first channel and how many it has
  int64_t item;
  __device__ __forceinline__ Place(const ScanArgs& a) {
    lane = threadIdx.x % 64;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int tiles = a.tiles_per_group * a.groups;
    tile = blockIdx.x % tiles;
    item = blockIdx.x / tiles;
    group = tile / a.tiles_per_group;
    const int in_group = (tile - group * a.tiles_per_group) * 64 + lane;
    // lanes past the group's last channel compute that one too: what they
    // store is the same value to the same place
    chan = group * a.wide + min(in_group, a.wide - 1);
    first = group * a.wide + in_group - lane;
    live = min(a.wide - (in_group - lane), 64);
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

// A as the exponent of two of a step of one.  A state that is forgotten at once,
// A = -inf, has the lowest finite one instead: past a sequence's last token
// steps are zero, and zero times it has to leave the state as it is.
__device__ __forceinline__ float rate_of(float a) {
  const float r = a * kLog2e;
  return r < -FLT_MAX ? -FLT_MAX : r;
}

// Orders a wave's own LDS writes before its lanes' reads of each other's.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's states [64 channels][NS] of a tensor [C][S], each lane its channel:
// read and written as whole stretches of memory and turned through LDS (rows
// padded by 16 bytes), not as 64 rows at once.
template <int NS>
struct StateBox {
  static constexpr int kRow = NS + 4, kSize = 64 * kRow;
};

template <int NS>
__device__ __forceinline__ void load_states(const float* p, int row, int states, int live, int lane, float* box, float (&v)[NS]) {
  using B = StateBox<NS>;
  wave_fence();
  if (row % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
    for (int k = 0; k < NS / 4; ++k) {
      const int i = lane + 64 * k, c = i / (NS / 4), s = i % (NS / 4) * 4;
      f32x4_s x{0.f, 0.f, 0.f, 0.f};
      if (c < live && s < states) x = *reinterpret_cast<const f32x4_s*>(p + int64_t(c) * row + s);
      *reinterpret_cast<f32x4_s*>(box + c * B::kRow + s) = x;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int i = lane + 64 * k, c = i / NS, s = i % NS;
      box[c * B::kRow + s] = c < live && s < states ? p[int64_t(c) * row + s] : 0.f;
    }
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = box[min(lane, live - 1) * B::kRow + i];
  wave_fence();
}

template <int NS>
__device__ __forceinline__ void store_states(float* p, int row, int states, int live, int lane, float* box, const float (&v)[NS]) {
  using B = StateBox<NS>;
  wave_fence();
#pragma unroll
  for (int i = 0; i < NS; ++i) box[lane * B::kRow + i] = v[i];
  wave_fence();
  if (row % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
    for (int k = 0; k < NS / 4; ++k) {
      const int i = lane + 64 * k, c = i / (NS / 4), s = i % (NS / 4) * 4;
      if (c < live && s < states)
        *reinterpret_cast<f32x4_s*>(p + int64_t(c) * row + s) = *reinterpret_cast<const f32x4_s*>(box + c * B::kRow + s);
    }
  } else {
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int i = lane + 64 * k, c = i / NS, s = i % NS;
      if (c < live && s < states) p[int64_t(c) * row + s] = box[c * B::kRow + s];
    }
  }
  wave_fence();
}

// One stream of tokens of a lane's channel: the wave's address of token `t0`
// of a chunk, moved on by whole groups of four tokens, with the lane's four
// tokens at 32-bit offsets behind it.
template <class T>
struct Stream {
  T* p;
  int64_t row;
  unsigned off[4];
  __device__ __forceinline__ Stream(const ScanRows& v, int n, int t0, int chan)
      : p(v.p ? static_cast<T*>(v.p) + int64_t(n) * v.batch + int64_t(t0) * v.row : nullptr), row(v.row) {
#pragma unroll
    for (int j = 0; j < 4; ++j) off[j] = unsigned(j) * unsigned(v.row) + unsigned(chan);
  }
  __device__ __forceinline__ void move(int groups) { p += int64_t(groups) * 4 * row; }
};

// Inputs of four tokens, as they are stored: those of the lane's channel, and
// the lane's share of the rows of B (and C) that the wave spreads through LDS.
template <class T, int NS, int ROWS>
struct Feed {
  static constexpr int kEach = (4 * NS * ROWS + 63) / 64;
  T dt[4], x[4], z[4], bc[kEach];
};

// Loads the four tokens at the streams' places, `left` of them valid (at
// least one).  For those past the valid ones the first is read, for states
// past the last the last: never used, and no branch between the loads.
template <class T, int NS, int ROWS>
__device__ __forceinline__ void feed(Feed<T, NS, ROWS>& f, int left, const Stream<T>& dt, const Stream<T>& x,
                                     const Stream<T>& z, const Stream<T>& b, const Stream<T>& c, int states, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = j < left ? j : 0;
    f.dt[j] = dt.p[dt.off[k]];
    f.x[j] = x.p[x.off[k]];
    f.z[j] = z.p ? z.p[z.off[k]] : T(0);
  }
#pragma unroll
  for (int r = 0; r < Feed<T, NS, ROWS>::kEach; ++r) {
    const int i = lane + 64 * r, which = ROWS == 2 ? i / (4 * NS) : 0;
    const unsigned t = unsigned(min(i / NS % 4, left - 1)), s = unsigned(min(i % NS, states - 1));
    f.bc[r] = ROWS == 2 && which ? c.p[t * unsigned(c.row) + s] : b.p[t * unsigned(b.row) + s];
  }
}

// The rows of B (and C) of four tokens into LDS, [ROWS][4][NS], zero past the
// valid tokens and the last state.
template <class T, int NS, int ROWS>
__device__ __forceinline__ void spread_rows(const Feed<T, NS, ROWS>& f, float* box, int tb, int te, int states, int lane) {
#pragma unroll
  for (int r = 0; r < Feed<T, NS, ROWS>::kEach; ++r) {
    const int i = lane + 64 * r;
    if (4 * NS * ROWS % 64 == 0 || i < 4 * NS * ROWS)
      box[i] = tb + i / NS % 4 < te && i % NS < states ? to_f32(f.bc[r]) : 0.f;
  }
}

// What a chunk adds to the state, starting from zero,
//   h = exp(delta A) h + delta u B,
// and its sum of delta, whose exponential is the whole chunk's decay.  BACK: also
// what it adds to the gradient that leaves it on the left,
//   G = sum_t exp(A sum_{s <= t} delta_s) C gy,  gy = dy silu(z),
// taken forward too, with the running product of the same decays: one walk and one
// exponential a token and state serve both.  2 x 2049 tokens of 2048 channels, 16
// states: 63 us, where a walk each way took 43 + 37.  Where decays grow (delta A
// > 0) that product may overflow beside a gradient that is zero; such a lane
// walks back over its chunk as the formula does, one token and state after
// another (all states at once in registers the compiler kept some for it through
// the whole walk, which then waited for its loads: 4 us more).
template <class T, int NS, bool BACK, bool MULTI>
__global__ __launch_bounds__(MULTI ? 64 * (cc3d::kScanMaxStates / NS) : 64) void scan_carry(ScanArgs a) {
  constexpr int kRows = BACK ? 2 : 1;
  // (LDS for the waves there are: it would limit how many workgroups a compute unit holds)
  __shared__ __attribute__((aligned(16))) float box_all[MULTI ? cc3d::kScanMaxStates / NS : 1][StateBox<NS>::kSize];
  const Place at(a);
  float* box = box_all[at.wave];
  const int n = int(at.item / a.chunks), ch = int(at.item - int64_t(n) * a.chunks);
  const int t0 = ch * a.chunk, te = min(min(t0 + a.chunk, a.t), valid_tokens(a, n));
  const int s0 = at.wave * NS, states = min(a.s - s0, NS);
  const float bias = a.bias ? a.bias[at.chan] : 0.f;
  Stream<T> dt(a.dt, n, t0, at.chan), u(a.u, n, t0, at.chan);
  Stream<T> z(BACK ? a.z : ScanRows{}, n, t0, at.chan), dy(BACK ? a.dy : ScanRows{}, n, t0, at.chan);
  Stream<T> bs(a.b, n, t0, 0), cs(BACK ? a.c : a.b, n, t0, 0);
  bs.p += at.group * a.s + s0;
  cs.p += at.group * a.s + s0;
  Feed<T, NS, kRows> next;
  T next_dy[4];
  auto fetch = [&](int left) {
    feed(next, left, dt, u, z, bs, cs, states, at.lane);
    if constexpr (BACK) {
#pragma unroll
      for (int j = 0; j < 4; ++j) next_dy[j] = dy.p[dy.off[j < left ? j : 0]];
    }
  };
  if (t0 < te) fetch(te - t0);
  float h[NS], a2[NS], g[BACK ? NS : 1], through[BACK ? NS : 1];
  load_states<NS>(a.a + int64_t(at.first) * a.s + s0, a.s, states, at.live, at.lane, box, a2);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    h[i] = 0.f;
    a2[i] = rate_of(a2[i]);
    if constexpr (BACK) {
      g[i] = 0.f;
      through[i] = 1.f;
    }
  }
  float total = 0.f;
  for (int tb = t0; tb < te; tb += 4) {
    wave_fence();
    spread_rows(next, box, tb, te, states, at.lane);
    float delta[4], x[4], gy[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      delta[j] = tb + j < te ? delta_of(a, to_f32(next.dt[j]) + bias) : 0.f;
      x[j] = tb + j < te ? delta[j] * to_f32(next.x[j]) : 0.f;
      total += delta[j];
    }
    if constexpr (BACK) {
#pragma unroll
      for (int j = 0; j < 4; ++j) gy[j] = to_f32(next_dy[j]);
      if (z.p) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = to_f32(next.z[j]);
          gy[j] *= v * sigmoid_f32(v);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) gy[j] = tb + j < te ? gy[j] : 0.f;
    }
    wave_fence();
    if (tb + 4 < te) {
      dt.move(1);
      u.move(1);
      z.move(z.p ? 1 : 0);
      dy.move(BACK ? 1 : 0);
      bs.move(1);
      cs.move(1);
      fetch(te - tb - 4);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float decay = __builtin_amdgcn_exp2f(delta[j] * a2[i]);
        h[i] = fmaf(decay, h[i], x[j] * box[j * NS + i]);
        if constexpr (BACK) {
          through[i] *= decay;
          g[i] = fmaf(through[i], gy[j] * box[(4 + j) * NS + i], g[i]);
        }
      }
    }
  }
  const int channels = a.groups * a.wide;
  const int64_t out = (at.item * a.s + s0) * channels + at.chan;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (i < states) {
      a.carry[out + int64_t(i) * channels] = h[i];
      if constexpr (BACK) a.gcarry[out + int64_t(i) * channels] = g[i];
    }
  if (at.wave == 0) a.sums[at.item * channels + at.chan] = total;
  if constexpr (BACK) {
    unsigned over = 0;  // once infinite, or not a number, a product stays so
#pragma unroll
    for (int i = 0; i < NS; ++i) over |= through[i] <= FLT_MAX ? 0 : 1u << i;
    if (over) {
#pragma nounroll
      for (int i = 0; i < states; ++i) {
        if (!(over >> i & 1)) continue;
        const float rate = rate_of(a.a[int64_t(at.chan) * a.s + s0 + i]);
        float back = 0.f;
#pragma nounroll
        for (int t = te - 1; t >= t0; --t) {
          auto token = [&](const ScanRows& v) { return rows<T>(v, n) + int64_t(t) * v.row; };
          const float delta = delta_of(a, to_f32(token(a.dt)[at.chan]) + bias);
          float gy = to_f32(token(a.dy)[at.chan]);
          if (a.z.p) {
            const float v = to_f32(token(a.z)[at.chan]);
            gy *= v * sigmoid_f32(v);
          }
          back = __builtin_amdgcn_exp2f(delta * rate) * fmaf(gy, to_f32(token(a.c)[at.group * a.s + s0 + i]), back);
        }
        a.gcarry[out + int64_t(i) * channels] = back;
      }
    }
  }
}

// Turns what every chunk adds into the state that enters it, from the
// sequence's first state on, and, in the grid's second half where there is one,
// the gradient that enters it from the right.
// A chunk's decay is kept as its square root and multiplied twice, as it may
// overflow where its product with the state does not: a root is held to 2^127,
// whose square takes every normal number past the largest.
// A workgroup takes 64 channels of one state; each wave loads 16 chunks at
// once and joins them, and the waves' joined stretches meet in LDS, so the
// loads of a long sequence are not one after another.  9.5 us for 128
// chunks of 2048 channels and 16 states.  A grid of up to kJoinGrid workgroups
// takes all of them in turns: `all` of up to 1024 threads each may be more
// threads than a launch holds.
constexpr int kJoinChunks = 16, kJoinWaves = 16;
constexpr unsigned kJoinGrid = 1u << 16;

__global__ __launch_bounds__(64 * kJoinWaves) void scan_join(ScanArgs a, unsigned half, unsigned all) {
  __shared__ float add_of[kJoinWaves][64], sum_of[kJoinWaves][64];
  const int channels = a.groups * a.wide, tiles = (channels + 63) / 64;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, waves = blockDim.x / 64;
  for (unsigned at = blockIdx.x; at < all; at += gridDim.x) {
    // block = (n * S + state) * tiles + tile
    const bool rev = at >= half;
    const unsigned block = rev ? at - half : at;
    const int64_t rest = block / tiles;
    const int tile = int(block - rest * tiles), n = int(rest / a.s), s = int(rest - int64_t(n) * a.s);
    const bool on = tile * 64 + lane < channels;
    const int chan = on ? tile * 64 + lane : channels - 1;
    const float half_a2 = 0.5f * rate_of(a.a[int64_t(chan) * a.s + s]);
    auto root_of = [&](float sum) {
      const float x = sum * half_a2;
      return __builtin_amdgcn_exp2f(x > 127.f ? 127.f : x);  // (NaN stays NaN)
    };
    auto join = [](float root, float h, float add) { return fmaf(root * h, root, add); };
    const float* first = rev ? a.dh_out : a.h_in;
    float enter = first ? first[(int64_t(n) * channels + chan) * a.s + s] : 0.f;
    float* carry = (rev ? a.gcarry : a.carry) + (int64_t(n) * a.chunks * a.s + s) * channels + chan;
    const float* sums = a.sums + int64_t(n) * a.chunks * channels + chan;
    const int64_t step = int64_t(a.s) * channels;
    for (int base = 0; base < a.chunks; base += kJoinChunks * waves) {
      const int c0 = base + wave * kJoinChunks;
      float add[kJoinChunks], root[kJoinChunks], total = 0.f, h = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinChunks; ++i) {
        const int k = min(c0 + i, a.chunks - 1), c = rev ? a.chunks - 1 - k : k;
        add[i] = carry[c * step];
        root[i] = sums[int64_t(c) * channels];
      }
#pragma unroll
      for (int i = 0; i < kJoinChunks; ++i) {
        const bool in = c0 + i < a.chunks;
        add[i] = in ? add[i] : 0.f;
        root[i] = in ? root[i] : 0.f;
        total += root[i];
        root[i] = root_of(root[i]);
        h = join(root[i], h, add[i]);
      }
      __syncthreads();
      add_of[wave][lane] = h;
      sum_of[wave][lane] = total;
      __syncthreads();
      float mine = enter;
      for (int w = 0; w < waves; ++w) {
        if (w == wave) mine = enter;
        enter = join(root_of(sum_of[w][lane]), enter, add_of[w][lane]);
      }
#pragma unroll
      for (int i = 0; i < kJoinChunks; ++i) {
        const int k = c0 + i, c = rev ? a.chunks - 1 - k : k;
        if (k < a.chunks && on) carry[c * step] = mine;
        mine = join(root[i], mine, add[i]);
      }
    }
  }
}

// BACK: both, in one launch.
inline int run_join(const ScanArgs& a, bool back, hipStream_t s) {
  const int waves = a.chunks >= kJoinChunks * kJoinWaves ? kJoinWaves : (a.chunks + kJoinChunks - 1) / kJoinChunks;
  // (below 2^30: the plan holds n * tiles * S / 16 * 64 threads below 2^32)
  const unsigned half = unsigned(int64_t(a.n) * a.s * ((a.groups * a.wide + 63) / 64)), all = back ? 2 * half : half;
  return launch(scan_join, std::min(all, kJoinGrid), 64 * waves, 0, s, a, half, all);
}

template <class T, int NS, bool BACK>
int run_carry(const ScanArgs& a, hipStream_t s) {
  const int64_t blocks = int64_t(a.groups) * a.tiles_per_group * a.n * a.chunks;
  if constexpr (NS == cc3d::kScanFwdStates)  // (fewer a wave: all of them in one)
    if (a.waves > 1) return launch(scan_carry<T, NS, BACK, true>, blocks, 64 * a.waves, 0, s, a);
  return launch(scan_carry<T, NS, BACK, false>, blocks, 64, 0, s, a);
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

}  // namespace
