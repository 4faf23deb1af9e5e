// Short cached causal convolution of each channel, forward and backward.
//
//   Z = [cache; x];  p[t] = b + sum_k w[k] * Z[t + k];  y[t] = act(p[t])
//
// K multiply-adds and one activation per element against one element read
// and one written: bound by memory.  A thread owns eight consecutive channels
// (16-byte loads and stores of bf16, neighbouring threads on neighbouring
// channels) and walks a run of tokens with the last K - 1 of them in
// registers, so x is read once but for K - 1 tokens a run; the next tokens load
// while some are computed.  Measured: 6240 ragged sequences of up to 17 tokens
// of 384 fp32 channels, K = 3, in 72 us (vector units busy 16% of the kernel);
// a full read and write of its tensors at a large copy's 4.74 TB/s would take
// 77.  One token of a few streams costs the launch, 4 us.
#include "cc3d_seq_device.h"

namespace {

struct Conv1dArgs {
  const void *x, *w, *b, *cache_in, *dy, *dcache_out;
  void *y, *cache_out, *dx, *dcache_in;
  const int* lengths;
  float* part;  // backward: [rows][K + 1][C]
  int64_t xb, xr, yb, yr, dyb, dyr, dxb, dxr;
  int n, t, c, seg, nseg;
  int vecs;      // threads side by side along the channels
  int64_t rows;  // backward: workgroups along the tokens
  int64_t items; // n * nseg
};

constexpr int kAhead = 4;

// A thread's eight channels.  Where C is no multiple of eight the last thread
// takes the last eight, some of which are the thread's before it too: both
// compute and store the same values there.  FEW: C is less than eight.
template <class T, bool FEW>
struct Lane {
  Raw8<T> r;
  __device__ __forceinline__ void load(const T* p, int n) {
    if (FEW) r = load_some(p, n);
    else r = load8(p);
  }
  __device__ __forceinline__ void zero() { r = zero8<T>(); }
  __device__ __forceinline__ float get(int j) const { return get8(r, j); }
  static __device__ __forceinline__ void store(T* p, const float* v, int n) {
    if (FEW) store_some(p, n, v);
    else store8(p, v);
  }
};

template <class T, int K, bool FEW, bool SILU>
__global__ __launch_bounds__(256) void conv1d_fwd(Conv1dArgs a) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t item = id / a.vecs;
  if (item >= a.items) return;
  const int cv = int(id - item * a.vecs);
  const int n = int(item / a.nseg), sg = int(item - int64_t(n) * a.nseg);
  const int c0 = FEW ? 0 : min(cv * 8, a.c - 8), left = a.c;
  const int len = a.lengths ? min(max(a.lengths[n], 0), a.t) : a.t;
  const T* x = static_cast<const T*>(a.x) + int64_t(n) * a.xb + c0;
  T* y = static_cast<T*>(a.y) + int64_t(n) * a.yb + c0;
  const T* w = static_cast<const T*>(a.w) + c0;
  const int64_t cache_at = int64_t(n) * (K - 1) * a.c + c0;
  const T* cin = a.cache_in ? static_cast<const T*>(a.cache_in) + cache_at : nullptr;

  Lane<T, FEW> ld;
  float wt[K][8], bias[8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    ld.load(w + int64_t(k) * a.c, left);
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[k][j] = ld.get(j);
  }
  ld.zero();
  if (a.b) ld.load(static_cast<const T*>(a.b) + c0, left);
#pragma unroll
  for (int j = 0; j < 8; ++j) bias[j] = ld.get(j);

  const int t0 = sg * a.seg, t1 = min(t0 + a.seg, a.t);
  // win[i]: token t0 - (K - 1) + i of x, or of the cache before token 0
  Lane<T, FEW> win[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int s = t0 - (K - 1) + i;
    win[i].zero();
    if (s >= 0) {
      if (s < len) win[i].load(x + int64_t(s) * a.xr, left);
    } else if (cin) {
      win[i].load(cin + int64_t(s + K - 1) * a.c, left);
    }
  }
  // kAhead tokens load while kAhead are computed; those past the last are read from it again
  const int te = min(t1, len);
  int t = t0;
  Lane<T, FEW> next[kAhead];
  auto fetch = [&](int from) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i].load(x + int64_t(min(from + i, te - 1)) * a.xr, left);
  };
  if (t < te) fetch(t);
  while (t < te) {
    Lane<T, FEW> now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
    if (t + kAhead < te) fetch(t + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i, ++t) {
      if (t >= te) break;
      win[K - 1] = now[i];
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float s = bias[j];
#pragma unroll
        for (int k = 0; k < K; ++k) s = fmaf(wt[k][j], win[k].get(j), s);
        p[j] = SILU ? s * sigmoid_f32(s) : s;
      }
      Lane<T, FEW>::store(y + int64_t(t) * a.yr, p, left);
#pragma unroll
      for (int q = 0; q < K - 1; ++q) win[q] = win[q + 1];
    }
  }
  float none[8] = {};
  for (; t < t1; ++t) Lane<T, FEW>::store(y + int64_t(t) * a.yr, none, left);

  if (K > 1 && sg == 0 && a.cache_out) {
    T* co = static_cast<T*>(a.cache_out) + cache_at;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int s = len - (K - 1) + i;
      ld.zero();
      if (s >= 0) ld.load(x + int64_t(s) * a.xr, left);
      else if (cin) ld.load(cin + int64_t(s + K - 1) * a.c, left);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = ld.get(j);
      Lane<T, FEW>::store(co + int64_t(i) * a.c, v, left);
    }
  }
}

// Backward.  With dp = dy * act'(p) (zero outside the valid tokens), token s
// of x receives dx[s] = sum_k w[k] dp[s + K - 1 - k], so a thread walks
// tokens t with the last K values of dp in registers and writes dx of token
// t - K + 1; a run ends K - 1 tokens after its last.  dw and db are sums over
// all tokens: a thread keeps them in registers over every run that it takes,
// the workgroup's rows add theirs in LDS, and each workgroup writes one row of
// partial sums; sum_rows adds those in their order.  Three elements move for
// the forward pass' two, against some 267 vector instructions for eight bf16
// channels of a token at K = 4, runs' overlaps included: 2 x 8193 tokens of 2048
// channels in 54 us and 5 for the sums, vector units busy 52% of the kernel; the
// bytes alone would take 42 at a large copy's rate.
template <class T, int K, bool FEW, bool SILU>
__global__ __launch_bounds__(256) void conv1d_bwd(Conv1dArgs a, int lanes) {
  // tokens loaded at once, and unrolled (whole turns of the rings)
  constexpr int kBack = K == 3 ? 3 : K > 4 ? 1 : 2, kGroup = K == 1 ? 2 : K;
  __shared__ float red[256 * 8];
  const int lane = threadIdx.x % lanes, line = threadIdx.x / lanes, lines = 256 / lanes;
  const int tiles = (a.vecs + lanes - 1) / lanes;
  const int tile = int(blockIdx.x % tiles);
  const int64_t row = blockIdx.x / tiles;
  const int cv = tile * lanes + lane;
  const bool on = cv < a.vecs;
  const int c0 = FEW || !on ? 0 : min(cv * 8, a.c - 8), left = a.c;

  Lane<T, FEW> ld;
  float wt[K][8], bias[8], dw[K][8] = {}, db[8] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    ld.load(static_cast<const T*>(a.w) + int64_t(k) * a.c + c0, left);
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[k][j] = ld.get(j);
  }
  ld.zero();
  if (a.b) ld.load(static_cast<const T*>(a.b) + c0, left);
#pragma unroll
  for (int j = 0; j < 8; ++j) bias[j] = ld.get(j);

  for (int64_t item = row * lines + line; on && item < a.items; item += a.rows * lines) {
    const int n = int(item / a.nseg), sg = int(item - int64_t(n) * a.nseg);
    const int len = a.lengths ? min(max(a.lengths[n], 0), a.t) : a.t;
    const T* x = static_cast<const T*>(a.x) + int64_t(n) * a.xb + c0;
    const T* dy = static_cast<const T*>(a.dy) + int64_t(n) * a.dyb + c0;
    T* dx = a.dx ? static_cast<T*>(a.dx) + int64_t(n) * a.dxb + c0 : nullptr;
    const int64_t cache_at = int64_t(n) * (K - 1) * a.c + c0;
    const T* cin = a.cache_in ? static_cast<const T*>(a.cache_in) + cache_at : nullptr;
    const T* dco = a.dcache_out ? static_cast<const T*>(a.dcache_out) + cache_at : nullptr;
    T* dci = a.dcache_in ? static_cast<T*>(a.dcache_in) + cache_at : nullptr;

    const int t0 = sg * a.seg, t1 = min(t0 + a.seg, a.t);
    // Rings of the last K tokens: token t0 + i of the run is in place i % K, so
    // that a group of K tokens, unrolled, moves nothing.
    float win[K][8], dp[K][8] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int s = t0 - K + i;  // place i, overwritten when i = 0
      ld.zero();
      if (i > 0) {
        if (s >= 0) {
          if (s < len) ld.load(x + int64_t(s) * a.xr, left);
        } else if (cin) {
          ld.load(cin + int64_t(s + K - 1) * a.c, left);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) win[i][j] = ld.get(j);
    }
    // kBack tokens load while kBack are computed; for those past the valid ones
    // the last is read, or none where all are, and they are taken as zero
    const int end = t1 + K - 1, last = min(end, len) - 1;
    Lane<T, FEW> next_x[kBack], next_d[kBack];
    auto fetch = [&](int from) {
      if (from > last) return;
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        const int64_t t = min(from + i, last);
        next_x[i].load(x + t * a.xr, left);
        next_d[i].load(dy + t * a.dyr, left);
      }
    };
    fetch(t0);
    for (int tb = t0; tb < end; tb += kGroup) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int t = tb + i;
        if (t >= end) break;
        Lane<T, FEW> now_x = next_x[i % kBack];
        const Lane<T, FEW> now_d = next_d[i % kBack];
        if (i % kBack == kBack - 1 && t + 1 < end) fetch(t + 1);
        if (t >= len) now_x.zero();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          win[i % K][j] = now_x.get(j);
          float g = now_d.get(j);
          if (SILU) {
            float s = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) s = fmaf(wt[k][j], win[(i + 1 + k) % K][j], s);
            const float sg_ = sigmoid_f32(s);
            g *= sg_ * (1.f + s * (1.f - sg_));
          }
          dp[i % K][j] = t < len ? g : 0.f;  // (also beside an infinite argument)
        }
        if (t < t1) {  // the K - 1 tokens after the run are another thread's
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            db[j] += dp[i % K][j];
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][j] = fmaf(dp[i % K][j], win[(i + 1 + k) % K][j], dw[k][j]);
          }
        }
        const int s = t - (K - 1);
        if (s >= t0 || sg == 0) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float acc = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) acc = fmaf(wt[k][j], dp[(i + K - k) % K][j], acc);
            v[j] = acc;
          }
          if (dco && s < len && s >= len - (K - 1)) {
            ld.load(dco + int64_t(s - len + K - 1) * a.c, left);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += ld.get(j);
          }
          if (s >= 0) {
            if (dx) Lane<T, FEW>::store(dx + int64_t(s) * a.dxr, v, left);
          } else if (dci) {
            Lane<T, FEW>::store(dci + int64_t(s + K - 1) * a.c, v, left);
          }
        }
      }
    }
  }

  float* part = a.part + row * (K + 1) * a.c + c0;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = k < K ? dw[k < K ? k : 0][j] : db[j];
    __syncthreads();
    if (line == 0 && on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (FEW && j >= left) continue;
        float s = 0.f;
        for (int l = 0; l < lines; ++l) s += red[(l * lanes + lane) * 8 + j];
        part[int64_t(k) * a.c + j] = s;
      }
    }
  }
}

template <class T, int K, bool SILU, bool FEW>
int run_conv1d(const Conv1dArgs& a, bool backward, hipStream_t s) {
  if (!backward) return launch(conv1d_fwd<T, K, FEW, SILU>, (a.items * a.vecs + 255) / 256, 256, 0, s, a);
  const int lanes = cc3d::conv1d_lanes(a.c);
  return launch(conv1d_bwd<T, K, FEW, SILU>, a.rows * ((a.vecs + lanes - 1) / lanes), 256, 0, s, a, lanes);
}

template <class T, int K, bool SILU>
int pick_few(const Conv1dArgs& a, bool backward, hipStream_t s) {
  return a.c < 8 ? run_conv1d<T, K, SILU, true>(a, backward, s) : run_conv1d<T, K, SILU, false>(a, backward, s);
}

template <class T, bool SILU>
int pick_taps(int k, const Conv1dArgs& a, bool backward, hipStream_t s) {
  switch (k) {
    case 1: return pick_few<T, 1, SILU>(a, backward, s);
    case 2: return pick_few<T, 2, SILU>(a, backward, s);
    case 3: return pick_few<T, 3, SILU>(a, backward, s);
    case 4: return pick_few<T, 4, SILU>(a, backward, s);
    case 5: return pick_few<T, 5, SILU>(a, backward, s);
    case 6: return pick_few<T, 6, SILU>(a, backward, s);
    case 7: return pick_few<T, 7, SILU>(a, backward, s);
    default: return pick_few<T, 8, SILU>(a, backward, s);
  }
}

int pick_type(const cc3d_conv1d_desc_t& d, const Conv1dArgs& a, bool backward, hipStream_t s) {
  const bool silu = d.act == CC3D_ACT_SILU;
  if (d.dtype == CC3D_BF16) return silu ? pick_taps<bf16_s, true>(d.k, a, backward, s) : pick_taps<bf16_s, false>(d.k, a, backward, s);
  return silu ? pick_taps<float, true>(d.k, a, backward, s) : pick_taps<float, false>(d.k, a, backward, s);
}

Conv1dArgs base_args(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c, int seg) {
  Conv1dArgs a{};
  a.n = p.d.n;
  a.t = p.d.t;
  a.c = p.d.c;
  a.vecs = int((int64_t(a.c) + 7) / 8);
  a.seg = seg;
  a.nseg = (a.t + seg - 1) / seg;
  a.items = int64_t(a.n) * a.nseg;
  a.x = c.x.p;
  a.xb = c.x.batch;
  a.xr = c.x.row;
  a.w = c.w;
  a.b = c.b;
  a.cache_in = c.cache_in;
  a.lengths = c.lengths;
  return a;
}

}  // namespace

namespace cc3d {

int launch_conv1d_forward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c, void* stream) {
  Conv1dArgs a = base_args(p, c, p.seg);
  a.y = c.y.p;
  a.yb = c.y.batch;
  a.yr = c.y.row;
  a.cache_out = c.cache_out;
  return pick_type(p.d, a, false, static_cast<hipStream_t>(stream));
}

int launch_conv1d_backward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c, void* stream) {
  Conv1dArgs a = base_args(p, c, p.bwd_seg);
  a.dy = c.dy.p;
  a.dyb = c.dy.batch;
  a.dyr = c.dy.row;
  a.dx = c.dx.p;
  a.dxb = c.dx.batch;
  a.dxr = c.dx.row;
  a.dcache_in = c.dcache_in;
  a.dcache_out = c.dcache_out;
  a.part = static_cast<float*>(c.workspace);
  a.rows = p.bwd_rows;
  const int e = pick_type(p.d, a, true, static_cast<hipStream_t>(stream));
  if (e) return e;
  const int64_t stride = int64_t(p.d.k + 1) * p.d.c, taps = int64_t(p.d.k) * p.d.c;
  const SumJob jobs[] = {{a.part, c.dw, a.rows, taps, stride}, {a.part + taps, c.db, a.rows, p.d.c, stride}};
  return launch_sums(jobs, 2, stream);
}

}  // namespace cc3d
