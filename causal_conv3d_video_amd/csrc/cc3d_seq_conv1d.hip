// Short cached causal convolution of each channel, forward and backward, and
// the fixed-order sum over rows of partial sums.
//
//   Z = [cache; x];  p[t] = b + sum_k w[k] * Z[t + k];  y[t] = act(p[t])
//
// K multiply-adds and one activation per element against one element read
// and one written: bound by memory.  A thread owns eight consecutive channels
// (16-byte loads and stores of bf16, neighbouring threads on neighbouring
// channels) and walks a run of tokens with the last K - 1 of them in
// registers, so x is read once but for K - 1 tokens a run.  Where a pointer
// or a stride does not allow 16-byte accesses a thread owns one channel.
#include "cc3d_seq_device.h"

namespace {

struct Conv1dArgs {
  const void *x, *w, *b, *cache_in, *dy, *dcache_out;
  void *y, *cache_out, *dx, *dcache_in;
  const int* lengths;
  float* part;  // backward: [rows][K + 1][C]
  int64_t xb, xr, yb, yr, dyb, dyr, dxb, dxr;
  int n, t, c, seg, nseg;
  int vecs;      // channel vectors (of 8, or of 1)
  int64_t rows;  // backward: workgroups along the tokens
  int64_t items; // n * nseg
};

// VEC channels of storage type T.
template <class T, int VEC>
struct Lane {
  std::conditional_t<VEC == 8, Raw8<T>, T> r;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 8) r = load8(p);
    else r = *p;
  }
  __device__ __forceinline__ void zero() {
    if constexpr (VEC == 8) r = zero8<T>();
    else r = T(0);
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (VEC == 8) return get8(r, j);
    else return to_f32(r);
  }
  static __device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (VEC == 8) store8(p, v);
    else *p = from_f32<T>(v[0]);
  }
};

template <class T, int K, int VEC, bool SILU>
__global__ __launch_bounds__(256) void conv1d_fwd(Conv1dArgs a) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t item = id / a.vecs;
  if (item >= a.items) return;
  const int cv = int(id - item * a.vecs);
  const int n = int(item / a.nseg), sg = int(item - int64_t(n) * a.nseg);
  const int c0 = cv * VEC;
  const int len = a.lengths ? min(max(a.lengths[n], 0), a.t) : a.t;
  const T* x = static_cast<const T*>(a.x) + int64_t(n) * a.xb + c0;
  T* y = static_cast<T*>(a.y) + int64_t(n) * a.yb + c0;
  const T* w = static_cast<const T*>(a.w) + c0;
  const int64_t cache_at = int64_t(n) * (K - 1) * a.c + c0;
  const T* cin = a.cache_in ? static_cast<const T*>(a.cache_in) + cache_at : nullptr;

  Lane<T, VEC> ld;
  float wt[K][VEC], bias[VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    ld.load(w + int64_t(k) * a.c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wt[k][j] = ld.get(j);
  }
  ld.zero();
  if (a.b) ld.load(static_cast<const T*>(a.b) + c0);
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = ld.get(j);

  const int t0 = sg * a.seg, t1 = min(t0 + a.seg, a.t);
  // win[i]: token t0 - (K - 1) + i of x, or of the cache before token 0
  Lane<T, VEC> win[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int s = t0 - (K - 1) + i;
    win[i].zero();
    if (s >= 0) {
      if (s < len) win[i].load(x + int64_t(s) * a.xr);
    } else if (cin) {
      win[i].load(cin + int64_t(s + K - 1) * a.c);
    }
  }
  const int te = min(t1, len);
  int t = t0;
  for (; t < te; ++t) {
    win[K - 1].load(x + int64_t(t) * a.xr);
    float p[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float s = bias[j];
#pragma unroll
      for (int k = 0; k < K; ++k) s = fmaf(wt[k][j], win[k].get(j), s);
      p[j] = SILU ? s * sigmoid_f32(s) : s;
    }
    Lane<T, VEC>::store(y + int64_t(t) * a.yr, p);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) win[i] = win[i + 1];
  }
  float none[VEC] = {};
  for (; t < t1; ++t) Lane<T, VEC>::store(y + int64_t(t) * a.yr, none);

  if (K > 1 && sg == 0 && a.cache_out) {
    T* co = static_cast<T*>(a.cache_out) + cache_at;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int s = len - (K - 1) + i;
      ld.zero();
      if (s >= 0) ld.load(x + int64_t(s) * a.xr);
      else if (cin) ld.load(cin + int64_t(s + K - 1) * a.c);
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = ld.get(j);
      Lane<T, VEC>::store(co + int64_t(i) * a.c, v);
    }
  }
}

// Backward.  With dp = dy * act'(p) (zero outside the valid tokens), token s
// of x receives dx[s] = sum_k w[k] dp[s + K - 1 - k], so a thread walks
// tokens t with the last K values of dp in registers and writes dx of token
// t - K + 1; a run ends K - 1 tokens after its last.  dw and db are sums over
// all tokens: a thread keeps them in registers over every run that it takes,
// the workgroup's rows add theirs in LDS, and each workgroup writes one row of
// partial sums; sum_rows adds those in their order.
template <class T, int K, int VEC, bool SILU>
__global__ __launch_bounds__(256) void conv1d_bwd(Conv1dArgs a, int lanes) {
  __shared__ float red[256 * VEC];
  const int lane = threadIdx.x % lanes, line = threadIdx.x / lanes, lines = 256 / lanes;
  const int tiles = (a.vecs + lanes - 1) / lanes;
  const int tile = int(blockIdx.x % tiles);
  const int64_t row = blockIdx.x / tiles;
  const int cv = tile * lanes + lane;
  const bool on = cv < a.vecs;
  const int c0 = on ? cv * VEC : 0;

  Lane<T, VEC> ld;
  float wt[K][VEC], bias[VEC], dw[K][VEC] = {}, db[VEC] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    ld.load(static_cast<const T*>(a.w) + int64_t(k) * a.c + c0);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wt[k][j] = ld.get(j);
  }
  ld.zero();
  if (a.b) ld.load(static_cast<const T*>(a.b) + c0);
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = ld.get(j);

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
    Lane<T, VEC> win[K];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int s = t0 - (K - 1) + i;
      win[i].zero();
      if (s >= 0) {
        if (s < len) win[i].load(x + int64_t(s) * a.xr);
      } else if (cin) {
        win[i].load(cin + int64_t(s + K - 1) * a.c);
      }
    }
    float dp[K][VEC] = {};  // dp[i]: token t - (K - 1) + i
    for (int t = t0; t < t1 + K - 1; ++t) {
      win[K - 1].zero();
#pragma unroll
      for (int j = 0; j < VEC; ++j) dp[K - 1][j] = 0.f;
      if (t < len) {
        win[K - 1].load(x + int64_t(t) * a.xr);
        ld.load(dy + int64_t(t) * a.dyr);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float g = ld.get(j);
          if (SILU) {
            float s = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) s = fmaf(wt[k][j], win[k].get(j), s);
            const float sg_ = sigmoid_f32(s);
            g *= sg_ * (1.f + s * (1.f - sg_));
          }
          dp[K - 1][j] = g;
          if (t < t1) {  // the K - 1 tokens after the run are another thread's
            db[j] += g;
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][j] = fmaf(g, win[k].get(j), dw[k][j]);
          }
        }
      }
      const int s = t - (K - 1);
      if (s >= t0 || sg == 0) {
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float acc = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) acc = fmaf(wt[k][j], dp[K - 1 - k][j], acc);
          v[j] = acc;
        }
        if (dco && s < len && s >= len - (K - 1)) {
          ld.load(dco + int64_t(s - len + K - 1) * a.c);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[j] += ld.get(j);
        }
        if (s >= 0) {
          if (dx) Lane<T, VEC>::store(dx + int64_t(s) * a.dxr, v);
        } else if (dci) {
          Lane<T, VEC>::store(dci + int64_t(s + K - 1) * a.c, v);
        }
      }
#pragma unroll
      for (int i = 0; i < K - 1; ++i) {
        win[i] = win[i + 1];
#pragma unroll
        for (int j = 0; j < VEC; ++j) dp[i][j] = dp[i + 1][j];
      }
    }
  }

  float* part = a.part + row * (K + 1) * a.c + c0;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[threadIdx.x * VEC + j] = k < K ? dw[k < K ? k : 0][j] : db[j];
    __syncthreads();
    if (line == 0 && on) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float s = 0.f;
        for (int l = 0; l < lines; ++l) s += red[(l * lanes + lane) * VEC + j];
        part[int64_t(k) * a.c + j] = s;
      }
    }
  }
}

// out[m] = sum over r of part[r * stride + m]: 16 rows at a time by 64 columns.
__global__ __launch_bounds__(1024) void sum_rows(const float* part, int64_t rows, int64_t cols, int64_t stride, float* out) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x % 64, line = threadIdx.x / 64;
  const int64_t m = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.f;
  if (m < cols)
    for (int64_t r = line; r < rows; r += 16) s += part[r * stride + m];
  red[line][lane] = s;
  __syncthreads();
  if (line == 0 && m < cols) {
#pragma unroll
    for (int l = 1; l < 16; ++l) s += red[l][lane];
    out[m] = s;
  }
}

bool vec_ok(const void* p, int64_t s0, int64_t s1) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0);
}

template <class T, int K, bool SILU>
void run_conv1d(const Conv1dArgs& in, bool vec, bool backward, hipStream_t s) {
  Conv1dArgs a = in;
  a.vecs = vec ? a.c / 8 : a.c;
  a.items = int64_t(a.n) * a.nseg;
  if (!backward) {
    const unsigned blocks = unsigned((a.items * a.vecs + 255) / 256);
    if (vec) conv1d_fwd<T, K, 8, SILU><<<blocks, 256, 0, s>>>(a);
    else conv1d_fwd<T, K, 1, SILU><<<blocks, 256, 0, s>>>(a);
    return;
  }
  int lanes = 1;
  while (lanes < 64 && lanes < a.vecs) lanes *= 2;
  const int64_t lines = 256 / lanes;
  const int64_t rows = (a.items + lines - 1) / lines;
  if (rows < a.rows) a.rows = rows;
  const unsigned blocks = unsigned(a.rows * ((a.vecs + lanes - 1) / lanes));
  if (vec) conv1d_bwd<T, K, 8, SILU><<<blocks, 256, 0, s>>>(a, lanes);
  else conv1d_bwd<T, K, 1, SILU><<<blocks, 256, 0, s>>>(a, lanes);
}

template <class T, bool SILU>
void pick_taps(int k, const Conv1dArgs& a, bool vec, bool backward, hipStream_t s) {
  switch (k) {
    case 1: return run_conv1d<T, 1, SILU>(a, vec, backward, s);
    case 2: return run_conv1d<T, 2, SILU>(a, vec, backward, s);
    case 3: return run_conv1d<T, 3, SILU>(a, vec, backward, s);
    case 4: return run_conv1d<T, 4, SILU>(a, vec, backward, s);
    case 5: return run_conv1d<T, 5, SILU>(a, vec, backward, s);
    case 6: return run_conv1d<T, 6, SILU>(a, vec, backward, s);
    case 7: return run_conv1d<T, 7, SILU>(a, vec, backward, s);
    default: return run_conv1d<T, 8, SILU>(a, vec, backward, s);
  }
}

void pick_type(const cc3d_conv1d_desc_t& d, const Conv1dArgs& a, bool vec, bool backward, hipStream_t s) {
  const bool silu = d.act == CC3D_ACT_SILU;
  if (d.dtype == CC3D_BF16) {
    if (silu) pick_taps<bf16_s, true>(d.k, a, vec, backward, s);
    else pick_taps<bf16_s, false>(d.k, a, vec, backward, s);
  } else {
    if (silu) pick_taps<float, true>(d.k, a, vec, backward, s);
    else pick_taps<float, false>(d.k, a, vec, backward, s);
  }
}

Conv1dArgs base_args(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c) {
  Conv1dArgs a{};
  a.n = p.d.n;
  a.t = p.d.t;
  a.c = p.d.c;
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

int launch_sum_rows(const float* part, int64_t rows, int64_t cols, int64_t stride, float* out, void* stream) {
  if (!out) return 0;
  sum_rows<<<unsigned((cols + 63) / 64), 1024, 0, static_cast<hipStream_t>(stream)>>>(part, rows, cols, stride, out);
  return int(hipGetLastError());
}

int launch_conv1d_forward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c, void* stream) {
  Conv1dArgs a = base_args(p, c);
  a.y = c.y.p;
  a.yb = c.y.batch;
  a.yr = c.y.row;
  a.cache_out = c.cache_out;
  a.seg = p.seg;
  a.nseg = (p.d.t + p.seg - 1) / p.seg;
  const bool vec = p.d.c % 8 == 0 && vec_ok(c.x.p, c.x.batch, c.x.row) && vec_ok(c.y.p, c.y.batch, c.y.row) &&
                   vec_ok(c.w, 0, 0) && vec_ok(c.b, 0, 0) && vec_ok(c.cache_in, 0, 0) && vec_ok(c.cache_out, 0, 0);
  pick_type(p.d, a, vec, false, static_cast<hipStream_t>(stream));
  return int(hipGetLastError());
}

int launch_conv1d_backward(const cc3d_conv1d_plan& p, const cc3d_conv1d_args_t& c, void* stream) {
  Conv1dArgs a = base_args(p, c);
  a.dy = c.dy.p;
  a.dyb = c.dy.batch;
  a.dyr = c.dy.row;
  a.dx = c.dx.p;
  a.dxb = c.dx.batch;
  a.dxr = c.dx.row;
  a.dcache_in = c.dcache_in;
  a.dcache_out = c.dcache_out;
  a.part = static_cast<float*>(c.workspace);
  a.seg = p.bwd_seg;
  a.nseg = (p.d.t + p.bwd_seg - 1) / p.bwd_seg;
  a.rows = p.bwd_rows;
  const bool vec = p.d.c % 8 == 0 && vec_ok(c.x.p, c.x.batch, c.x.row) && vec_ok(c.dy.p, c.dy.batch, c.dy.row) &&
                   vec_ok(c.dx.p, c.dx.batch, c.dx.row) && vec_ok(c.w, 0, 0) && vec_ok(c.b, 0, 0) &&
                   vec_ok(c.cache_in, 0, 0) && vec_ok(c.dcache_in, 0, 0) && vec_ok(c.dcache_out, 0, 0);
  // rows actually launched: as run_conv1d works them out
  const int64_t vecs = vec ? p.d.c / 8 : p.d.c;
  int64_t lanes = 1;
  while (lanes < 64 && lanes < vecs) lanes *= 2;
  const int64_t lines = 256 / lanes;
  a.rows = std::min<int64_t>(a.rows, (int64_t(a.n) * a.nseg + lines - 1) / lines);
  pick_type(p.d, a, vec, true, static_cast<hipStream_t>(stream));
  int e = int(hipGetLastError());
  const int64_t stride = int64_t(p.d.k + 1) * p.d.c;
  if (!e) e = launch_sum_rows(a.part, a.rows, int64_t(p.d.k) * p.d.c, stride, c.dw, stream);
  if (!e) e = launch_sum_rows(a.part + int64_t(p.d.k) * p.d.c, a.rows, p.d.c, stride, c.db, stream);
  return e;
}

}  // namespace cc3d
