// Linear attention with a decay for each head: the kernels beside the
// recurrence (cc3d_heads_linear.h), and the launches.
#include "cc3d_heads_linear.h"

#include <algorithm>

namespace {

struct ShortArgs {
  const void *q, *k, *v;
  void* o;
  int64_t qb, kb, vb, ob, qr, kr, vr, orow;
  int qper, kper, vper;
  int heads, t, dk, dv, blocks;
  float scale;
  const float *log_decay, *h_in;
  float* h_out;
  const int* lengths;
};

// v added over the four groups of 16 lanes of a wave, in all of them.
__device__ __forceinline__ float group_quads(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One value of two of a pair's, added to the other half of the pair's lanes: x
// of the lower half of 64 (or of each 32) lanes, y of the upper.
__device__ __forceinline__ float fold32(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Few tokens: the recurrence itself, S = f S + k^T v, o = scale q S, in fp32.
// Reads and writes each state once and does little besides: bound by memory (64
// sequences of 12 heads of 64, one token, 26 MB, in 6.7 us; 1560 of 6 heads, two
// tokens, 320 MB, in 85).  A workgroup has 64 columns of a head's state, four a lane, 16 lines of R rows in
// registers.  The rows of TOK tokens at a time pass through LDS, the next ones in
// flight; q S of a token is summed over a thread's rows, and for all TOK together
// across the lanes of a wave (each step adds two tokens' values at once, so half
// remain) and, through LDS, across the waves.
template <class T, int R, int TOK>
__global__ __launch_bounds__(256) void linear_short(ShortArgs a) {
  constexpr int kRows = 16 * R, kLoads = (2 * kRows + 64) * TOK / 256 + 1;
  __shared__ float tile[TOK * (2 * kRows + 64)];  // [TOK][rows of q, of k, columns of v]
  __shared__ float sums[4][TOK][64];
  const int tid = threadIdx.x, line = tid / 16, e = tid % 16 * 4;
  const unsigned nhb = blockIdx.x, nh = nhb / a.blocks, n = nh / a.heads;
  const int h = int(nh - n * a.heads), e0 = int(nhb - nh * a.blocks) * 64, width = min(64, a.dv - e0);
  const int len = valid_tokens(a.lengths, int(n), a.t);
  const T* q = static_cast<const T*>(a.q) + n * a.qb + int64_t(h / a.qper) * a.dk;
  const T* k = static_cast<const T*>(a.k) + n * a.kb + int64_t(h / a.kper) * a.dk;
  const T* v = static_cast<const T*>(a.v) + n * a.vb + int64_t(h / a.vper) * a.dv + e0;
  T* o = static_cast<T*>(a.o) + n * a.ob + int64_t(h) * a.dv + e0;
  const int64_t state = (int64_t(nh) * a.dk) * a.dv + e0 + e;
  const float f = a.log_decay ? __builtin_amdgcn_exp2f(a.log_decay[h] * kLog2e) : 1.f;

  // (every load is made, where there is nothing to load from a place inside, and put right when it is used)
  T next[kLoads];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int i = tid + 256 * x, tok = min(i / (2 * kRows + 64), TOK - 1), at = i - i / (2 * kRows + 64) * (2 * kRows + 64);
      const int64_t t = min(t0 + tok, max(len - 1, 0));
      const T* p = at < kRows ? q + t * a.qr + min(at, a.dk - 1)
                   : at < 2 * kRows ? k + t * a.kr + min(at - kRows, a.dk - 1) : v + t * a.vr + min(at - 2 * kRows, width - 1);
      next[x] = *p;
    }
  };
  if (len > 0) fetch(0);
  f32x4_s s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = line * R + r;
    s[r] = zero4();
    if (a.h_in && (c < a.dk) & (e < width)) {
      const float* p = a.h_in + state + int64_t(c) * a.dv;
      if (e + 4 <= width) s[r] = __builtin_bit_cast(f32x4_s, *reinterpret_cast<const u32x4_by4*>(p));
      else
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (e + i < width) s[r][i] = p[i];
    }
  }
  for (int t0 = 0; t0 < len; t0 += TOK) {
    const int m = min(TOK, len - t0);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const int i = tid + 256 * x, tok = i / (2 * kRows + 64), at = i - tok * (2 * kRows + 64);
      const bool in = (tok < m) & (at < kRows ? at < a.dk : at < 2 * kRows ? at - kRows < a.dk : at - 2 * kRows < width);
      if (i < TOK * (2 * kRows + 64)) tile[i] = in ? to_f32(next[x]) : 0.f;
    }
    __syncthreads();
    if (t0 + TOK < len) fetch(t0 + TOK);
    f32x4_s part[TOK];
#pragma unroll
    for (int tok = 0; tok < TOK; ++tok) {
      part[tok] = zero4();
      if (tok < m) {
        const float* row = tile + tok * (2 * kRows + 64);
        const f32x4_s vv = *reinterpret_cast<const f32x4_s*>(row + 2 * kRows + e);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float qq = row[line * R + r], kk = row[kRows + line * R + r];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[r][i] = fmaf(f, s[r][i], kk * vv[i]);
            part[tok][i] = fmaf(qq, s[r][i], part[tok][i]);
          }
        }
      }
    }
    const int wave = tid / 64, quad = tid % 64 / 16;
    if constexpr (TOK == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) part[0][i] = group_quads(part[0][i]);
      if (quad == 0) *reinterpret_cast<f32x4_s*>(&sums[wave][0][e]) = part[0];
    } else {
      // token x + TOK / 2 half in the upper lanes, then x + TOK / 4
#pragma unroll
      for (int x = 0; x < TOK / 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[x][i] = fold32(part[x][i], part[x + TOK / 2][i]);
#pragma unroll
      for (int x = 0; x < TOK / 4; ++x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[x][i] = fold16(part[x][i], part[x + TOK / 4][i]);
        *reinterpret_cast<f32x4_s*>(&sums[wave][quad / 2 * (TOK / 2) + quad % 2 * (TOK / 4) + x][e]) = part[x];
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < (TOK * 64 + 255) / 256; ++x) {
      const int i = tid + 256 * x, tok = i / 64, col = i % 64;
      if ((tok < m) & (col < width)) {
        const float sum = (sums[0][tok][col] + sums[1][tok][col]) + (sums[2][tok][col] + sums[3][tok][col]);
        o[(t0 + tok) * a.orow + col] = from_f32<T>(sum * a.scale);
      }
    }
  }
  for (int i = len * 64 + tid; i < a.t * 64; i += 256)
    if (i % 64 < width) o[i / 64 * a.orow + i % 64] = T(0);
  if (!a.h_out) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = line * R + r;
    if (!((c < a.dk) & (e < width))) continue;
    float* p = a.h_out + state + int64_t(c) * a.dv;
    if (e + 4 <= width) *reinterpret_cast<u32x4_by4*>(p) = __builtin_bit_cast(u32x4_s, s[r]);
    else
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (e + i < width) p[i] = s[r][i];
  }
}

template <class T>
int start_short(const ShortArgs& a, int64_t workgroups, hipStream_t s) {
  auto go = [&](auto tok) {
    constexpr int TOK = decltype(tok)::value;
    if (a.dk <= 64) return launch(linear_short<T, 4, TOK>, workgroups, 256, 0, s, a);
    if (a.dk <= 128) return launch(linear_short<T, 8, TOK>, workgroups, 256, 0, s, a);
    return launch(linear_short<T, 16, TOK>, workgroups, 256, 0, s, a);
  };
  return a.t == 1 ? go(std::integral_constant<int, 1>()) : go(std::integral_constant<int, 8>());
}

struct JoinArgs {
  struct Way {
    const float* from;  // [N][H][size], or null
    float* segs;        // [N][H][segments - 1][size]: what a segment adds; becomes the state between two
    float* copy;        // of `from`, or null
    int rev;            // from the last segment to the first
  } way[2];
  int64_t items, size;  // states of all heads, floats of one
  int heads, t, seg, segs;
  const float* log_decay;
  const int* lengths;
};

// States across segments: after[s] = f[tokens of s] before[s] + added[s] in 64 bits.  Eight
// segments' loads are in flight.
__global__ __launch_bounds__(256) void linear_join(JoinArgs a) {
  const JoinArgs::Way w = a.way[blockIdx.y];
  const int between = a.segs - 1;
  for (int64_t item = int64_t(blockIdx.x) * 256 + threadIdx.x; item < a.items; item += int64_t(gridDim.x) * 256) {
    const int64_t nh = item / a.size, off = item - nh * a.size, n = nh / a.heads;
    const float g = a.log_decay ? a.log_decay[nh - n * a.heads] : 0.f;
    const int len = valid_tokens(a.lengths, int(n), a.t);
    // (never zero while a token's is not, nor an infinity: infinite states stay so, and no state stays none)
    const double least = lasting(g) ? 0x1p-1074 : 0.0;
    auto fade_of = [&](int tokens) {
      const double f = fade64(g, tokens);
      return f < least ? least : f > 0x1.fffffffffffffp1023 ? 0x1.fffffffffffffp1023 : f;
    };
    const double whole = fade_of(a.seg);
    // (slot x lies between segments x and x + 1)
    float* p = w.segs + (nh * between + (w.rev ? between - 1 : 0)) * a.size + off;
    const int64_t step = w.rev ? -a.size : a.size;
    const float from = w.from ? w.from[item] : 0.f;
    if (w.copy) w.copy[item] = from;
    double s = from;
    for (int x0 = 0; x0 < between; x0 += 8) {
      float u[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) u[x] = p[min(x0 + x, between - 1) * step];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        if (x0 + x >= between) break;
        const int segment = w.rev ? between - x0 - x : x0 + x;
        const int tokens = min(max(len - segment * a.seg, 0), a.seg);
        s = fma(s, tokens == a.seg ? whole : fade_of(tokens), double(u[x]));
        p[(x0 + x) * step] = float(s);
      }
    }
  }
}

struct HeadSum {
  const float* part;  // [N][T][heads][per][D]
  void* out;
  int64_t batch, row, rows;  // rows: N T heads
  int per, d, lanes, t, heads;  // heads: of the result; lanes: of a row, four columns each (a power of two)
};
// dlog_decay's partial sums [n][heads][each]
struct DecaySum {
  const double* part;
  float* out;
  int n, heads, each;
};
struct HeadSums {
  HeadSum job[3];
  DecaySum decay;
  int jobs;
};

__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a >> 32 ? a / b : int64_t(unsigned(a) / unsigned(b));
}

// What the recurrences leave in parts.  Gradients of shared heads: sums over the heads
// that share one, in order (2 by 2049 tokens, two gradients of 4 heads of 64 from 16: 8 us,
// a value a thread 12).  Behind them dlog_decay, a head a workgroup: each thread's partial
// sums in order, then a tree (5 us as a launch of its own).
template <class T>
__global__ __launch_bounds__(256) void linear_sums(HeadSums a) {
  const int tid = threadIdx.x;
  if (int(blockIdx.y) == a.jobs) {
    __shared__ double box[256];
    const DecaySum& j = a.decay;
    for (int h = blockIdx.x; h < j.heads; h += gridDim.x) {
      double s = 0.0;
      for (int64_t i = tid; i < int64_t(j.n) * j.each; i += 256) {
        const int64_t b = quotient(i, j.each);
        s += j.part[(b * j.heads + h) * j.each + (i - b * j.each)];
      }
      box[tid] = s;
      __syncthreads();
      for (int half = 128; half > 0; half /= 2) {
        if (tid < half) box[tid] += box[tid + half];
        __syncthreads();
      }
      if (tid == 0) j.out[h] = float(box[0]);
      __syncthreads();
    }
    return;
  }
  const HeadSum j = a.job[blockIdx.y];
  const int each = 256 / j.lanes, c = tid % j.lanes * 4;
  if (c >= j.d) return;
  for (int64_t row = int64_t(blockIdx.x) * each + tid / j.lanes; row < j.rows; row += int64_t(gridDim.x) * each) {
    const int64_t tok = quotient(row, j.heads), head = row - tok * j.heads, n = quotient(tok, j.t);
    const float* p = j.part + row * j.per * j.d + c;
    T* out = static_cast<T*>(j.out) + n * j.batch + (tok - n * j.t) * j.row + head * j.d + c;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c + 4 <= j.d) {
      for (int x = 0; x < j.per; ++x) {
        const f32x4_s v = __builtin_bit_cast(f32x4_s, *reinterpret_cast<const u32x4_by4*>(p + int64_t(x) * j.d));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
      }
    } else {
      for (int x = 0; x < j.per; ++x)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (c + i < j.d) s[i] += p[int64_t(x) * j.d + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < j.d) out[i] = from_f32<T>(s[i]);
  }
}

constexpr int64_t kGrid = 1 << 16;  // workgroups of the kernels that walk their work in turns

int run(cc3d::LinArgs& a, const cc3d_linear_desc_t& d, bool out, bool dec, hipStream_t s) {
  static cc3d::LinStart* const of[2][3] = {
      {cc3d::linear_f32_eights, cc3d::linear_f32_rest, cc3d::linear_f32_less},
      {cc3d::linear_bf16_eights, cc3d::linear_bf16_rest, cc3d::linear_bf16_less}};
  const int kind = std::min(d.dk, d.dv) < 8 ? kLess : d.dk % 8 || d.dv % 8 ? kRest : kEights;
  int widest = 0;
  for (int i = 0; i < a.runs; ++i) widest = std::max(widest, a.run[i].c);
  return of[d.dtype == CC3D_BF16][kind](a, cc3d::linear_pad(widest), out, dec, s);
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

void set_rows(cc3d::LinRun& r, const cc3d_rows_t& q, int qper, const cc3d_rows_t& k, int kper, const cc3d_rows_t& v, int vper) {
  r.q = q.p;
  r.qb = q.batch;
  r.qr = q.row;
  r.qper = qper;
  r.k = k.p;
  r.kb = k.batch;
  r.kr = k.row;
  r.kper = kper;
  r.v = v.p;
  r.vb = v.batch;
  r.vr = v.row;
  r.vper = vper;
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
  if (p.steps) {
    const ShortArgs a{c.q.p, c.k.p, c.v.p, c.o.p, c.q.batch, c.k.batch, c.v.batch, c.o.batch, c.q.row, c.k.row, c.v.row,
                      c.o.row, d.heads / d.q_heads, d.heads / d.k_heads, d.heads / d.v_heads, d.heads, d.t, d.dk, d.dv,
                      int((d.dv + 63) / 64), d.scale, c.log_decay, c.h_in, c.h_out, c.lengths};
    const int64_t workgroups = int64_t(d.n) * d.heads * a.blocks;
    return d.dtype == CC3D_BF16 ? start_short<bf16_s>(a, workgroups, s) : start_short<float>(a, workgroups, s);
  }
  LinArgs a = common(p, c, p.seg, p.segs);
  a.runs = 1;
  LinRun& r = a.run[0];
  set_rows(r, c.q, d.heads / d.q_heads, c.k, d.heads / d.k_heads, c.v, d.heads / d.v_heads);
  r.o = c.o.p;
  r.ob = c.o.batch;
  r.orow = c.o.row;
  r.c = d.dk;
  r.e = d.dv;
  r.sc = d.dv;
  r.se = 1;
  r.lead = 1;
  r.score = r.inter = d.scale;
  r.update = 1.f;
  r.from = c.h_in;
  r.to = c.h_out;
  r.segs = static_cast<float*>(c.workspace);
  if (a.segs > 1) {
    int e = run(a, d, false, false, s);
    if (e) return e;
    JoinArgs j = join_of(a, int64_t(d.dk) * d.dv);
    // (the last segment may be done before the first one reads its state: not from where the last one's goes)
    float* copy = c.h_in && c.h_in == c.h_out ? r.segs + j.items * (a.segs - 1) : nullptr;
    j.way[0] = {c.h_in, r.segs, copy, 0};
    if (copy) r.from = copy;
    if ((e = start_join(j, 1, s))) return e;
  }
  return run(a, d, true, false, s);
}

int launch_linear_backward(const cc3d_linear_plan& p, const cc3d_linear_args_t& c, void* stream) {
  const auto& d = p.d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LinearSpace space = linear_bwd_space(p);
  float* states = static_cast<float*>(c.workspace);
  float* grads = states + space.state;
  float* blocks = grads + space.state;
  float* part_q = blocks + space.blocks;
  float* part_k = part_q + space.dq;
  float* part_v = part_k + space.dk;
  double* decay = reinterpret_cast<double*>(part_v + space.dv);
  const int qper = d.heads / d.q_heads, kper = d.heads / d.k_heads, vper = d.heads / d.v_heads;
  const bool dec = c.dlog_decay;
  // results go to the caller's view, or where heads are shared to partial sums [N][T][heads][D]
  auto out = [&](LinRun& r, const cc3d_rows_t& v, int per, float* part) {
    if (!v.p) return;
    r.o = per == 1 ? v.p : part;
    r.o_f32 = per > 1;
    r.ob = per == 1 ? v.batch : int64_t(d.t) * d.heads * r.e;
    r.orow = per == 1 ? v.row : int64_t(d.heads) * r.e;
  };
  // dq: the recurrence of (do, v, k) over the transposed state
  LinRun q{};
  set_rows(q, c.grad_o, 1, c.v, vper, c.k, kper);
  q.c = d.dv;
  q.e = d.dk;
  q.sc = 1;
  q.se = d.dv;
  q.lead = 1;
  q.score = q.inter = d.scale;
  q.update = 1.f;
  q.from = c.h_in;
  q.segs = states;
  out(q, c.dq, qper, part_q);
  // dk: that of (v, do, q), reversed
  LinRun k = q;
  set_rows(k, c.v, vper, c.grad_o, 1, c.q, qper);
  k.o = nullptr;
  k.rev = 1;
  k.lead = 0;
  k.inter = 1.f;
  k.update = d.scale;
  k.from = c.dh_out;
  k.segs = grads;
  out(k, c.dk, kper, part_k);
  // dv: of (k, q, do), reversed
  LinRun v = k;
  set_rows(v, c.k, kper, c.q, qper, c.grad_o, 1);
  v.o = nullptr;
  v.c = d.dk;
  v.e = d.dv;
  v.sc = d.dv;
  v.se = 1;
  v.to = c.dh_in;
  out(v, c.dv, vper, part_v);
  // the decay's gradient
  auto meets = [&](LinRun& r, const cc3d_rows_t& x, int per) {
    r.x = x.p;
    r.xb = x.batch;
    r.xr = x.row;
    r.xper = per;
  };
  const int64_t parts = int64_t(d.n) * d.heads * p.bwd_segs * linear_blocks(d.dk, linear_cols(d.dk));
  meets(q, c.q, qper);
  q.pairs = 1;
  q.put = blocks;
  q.part = decay;
  meets(k, c.k, kper);
  k.get = blocks;
  k.part = decay + parts;

  LinArgs a = common(p, c, p.bwd_seg, p.bwd_segs);
  const bool forth = dec || c.dq.p, back = dec || c.dk.p || c.dv.p || c.dh_in;
  int e = 0;
  if (a.segs > 1) {
    JoinArgs j = join_of(a, int64_t(d.dk) * d.dv);
    int ways = 0;
    if (forth) {
      a.run[a.runs++] = q;
      j.way[ways++] = {c.h_in, states, nullptr, 0};
    }
    if (back) {
      a.run[a.runs++] = v;
      j.way[ways++] = {c.dh_out, grads, nullptr, 1};
    }
    if (ways && (e = run(a, d, false, false, s))) return e;
    if (ways && (e = start_join(j, ways, s))) return e;
  }
  a.runs = 0;
  if (dec) {
    for (const LinRun* r : {&q, &k}) {  // (one after the other: the second reads what the first leaves)
      a.runs = 1;
      a.run[0] = *r;
      if ((e = run(a, d, true, true, s))) return e;
    }
    a.runs = 0;
  } else {
    if (c.dq.p) a.run[a.runs++] = q;
    if (c.dk.p) a.run[a.runs++] = k;
  }
  if (c.dv.p || c.dh_in) a.run[a.runs++] = v;
  if (a.runs && (e = run(a, d, true, false, s))) return e;
  HeadSums sums{};
  int64_t most = 0;
  auto add = [&](const cc3d_rows_t& v, int per, const float* part, int heads, int width) {
    if (!v.p || per == 1) return;
    const int64_t rows = int64_t(d.n) * d.t * heads;
    int lanes = 1;
    while (lanes * 4 < width) lanes *= 2;
    sums.job[sums.jobs++] = HeadSum{part, v.p, v.batch, v.row, rows, per, width, lanes, d.t, heads};
    most = std::max(most, (rows * lanes + 255) / 256);
  };
  add(c.dq, qper, part_q, d.q_heads, d.dk);
  add(c.dk, kper, part_k, d.k_heads, d.dk);
  add(c.dv, vper, part_v, d.v_heads, d.dv);
  if (dec) {
    sums.decay = DecaySum{decay, c.dlog_decay, 2 * d.n, d.heads, int(parts / (int64_t(d.n) * d.heads))};
    most = std::max<int64_t>(most, d.heads);
  }
  if (sums.jobs || dec) {
    void* at[] = {&sums};
    const void* kernel = d.dtype == CC3D_BF16 ? reinterpret_cast<const void*>(&linear_sums<bf16_s>)
                                              : reinterpret_cast<const void*>(&linear_sums<float>);
    const hipError_t err = hipLaunchKernel(kernel, dim3(unsigned(std::min(most, kGrid)), unsigned(sums.jobs + (dec ? 1 : 0))),
                                           dim3(256), at, 0, s);
    if (err != hipSuccess) (void)hipGetLastError();
    return int(err);
  }
  return 0;
}

}  // namespace cc3d
