// Linear attention with a decay for each head: the kernels.
//
//   S[t] = exp(g) S[t-1] + k[t]^T v[t];   o[t] = scale * q[t] S[t]
//
// Over blocks of m <= 64 tokens, i and j counted inside the block, S the state
// before it and f[d] = exp(g d):
//
//   o[i]  = scale * ( f[i+1] q[i] S  +  sum over j <= i of f[i-j] (q[i] . k[j]) v[j] )
//   S'    = f[m] S  +  sum over j of k[j]^T (f[m-1-j] v[j])
//
// The gradients are three such recurrences on other operands: dq is that of
// (do, v, k) over S^T, and dk and dv are those of (v, do, q) and (k, q, do) with
// time reversed, over the gradient of S.  So one kernel (`linear_run`) does all;
// the operands keep the names of the first here: contraction width C (of q and k)
// and value width E (of v and o).
//
// A workgroup of four waves walks a segment of the time axis with the state of
// one head, C by up to 64 columns of E, in registers (fp32, in the layout of the
// matrix products' results) and, for the products with q, as a bf16 copy in LDS.
// Wave w takes tokens 16w..16w+15 of a block: its rows of q stay in its registers
// as operands of both products, and the products q.k, computed transposed, leave
// the matrix cores in the very layout that their second product wants (the order
// of the tokens inside a sum is free as long as both operands agree), so they
// never pass through LDS.  Operands that need tokens along the registers are read
// from LDS with the transposing load.  The next block's rows load while one is
// computed.
//
// Few heads leave compute units idle, so the time axis is split: linear_run
// without outputs gives what each segment adds to the state, linear_join carries
// the states across, and linear_run starts each segment from its own.
//
// Rounding.  bf16 operands of a product are exact; what is computed and then
// multiplied again is rounded: f (q.k) to bf16 (half a step, 2^-8 at most, beside the
// result's own), the state to bf16 for the product with q (the same), and f v, which
// is added to the state, to two bf16 (rounded, and the rest: 2^-16): a state is an
// fp32 result and is carried.  The decay's gradient, fp32 too, takes the state
// as two bf16 as well and multiplies both products of its pairs in fp32.  fp32 tensors
// use the fp32 matrix products throughout.
#pragma once
#include "cc3d_heads_internal.h"
#include "cc3d_seq_device.h"

namespace cc3d {

// One recurrence: operands in their roles.  Element (c, e) of a state is at
// c * sc + e * se of its Dk * Dv floats.
struct LinRun {
  const void *q, *k, *v;
  void* o;
  int64_t qb, qr, kb, kr, vb, vr, ob, orow;  // strides of sequences and tokens
  int qper, kper, vper;                      // heads of the state that share one of theirs
  int c, e, sc, se;
  int blocks;                                // workgroups side by side along E
  int rev;                                   // time reversed inside the valid tokens
  int lead;                                  // 1: the state before a block meets its token i as f[i+1]; 0: as f[i]
  int o_f32;                                 // o is fp32 whatever T
  float score, inter, update;                // factors of the three sums
  const float* from;                         // state before the first token, or null
  float* to;                                 // after the last valid one, or null
  float* segs;                               // [N][H][segments - 1]: states before segments 1, 2, ...
  unsigned first;                            // its first workgroup
};

struct LinArgs {
  LinRun run[3];
  int runs;
  int n, heads, t, seg, segs;
  const float* log_decay;
  const int* lengths;
  // the decay's gradient (of run[0], dq's): the derivative of the states by the decay, q itself, dh_out
  float* segs2;
  const void* x;
  int64_t xb, xr;
  int xper;
  const float* dto;
  double* part;  // [N][H][segments][blocks]
};

// Runs of one type (cc3d_heads_linear_bf16.hip, cc3d_heads_linear_f32.hip):
// out: with outputs, else what each segment adds to the state; dec: with the
// decay's derivative.
int linear_runs_bf16(LinArgs& a, int pad, bool out, bool dec, hipStream_t s);
int linear_runs_f32(LinArgs& a, int pad, bool out, bool dec, hipStream_t s);

}  // namespace cc3d

namespace {

using cc3d::LinArgs;
using cc3d::LinRun;
constexpr int kTok = cc3d::kLinTokens;

typedef __bf16 bf16x8_h __attribute__((ext_vector_type(8)));
typedef short s16x4_h __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_h __attribute__((ext_vector_type(2)));
typedef u32x2_h u32x2_by2 __attribute__((aligned(2)));

__device__ __forceinline__ int valid_tokens(const int* lengths, int n, int t) {
  return lengths ? min(max(lengths[n], 0), t) : t;
}

// exp(g d), 1 where d is zero even for g = -inf; g2 = g log2(e).
__device__ __forceinline__ float fade(float g2, int d) { return d == 0 ? 1.f : __builtin_amdgcn_exp2f(g2 * float(d)); }
// exp(g d) - 1: a state that fades by a little is moved by it, S + S (exp(g d) - 1), so that
// the factor's own rounding (up to 2^-25 beside 1) is not taken again at every block.
__device__ __forceinline__ float fade_m1(float g, int d) { return d == 0 ? 0.f : float(expm1(double(g) * d)); }

__device__ __forceinline__ f32x4_s zero4() { return f32x4_s{0.f, 0.f, 0.f, 0.f}; }

// v rounded to bf16 and the rest, rounded too: v = hi + lo but for 2^-16 of it.
__device__ __forceinline__ void split_bf16(float v, float w, unsigned& hi, unsigned& lo) {
  hi = pack_bf16(v, w);
  const float hv = __uint_as_float(hi << 16), hw = __uint_as_float(hi & 0xffff0000u);
  // (infinite, or rounded to an infinity: no rest)
  lo = pack_bf16(__builtin_fabsf(hv) == __builtin_inff() ? 0.f : v - hv, __builtin_fabsf(hw) == __builtin_inff() ? 0.f : w - hw);
}

// Operands of the matrix products: 32 terms of a sum for 16 rows, eight a lane
// (row lane % 16, terms 8 (lane / 16) .. + 7 of a row in memory, or tokens
// 4 (lane / 16) .. + 3 of two tiles of 16 where tokens are summed over).
template <class T>
struct Mat;

template <>
struct Mat<bf16_s> {
  using Frag = bf16x8_h;
  static constexpr int kPad = 8;
  static constexpr int kParts = 2;  // of what is rounded on its way into a state
  static __device__ __forceinline__ f32x4_s mma(Frag a, Frag b, f32x4_s c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Frag of(const Raw8<bf16_s>& r) { return __builtin_bit_cast(Frag, r.q[0]); }
  static __device__ __forceinline__ Frag row(const bf16_s* p) {
    return __builtin_bit_cast(Frag, *reinterpret_cast<const u32x4_s*>(p));
  }
  // four tokens below each other, at p and 16 rows on, of column lane % 16: p is the lane's place among
  // the four rows of 16 columns that its 16 lanes read together
  static __device__ __forceinline__ const bf16_s* col_at(const bf16_s* tile, int stride, int lane) {
    return tile + (4 * (lane / 16) + lane % 16 / 4) * stride + 4 * (lane % 4);
  }
  static __device__ __forceinline__ s16x4_h col4(const bf16_s* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4_h*)(const_cast<bf16_s*>(p)));
  }
  static __device__ __forceinline__ Frag col(const bf16_s* p, int stride) {
    const s16x4_h a = col4(p), b = col4(p + 16 * stride);
    return __builtin_bit_cast(Frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  static __device__ __forceinline__ Frag of(f32x4_s a, f32x4_s b) {
    return __builtin_bit_cast(Frag, u32x4_s{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]),
                                            pack_bf16(b[2], b[3])});
  }
  static __device__ __forceinline__ void put4(bf16_s* p, f32x4_s v) {
    *reinterpret_cast<u32x2_h*>(p) = u32x2_h{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  }
  static __device__ __forceinline__ void put4_split(bf16_s* p, bf16_s* q, f32x4_s v) {
    u32x2_h hi, lo;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unsigned h, l;
      split_bf16(v[2 * i], v[2 * i + 1], h, l);
      hi[i] = h;
      lo[i] = l;
    }
    *reinterpret_cast<u32x2_h*>(p) = hi;
    *reinterpret_cast<u32x2_h*>(q) = lo;
  }
  static __device__ __forceinline__ void put8(bf16_s* p, const Raw8<bf16_s>& r) {
    *reinterpret_cast<u32x4_s*>(p) = r.q[0];
  }
  static __device__ __forceinline__ void put8_split(bf16_s* p, bf16_s* q, const float* v) {
    put4_split(p, q, f32x4_s{v[0], v[1], v[2], v[3]});
    put4_split(p + 4, q + 4, f32x4_s{v[4], v[5], v[6], v[7]});
  }
};

template <>
struct Mat<float> {
  struct Frag {
    float x[8];
  };
  static constexpr int kPad = 4;
  static constexpr int kParts = 1;
  // (the eight products take the lanes' terms one after another: any order of the 32 does)
  static __device__ __forceinline__ f32x4_s mma(const Frag& a, const Frag& b, f32x4_s c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[i], b.x[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag of(const Raw8<float>& r) { return __builtin_bit_cast(Frag, r); }
  static __device__ __forceinline__ Frag row(const float* p) {
    Raw8<float> r;
    r.q[0] = reinterpret_cast<const u32x4_s*>(p)[0];
    r.q[1] = reinterpret_cast<const u32x4_s*>(p)[1];
    return of(r);
  }
  static __device__ __forceinline__ const float* col_at(const float* tile, int stride, int lane) {
    return tile + 4 * (lane / 16) * stride + lane % 16;
  }
  static __device__ __forceinline__ Frag col(const float* p, int stride) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.x[i] = p[(i % 4 + i / 4 * 16) * stride];
    return f;
  }
  static __device__ __forceinline__ Frag of(f32x4_s a, f32x4_s b) {
    return Frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  static __device__ __forceinline__ void put4(float* p, f32x4_s v) { *reinterpret_cast<f32x4_s*>(p) = v; }
  static __device__ __forceinline__ void put4_split(float* p, float*, f32x4_s v) { put4(p, v); }
  static __device__ __forceinline__ void put8(float* p, const Raw8<float>& r) {
    reinterpret_cast<u32x4_s*>(p)[0] = r.q[0];
    reinterpret_cast<u32x4_s*>(p)[1] = r.q[1];
  }
  static __device__ __forceinline__ void put8_split(float* p, float* q, const float* v) {
    put4_split(p, q, f32x4_s{v[0], v[1], v[2], v[3]});
    put4_split(p + 4, q + 4, f32x4_s{v[4], v[5], v[6], v[7]});
  }
};

// Eight columns from `col` of a row `width` wide; zeros past it.
template <class T>
__device__ __forceinline__ Raw8<T> load_cols(const T* row, int col, int width) {
  if (col + 8 <= width) return load8(row + col);
  if (col < width) return load_some(row + col, width - col);
  return zero8<T>();
}

// Four columns of a result.
template <class T>
__device__ __forceinline__ void store_cols(T* row, int col, int width, f32x4_s v) {
  if (col + 4 <= width) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x2_by2*>(row + col) = u32x2_h{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
      *reinterpret_cast<u32x4_by4*>(row + col) = __builtin_bit_cast(u32x4_s, v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (col + i < width) row[col + i] = from_f32<T>(v[i]);
}

// LDS of a workgroup, in elements of T: rows of k, rows of v, the rows of f v in
// kParts (twice with the decay's derivative), the state's columns (with the
// derivative: both, each in kParts; not without outputs).
template <class T, int DP, bool OUT, bool DEC>
struct LinTiles {
  using M = Mat<T>;
  static constexpr int kCols = cc3d::linear_cols(DP);
  static constexpr int kRowK = DP + M::kPad, kRowV = kCols + M::kPad;
  static constexpr int kK = 0, kV = kK + kTok * kRowK, kF = kV + (OUT ? kTok * kRowV : 0);
  static constexpr int kS = kF + kTok * kRowV * M::kParts * (DEC ? 2 : 1);
  static constexpr int kStates = !OUT ? 0 : DEC ? 2 * M::kParts : 1;
  static constexpr int kTotal = kS + kCols * kRowK * kStates;
  static constexpr int kBytes = kTotal * int(sizeof(T));
};

template <class T, int DP, bool OUT, bool DEC>
__global__ __launch_bounds__(cc3d::kLinThreads) void linear_run(LinArgs a) {
  using M = Mat<T>;
  using L = LinTiles<T, DP, OUT, DEC>;
  using Frag = typename M::Frag;
  constexpr int kCols = L::kCols, kRowK = L::kRowK, kRowV = L::kRowV;
  constexpr int kMt = DP / 64, kNt = kCols / 16, kSteps = DP / 32;  // a wave's tiles of the state, steps of a sum over C
  constexpr int kVecK = DP / 32, kVecV = kCols / 32;                // eights of k and v that a thread stages
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int odd[2];  // a block of v holds an infinity or NaN
  T* lds = reinterpret_cast<T*>(smem);
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, lane16 = lane % 16, quad = lane / 16;

  int which = 0;
  while (which + 1 < a.runs && blockIdx.x >= a.run[which + 1].first) ++which;
  const LinRun& r = a.run[which];
  const int starts = OUT ? a.segs : a.segs - 1;
  int64_t id = blockIdx.x - r.first;
  const int block = int(id % r.blocks);
  id /= r.blocks;
  const int s = int(id % starts);
  id /= starts;
  const int h = int(id % a.heads);
  const int64_t n = id / a.heads, nh = n * a.heads + h;
  const int e0 = block * kCols;
  const int len = valid_tokens(a.lengths, int(n), a.t);
  const int begin = s * a.seg, end = min(begin + a.seg, len);

  const T* q = static_cast<const T*>(r.q) + n * r.qb + int64_t(h / r.qper) * r.c;
  const T* k = static_cast<const T*>(r.k) + n * r.kb + int64_t(h / r.kper) * r.c;
  const T* v = static_cast<const T*>(r.v) + n * r.vb + int64_t(h / r.vper) * r.e + e0;
  const int width = min(kCols, r.e - e0);
  // token p of the recurrence
  auto at = [&](int p) { return int64_t(r.rev ? len - 1 - p : p); };

  const float g = a.log_decay ? a.log_decay[h] : 0.f, g2 = g * kLog2e;
  const float whole_m1 = fade_m1(g, kTok);

  // ---- the state before the segment, in the products' layout: element i of tile (mt, nt) is
  // c = 16 (wave kMt + mt) + 4 quad + i, e = 16 nt + lane16
  f32x4_s st[kMt][kNt], st2[DEC ? kMt : 1][DEC ? kNt : 1];
  auto each_state = [&](auto&& f) {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 16 * (wave * kMt + mt) + 4 * quad + i, e = 16 * nt + lane16;
          f(mt, nt, i, c < r.c && e < width, c * r.sc + (e0 + e) * r.se);
        }
  };
  const int64_t size = int64_t(r.c) * r.e;
  const float* from = nullptr;
  if constexpr (OUT) from = s > 0 ? r.segs + (nh * (a.segs - 1) + s - 1) * size : r.from ? r.from + nh * size : nullptr;
  each_state([&](int mt, int nt, int i, bool in, int off) { st[mt][nt][i] = from && in ? from[off] : 0.f; });
  if constexpr (DEC) {
    const float* from2 = OUT && s > 0 ? a.segs2 + (nh * (a.segs - 1) + s - 1) * size : nullptr;
    each_state([&](int mt, int nt, int i, bool in, int off) { st2[mt][nt][i] = from2 && in ? from2[off] : 0.f; });
  }
  // its columns as rows of an operand
  auto put_state = [&] {
    if constexpr (OUT) {
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          T* p = lds + L::kS + (16 * nt + lane16) * kRowK + 16 * (wave * kMt + mt) + 4 * quad;
          constexpr int kOne = kCols * kRowK;
          if constexpr (DEC) {
            M::put4_split(p, p + kOne, st[mt][nt]);
            M::put4_split(p + kOne * M::kParts, p + kOne * (M::kParts + 1), st2[mt][nt]);
          } else {
            M::put4(p, st[mt][nt]);
          }
        }
    }
  };

  // ---- constants of a lane: its token i of a block, the factors f[i-j] of its products q.k
  const int i_tok = 16 * wave + lane16;
  float near[4][4], lead = 0.f;
  if constexpr (OUT) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = i_tok - (16 * t + 4 * quad + i);
        near[t][i] = d >= 0 ? r.score * fade(g2, d) : 0.f;
      }
    lead = r.inter * fade(g2, i_tok + r.lead);
  }

  // ---- rows of a block in flight
  Raw8<T> kn[kVecK], vn[kVecV], qn[OUT ? kSteps : 1];
  const int kc = tid % (DP / 8) * 8, krow = tid / (DP / 8), vc = tid % (kCols / 8) * 8, vrow = tid / (kCols / 8);
  constexpr int kStepK = 256 / (DP / 8), kStepV = 256 / (kCols / 8);
  auto fetch = [&](int p0) {
#pragma unroll
    for (int x = 0; x < kVecK; ++x) {
      const int p = p0 + krow + x * kStepK;
      kn[x] = p < end ? load_cols(k + at(p) * r.kr, kc, r.c) : zero8<T>();
    }
#pragma unroll
    for (int x = 0; x < kVecV; ++x) {
      const int p = p0 + vrow + x * kStepV;
      vn[x] = p < end ? load_cols(v + at(p) * r.vr, vc, width) : zero8<T>();
    }
    if constexpr (OUT) {
      const int p = p0 + i_tok;
#pragma unroll
      for (int x = 0; x < kSteps; ++x)
        qn[x] = p < end ? load_cols(q + at(p) * r.qr, 32 * x + 8 * quad, r.c) : zero8<T>();
    }
  };
  if (begin < end) fetch(begin);
  put_state();
  if (tid < 2) odd[tid] = 0;
  __syncthreads();

  double decay = 0.0;
  const bool keeps = OUT ? s + 1 == a.segs && (r.to || (DEC && a.dto)) : true;  // the state after the segment is asked for
  int turn = 0;
  for (int p0 = begin; p0 < end; p0 += kTok, turn ^= 1) {
    const int m = min(kTok, end - p0);
    // ---- stage k, v and f v
#pragma unroll
    for (int x = 0; x < kVecK; ++x) M::put8(lds + L::kK + (krow + x * kStepK) * kRowK + kc, kn[x]);
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kVecV; ++x) {
      const int j = vrow + x * kStepV, place = j * kRowV + vc;
      float f[8], f2[8];
      const int left = m - 1 - j;
      const float w = left >= 0 ? r.update * fade(g2, left + 1 - r.lead) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = get8(vn[x], i);
        bad |= !(__builtin_fabsf(u) < __builtin_inff());
        f[i] = u * w;
        f2[i] = f[i] * float(left);
      }
      T* p = lds + L::kF + place;
      constexpr int kOne = kTok * kRowV;
      M::put8_split(p, p + kOne, f);
      if constexpr (DEC) M::put8_split(p + kOne * M::kParts, p + kOne * (M::kParts + 1), f2);
      if constexpr (OUT) M::put8(lds + L::kV + place, vn[x]);
    }
    Frag qf[OUT ? kSteps : 1];
    if constexpr (OUT) {
#pragma unroll
      for (int x = 0; x < kSteps; ++x) qf[x] = M::of(qn[x]);
      if (bad) odd[turn] = 1;
    }
    __syncthreads();
    if (p0 + kTok < end) fetch(p0 + kTok);

    if constexpr (OUT) {
      if (tid == 0) odd[turn ^ 1] = 0;
      if (16 * wave < m) {
        // ---- products q.k, transposed: element i of tile t is j = 16 t + 4 quad + i of the lane's token
        f32x4_s pr[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          pr[t] = zero4();
          if (t <= wave) {
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
              pr[t] = M::mma(M::row(lds + L::kK + (16 * t + lane16) * kRowK + 32 * x + 8 * quad), qf[x], pr[t]);
          }
        }
        const T* state = lds + L::kS + lane16 * kRowK + 8 * quad;
        if constexpr (!DEC) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[t][i] = 16 * t + 4 * quad + i <= i_tok ? pr[t][i] * near[t][i] : 0.f;
          const Frag pf[2] = {M::of(pr[0], pr[1]), M::of(pr[2], pr[3])};
          f32x4_s o[kNt];
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            o[nt] = zero4();
#pragma unroll
            for (int x = 0; x < kSteps; ++x) o[nt] = M::mma(M::row(state + 16 * nt * kRowK + 32 * x), qf[x], o[nt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][i] *= lead;
          }
          if (!odd[turn]) {
            const T* vt = M::col_at(lds + L::kV, kRowV, lane);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (2 * y <= wave) {
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                  o[nt] = M::mma(M::col(vt + 32 * y * kRowV + 16 * nt, kRowV), pf[y], o[nt]);
              }
            }
          } else {
            // an infinity or NaN among the block's v meets no product of an earlier token, not even a zero one
            for (int j = 0; j < kTok; ++j) {
              float p = 0.f;
#pragma unroll
              for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) p = 16 * t + i == j / 16 * 16 + j % 4 ? pr[t][i] : p;
              p = __shfl(p, j % 16 / 4 * 16 + lane16);
              if (j <= i_tok) {
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    o[nt][i] = fmaf(p, to_f32(lds[L::kV + j * kRowV + 16 * nt + 4 * quad + i]), o[nt][i]);
              }
            }
          }
          if (i_tok < m) {
            const int64_t row = n * r.ob + at(p0 + i_tok) * r.orow + int64_t(h) * r.e + e0;
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              if (r.o_f32) store_cols(static_cast<float*>(r.o) + row, 16 * nt + 4 * quad, width, o[nt]);
              else store_cols(static_cast<T*>(r.o) + row, 16 * nt + 4 * quad, width, o[nt]);
            }
          }
        } else {
          // ---- the decay's gradient: with x the rows of q, (i - j) f[i-j] (do[i] . v[j]) (x[i] . k[j]) of every pair
          // (here only these columns of x and k), and x[i] . f[i+1] (S2 + (i + 1) S) do[i]
          const T* xrow = static_cast<const T*>(a.x) + n * a.xb + int64_t(h / a.xper) * r.e + e0;
          const bool there = i_tok < m;
          if (there) xrow += at(p0 + i_tok) * a.xr;
          Frag xf[kCols / 32];
#pragma unroll
          for (int x = 0; x < kCols / 32; ++x)
            xf[x] = M::of(there ? load_cols(xrow, 32 * x + 8 * quad, width) : zero8<T>());
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (t <= wave) {
              f32x4_s xk = zero4();
#pragma unroll
              for (int x = 0; x < kCols / 32; ++x)
                xk = M::mma(M::row(lds + L::kV + (16 * t + lane16) * kRowV + 32 * x + 8 * quad), xf[x], xk);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int d = i_tok - (16 * t + 4 * quad + i);
                sum += d > 0 ? float(d) * near[t][i] * pr[t][i] * xk[i] : 0.f;
              }
            }
          }
          constexpr int kOne = kCols * kRowK;
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            f32x4_s u = zero4(), w = zero4();
#pragma unroll
            for (int y = 0; y < M::kParts; ++y)
#pragma unroll
              for (int x = 0; x < kSteps; ++x) {
                w = M::mma(M::row(state + y * kOne + 16 * nt * kRowK + 32 * x), qf[x], w);
                u = M::mma(M::row(state + (M::kParts + y) * kOne + 16 * nt * kRowK + 32 * x), qf[x], u);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 16 * nt + 4 * quad + i;
              if (there && e < width) sum += lead * fmaf(float(i_tok + 1), w[i], u[i]) * to_f32(xrow[e]);
            }
          }
          decay += double(sum);
        }
      }
    }

    // ---- the state after the block
    if (keeps || p0 + kTok < end) {
      const float m1 = m == kTok ? whole_m1 : fade_m1(g, m);
      const T* kt = M::col_at(lds + L::kK, kRowK, lane);
      const T* ft = M::col_at(lds + L::kF, kRowV, lane);
      constexpr int kOne = kTok * kRowV;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (DEC) {
              const float both = fmaf(float(m), st[mt][nt][i], st2[mt][nt][i]);
              st2[mt][nt][i] = fmaf(both, m1, both);
            }
            st[mt][nt][i] = fmaf(st[mt][nt][i], m1, st[mt][nt][i]);
          }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (32 * y < m) {
          Frag kf[kMt];
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) kf[mt] = M::col(kt + 32 * y * kRowK + 16 * (wave * kMt + mt), kRowK);
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int part = 0; part < M::kParts; ++part) {
              const Frag f = M::col(ft + part * kOne + 32 * y * kRowV + 16 * nt, kRowV);
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt) st[mt][nt] = M::mma(kf[mt], f, st[mt][nt]);
              if constexpr (DEC) {
                const Frag f2 = M::col(ft + (M::kParts + part) * kOne + 32 * y * kRowV + 16 * nt, kRowV);
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt) st2[mt][nt] = M::mma(kf[mt], f2, st2[mt][nt]);
              }
            }
        }
      }
    }
    __syncthreads();
    if (p0 + kTok < end) put_state();
  }

  // ---- what is left behind: the state, zeros for the tokens that are not valid, the decay's sum
  float* to = nullptr;
  if constexpr (OUT) to = keeps && r.to ? r.to + nh * size : nullptr;
  else to = r.segs + (nh * (a.segs - 1) + s) * size;
  if (to) each_state([&](int mt, int nt, int i, bool in, int off) { if (in) to[off] = st[mt][nt][i]; });
  if constexpr (DEC && !OUT) {
    float* to2 = a.segs2 + (nh * (a.segs - 1) + s) * size;
    each_state([&](int mt, int nt, int i, bool in, int off) { if (in) to2[off] = st2[mt][nt][i]; });
  }
  if constexpr (OUT && !DEC) {
    const int last = min(begin + a.seg, a.t);
    for (int t = max(begin, len) + tid / kCols; t < last; t += cc3d::kLinThreads / kCols) {
      const int e = tid % kCols;
      const int64_t place = n * r.ob + int64_t(t) * r.orow + int64_t(h) * r.e + e0 + e;
      if (e < width) {
        if (r.o_f32) static_cast<float*>(r.o)[place] = 0.f;
        else static_cast<T*>(r.o)[place] = T(0);
      }
    }
  }
  if constexpr (OUT && DEC) {
    if (keeps) {
      const float* dto = a.dto + nh * size;
      each_state([&](int mt, int nt, int i, bool in, int off) { if (in) decay += double(dto[off]) * double(st2[mt][nt][i]); });
    }
    double* box = reinterpret_cast<double*>(smem);  // (the last barrier above is behind every read of the tiles)
    __syncthreads();
    box[tid] = decay;
    __syncthreads();
    for (int half = cc3d::kLinThreads / 2; half > 0; half /= 2) {
      if (tid < half) box[tid] += box[tid + half];
      __syncthreads();
    }
    if (tid == 0) a.part[(nh * a.segs + s) * r.blocks + block] = box[0];
  }
}

template <class T, int DP, bool OUT, bool DEC>
int start_run(const LinArgs& a, int64_t workgroups, hipStream_t s) {
  constexpr int lds = LinTiles<T, DP, OUT, DEC>::kBytes;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_run<T, DP, OUT, DEC>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return int(e);
    }
  }
  return launch(linear_run<T, DP, OUT, DEC>, workgroups, cc3d::kLinThreads, lds, s, a);
}

template <class T>
int start_runs(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  const int starts = out ? a.segs : a.segs - 1;
  int64_t workgroups = 0;
  for (int i = 0; i < a.runs; ++i) {
    a.run[i].blocks = int(cc3d::linear_blocks(a.run[i].e, pad));
    a.run[i].first = unsigned(workgroups);
    workgroups += int64_t(a.n) * a.heads * starts * a.run[i].blocks;
  }
  if (workgroups == 0) return 0;
  auto go = [&](auto d) {
    constexpr int DP = decltype(d)::value;
    if (out) return dec ? start_run<T, DP, true, true>(a, workgroups, s) : start_run<T, DP, true, false>(a, workgroups, s);
    return dec ? start_run<T, DP, false, true>(a, workgroups, s) : start_run<T, DP, false, false>(a, workgroups, s);
  };
  if (pad == 64) return go(std::integral_constant<int, 64>());
  if (pad == 128) return go(std::integral_constant<int, 128>());
  return go(std::integral_constant<int, 256>());
}

}  // namespace
