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
};

struct LinArgs {
  LinRun run[3];
  int runs, parts;   // parts: workgroups of all runs that share a head and segment
  unsigned units;    // heads of all sequences times segments
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

// Runs of one type and kind of widths (cc3d_heads_linear_*.hip).  out: with
// outputs, else what each segment adds to the state; dec: with the decay's
// derivative.
using LinStart = int(LinArgs& a, int pad, bool out, bool dec, hipStream_t s);
LinStart linear_bf16_eights, linear_bf16_rest, linear_bf16_less, linear_f32_eights, linear_f32_rest, linear_f32_less;

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

// A value that is the same for all lanes, kept in a scalar register: arguments
// would be read from memory again wherever they are used.
__device__ __forceinline__ int pin(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float pin(float v) { return __uint_as_float(unsigned(pin(int(__float_as_uint(v))))); }
__device__ __forceinline__ int64_t pin(int64_t v) {
  return int64_t(uint64_t(unsigned(pin(int(uint64_t(v) >> 32)))) << 32 | unsigned(pin(int(uint64_t(v)))));
}
// (by way of the global address space, which an address made of a number has lost)
template <class T>
__device__ __forceinline__ T* pin(T* p) {
  return (T*)(__attribute__((address_space(1))) T*)(pin(int64_t(reinterpret_cast<intptr_t>(p))));
}

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

// How the widths C and E divide into eights.
enum {
  kEights,  // both are multiples of eight
  kRest,    // both are eight or more
  kLess     // one is less than eight
};

// Eight columns from `col` of rows `width` wide, zeros past it, loaded a block
// ahead: a load under a condition would be waited for where the branches meet, so
// every load is made, from the last valid token where there is no further one and
// from the row's last eight columns (before which the row, if not this part of it,
// has others) where it would leave the row; it is put right when it is used.
template <class T, int KIND>
struct Cols8 {
  int c, shift;  // where it is loaded, and how many elements too early; 8: all is zero
  __device__ __forceinline__ Cols8(int col, int width)
      : c(KIND == kLess ? col : min(col, width - 8)), shift(col >= width ? 8 : KIND == kRest ? col - c : 0) {}
  __device__ __forceinline__ Raw8<T> load(const T* row, int width) const {
    if constexpr (KIND == kLess) {
      Raw8<T> r;
#pragma unroll
      for (int j = 0; j < 8; ++j) set8(r, j, row[min(c + j, width - 1)]);
      return r;
    } else {
      return load8(row + c);
    }
  }
  __device__ __forceinline__ Raw8<T> finish(Raw8<T> v, bool on, int width) const {
    constexpr int kWords = int(sizeof(T)) * 2;
    unsigned w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = v.q[i / 4][i % 4];
    if constexpr (KIND == kRest) {
      auto down = [&](int words, bool by) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = by ? (i + words < kWords ? w[i + words] : 0u) : w[i];
      };
      if constexpr (sizeof(T) == 2) {
        down(2, shift & 4);
        down(1, shift & 2);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
          w[i] = shift & 1 ? (w[i] >> 16 | (i + 1 < kWords ? w[i + 1] << 16 : 0u)) : w[i];
      } else {
        down(4, shift & 4);
        down(2, shift & 2);
        down(1, shift & 1);
      }
    }
    on = on & (shift < 8);
#pragma unroll
    for (int i = 0; i < kWords; ++i) v.q[i / 4][i % 4] = on ? w[i] : 0u;
    if constexpr (KIND == kLess) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= width) set8(v, j, T(0));
    }
    return v;
  }
};

// Four columns of a result.
template <class T, int KIND>
__device__ __forceinline__ void store_cols(T* row, int col, int width, f32x4_s v) {
  if (KIND == kEights ? col < width : col + 4 <= width) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x2_by2*>(row + col) = u32x2_h{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
      *reinterpret_cast<u32x4_by4*>(row + col) = __builtin_bit_cast(u32x4_s, v);
    }
  } else if (KIND != kEights) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (col + i < width) row[col + i] = from_f32<T>(v[i]);
  }
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

template <class T, int DP, int KIND, bool OUT, bool DEC>
__global__ __launch_bounds__(cc3d::kLinThreads, DEC || sizeof(T) == 4 || DP == 256 ? 1 : 2) void linear_run(LinArgs a) {
  using M = Mat<T>;
  using L = LinTiles<T, DP, OUT, DEC>;
  using Frag = typename M::Frag;
  constexpr int kCols = L::kCols, kRowK = L::kRowK, kRowV = L::kRowV;
  constexpr int kMt = DP / 64, kNt = kCols / 16, kSteps = DP / 32;  // a wave's tiles of the state, steps of a sum over C
  constexpr int kVecK = DP / 32, kVecV = kCols / 32;                // eights of k and v that a thread stages
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int odd[2];  // a block of v holds an infinity or NaN
  T* lds = reinterpret_cast<T*>(smem);
  const int tid = threadIdx.x, lane = tid % 64, wave = pin(tid / 64), lane16 = lane % 16, quad = lane / 16;

  // Workgroups go to the eight dies in turn, each with a cache of its own: those
  // of one head and segment (its columns, its recurrences), which read the same
  // rows, follow each other on one die.
  const int starts = OUT ? a.segs : a.segs - 1;
  unsigned id = blockIdx.x / 8, unit = id / a.parts * 8 + blockIdx.x % 8;
  int block = int(id % a.parts), which = 0;
  while (which + 1 < a.runs && block >= a.run[which].blocks) block -= a.run[which++].blocks;
  if (unit >= a.units) return;
  const LinRun& r = a.run[which];
  const int blocks = r.blocks;
  const int turned = int(unit % starts);
  unit /= starts;
  const int h = pin(int(unit % a.heads)), n = pin(int(unit / a.heads));
  // (a reversed recurrence of the same rows is at the other end of its segments)
  const int s = pin(OUT && r.rev ? starts - 1 - turned : turned);
  const int64_t nh = int64_t(n) * a.heads + h;
  const int e0 = block * kCols;
  const int len = pin(valid_tokens(a.lengths, n, a.t));
  const int begin = s * a.seg, end = pin(min(begin + a.seg, len));
  const int c_all = pin(r.c), width = pin(min(kCols, r.e - e0));
  const int sc = pin(r.sc), se = pin(r.se), rev = pin(r.rev), r_lead = pin(r.lead);
  const float update = pin(r.update);

  const T* q = pin(static_cast<const T*>(r.q) + n * r.qb + int64_t(h / r.qper) * r.c);
  const T* k = pin(static_cast<const T*>(r.k) + n * r.kb + int64_t(h / r.kper) * r.c);
  const T* v = pin(static_cast<const T*>(r.v) + n * r.vb + int64_t(h / r.vper) * r.e + e0);
  const int64_t qr = pin(r.qr), kr = pin(r.kr), vr = pin(r.vr), o_row = pin(r.orow);
  const int64_t o_at = pin(n * r.ob + int64_t(h) * r.e + e0);
  char* o_p = pin(static_cast<char*>(r.o));
  const int o_f32 = pin(r.o_f32);
  // token p of the recurrence
  auto at = [&](int p) { return int64_t(rev ? len - 1 - p : p); };

  const float g = a.log_decay ? a.log_decay[h] : 0.f, g2 = g * kLog2e;
  const float whole_m1 = pin(fade_m1(g, kTok));

  // ---- the state before the segment, in the products' layout: element i of tile (mt, nt) is
  // c = 16 (wave kMt + mt) + 4 quad + i, e = 16 nt + lane16
  f32x4_s st[kMt][kNt], st2[DEC ? kMt : 1][DEC ? kNt : 1];
  // f(mt, nt, c, e): the four elements from c on of column e
  auto each_state = [&](auto&& f) {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) f(mt, nt, 16 * (wave * kMt + mt) + 4 * quad, 16 * nt + lane16);
  };
  // (unconditional loads, for the same reason as those of the rows)
  auto load_state = [&](const float* p, int c, int e) {
    f32x4_s v = zero4();
    if (!p) return v;
    const bool in = e < width;
    p += (e0 + min(e, width - 1)) * se;
    if (KIND == kEights && sc == 1) {
      v = __builtin_bit_cast(f32x4_s, *reinterpret_cast<const u32x4_by4*>(p + min(c, c_all - 4)));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (in & (c < c_all)) ? v[i] : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[min(c + i, c_all - 1) * sc];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (in & (c + i < c_all)) ? v[i] : 0.f;
    }
    return v;
  };
  auto store_state = [&](float* p, int c, int e, f32x4_s v) {
    if (!((e < width) & (c < c_all))) return;
    p += (e0 + e) * se + c * sc;
    if (KIND == kEights) {
      if (sc == 1) {
        *reinterpret_cast<u32x4_by4*>(p) = __builtin_bit_cast(u32x4_s, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i * sc] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < c_all) p[i * sc] = v[i];
    }
  };
  const int64_t size = int64_t(r.c) * r.e;
  const float* from = nullptr;
  if constexpr (OUT) from = s > 0 ? r.segs + (nh * (a.segs - 1) + s - 1) * size : r.from ? r.from + nh * size : nullptr;
  each_state([&](int mt, int nt, int c, int e) { st[mt][nt] = load_state(from, c, e); });
  if constexpr (DEC) {
    const float* from2 = OUT && s > 0 ? a.segs2 + (nh * (a.segs - 1) + s - 1) * size : nullptr;
    each_state([&](int mt, int nt, int c, int e) { st2[mt][nt] = load_state(from2, c, e); });
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
    const float score = pin(r.score), inter = pin(r.inter);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = i_tok - (16 * t + 4 * quad + i);
        near[t][i] = score * fade(g2, max(d, 0));
      }
    lead = inter * fade(g2, i_tok + r_lead);
  }

  // ---- rows of a block in flight
  Raw8<T> kn[kVecK], vn[kVecV], qn[OUT ? kSteps : 1], xn[DEC && OUT ? kCols / 32 : 1];
  f32x4_s xe[DEC && OUT ? kNt : 1];
  const int krow = tid / (DP / 8), vrow = tid / (kCols / 8);
  constexpr int kStepK = 256 / (DP / 8), kStepV = 256 / (kCols / 8);
  const Cols8<T, KIND> kc(tid % (DP / 8) * 8, c_all), vc(tid % (kCols / 8) * 8, width);
  const T* x = DEC && OUT ? static_cast<const T*>(a.x) + n * a.xb + int64_t(h / a.xper) * r.e + e0 : nullptr;
  auto fetch = [&](int p0) {
#pragma unroll
    for (int y = 0; y < kVecK; ++y) kn[y] = kc.load(k + at(min(p0 + krow + y * kStepK, end - 1)) * kr, c_all);
#pragma unroll
    for (int y = 0; y < kVecV; ++y) vn[y] = vc.load(v + at(min(p0 + vrow + y * kStepV, end - 1)) * vr, width);
    if constexpr (OUT) {
      const int64_t i = at(min(p0 + i_tok, end - 1));
#pragma unroll
      for (int y = 0; y < kSteps; ++y) qn[y] = Cols8<T, KIND>(32 * y + 8 * quad, c_all).load(q + i * qr, c_all);
      if constexpr (DEC) {
        const T* row = x + i * a.xr;
#pragma unroll
        for (int y = 0; y < kCols / 32; ++y) xn[y] = Cols8<T, KIND>(32 * y + 8 * quad, width).load(row, width);
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int y = 0; y < 4; ++y) xe[nt][y] = to_f32(row[min(16 * nt + 4 * quad + y, width - 1)]);
      }
    }
  };
  // the factors of f v: all blocks but the last are whole
  float fv[kVecV];
  auto factors = [&](int m) {
#pragma unroll
    for (int y = 0; y < kVecV; ++y) {
      const int left = m - 1 - (vrow + y * kStepV);
      const float f = update * fade(g2, max(left + 1 - r_lead, 0));
      fv[y] = left >= 0 ? f : 0.f;
    }
  };
  factors(kTok);
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
    for (int y = 0; y < kVecK; ++y) {
      const int j = krow + y * kStepK;
      M::put8(lds + L::kK + j * kRowK + tid % (DP / 8) * 8, kc.finish(kn[y], j < m, c_all));
    }
    if (m < kTok) factors(m);
    bool bad = false;
#pragma unroll
    for (int y = 0; y < kVecV; ++y) {
      const int j = vrow + y * kStepV, place = j * kRowV + tid % (kCols / 8) * 8;
      const Raw8<T> raw = vc.finish(vn[y], j < m, width);
      float f[8], f2[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = get8(raw, i);
        bad = bad | !(__builtin_fabsf(u) < __builtin_inff());
        f[i] = u * fv[y];
        f2[i] = f[i] * float(m - 1 - j);
      }
      T* p = lds + L::kF + place;
      constexpr int kOne = kTok * kRowV;
      M::put8_split(p, p + kOne, f);
      if constexpr (DEC) M::put8_split(p + kOne * M::kParts, p + kOne * (M::kParts + 1), f2);
      if constexpr (OUT) M::put8(lds + L::kV + place, raw);
    }
    Frag qf[OUT ? kSteps : 1], xf[DEC && OUT ? kCols / 32 : 1];
    f32x4_s xv[DEC && OUT ? kNt : 1];
    if constexpr (OUT) {
#pragma unroll
      for (int y = 0; y < kSteps; ++y) qf[y] = M::of(Cols8<T, KIND>(32 * y + 8 * quad, c_all).finish(qn[y], i_tok < m, c_all));
      if (bad) odd[turn] = 1;
    }
    if constexpr (DEC && OUT) {
#pragma unroll
      for (int y = 0; y < kCols / 32; ++y)
        xf[y] = M::of(Cols8<T, KIND>(32 * y + 8 * quad, width).finish(xn[y], i_tok < m, width));
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int y = 0; y < 4; ++y) xv[nt][y] = ((i_tok < m) & (16 * nt + 4 * quad + y < width)) ? xe[nt][y] : 0.f;
    }
    __syncthreads();
    if (p0 + kTok < end) fetch(p0 + kTok);

    if constexpr (OUT) {
      if (tid == 0) odd[turn ^ 1] = 0;
      if (16 * wave < m) {
        // ---- products q.k, transposed: element i of tile t is j = 16 t + 4 quad + i of the lane's token
        // (waves 0 and 1 need the first two tiles)
        f32x4_s pr[4] = {zero4(), zero4(), zero4(), zero4()};
        const T* krows = lds + L::kK + lane16 * kRowK + 8 * quad;
        auto scores = [&](auto first) {
          constexpr int t0 = decltype(first)::value;
#pragma unroll
          for (int y = 0; y < kSteps; ++y)
#pragma unroll
            for (int t = t0; t < t0 + 2; ++t) pr[t] = M::mma(M::row(krows + 16 * t * kRowK + 32 * y), qf[y], pr[t]);
        };
        scores(std::integral_constant<int, 0>());
        if (wave >= 2) scores(std::integral_constant<int, 2>());
        const T* state = lds + L::kS + lane16 * kRowK + 8 * quad;
        if constexpr (!DEC) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[t][i] = 16 * t + 4 * quad + i <= i_tok ? pr[t][i] * near[t][i] : 0.f;
          const Frag pf[2] = {M::of(pr[0], pr[1]), M::of(pr[2], pr[3])};
          f32x4_s o[kNt];
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) o[nt] = zero4();
#pragma unroll
          for (int y = 0; y < kSteps; ++y)
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) o[nt] = M::mma(M::row(state + 16 * nt * kRowK + 32 * y), qf[y], o[nt]);
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][i] *= lead;
          if (!odd[turn]) {
            const T* vt = M::col_at(lds + L::kV, kRowV, lane);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (y == 0 || wave >= 2) {
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
            const int64_t row = o_at + at(p0 + i_tok) * o_row;
            if (o_f32) {
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
                store_cols<float, KIND>(reinterpret_cast<float*>(o_p) + row, 16 * nt + 4 * quad, width, o[nt]);
            } else {
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
                store_cols<T, KIND>(reinterpret_cast<T*>(o_p) + row, 16 * nt + 4 * quad, width, o[nt]);
            }
          }
        } else {
          // ---- the decay's gradient: with x the rows of q, (i - j) f[i-j] (do[i] . v[j]) (x[i] . k[j]) of every pair
          // (here only these columns of x and k), and x[i] . f[i+1] (S2 + (i + 1) S) do[i]
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (t < 2 || wave >= 2) {
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
              const float term = lead * fmaf(float(i_tok + 1), w[i], u[i]) * xv[nt][i];
              sum += ((i_tok < m) & (16 * nt + 4 * quad + i < width)) ? term : 0.f;
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
  if (to) each_state([&](int mt, int nt, int c, int e) { store_state(to, c, e, st[mt][nt]); });
  if constexpr (DEC && !OUT) {
    float* to2 = a.segs2 + (nh * (a.segs - 1) + s) * size;
    each_state([&](int mt, int nt, int c, int e) { store_state(to2, c, e, st2[mt][nt]); });
  }
  if constexpr (OUT && !DEC) {
    const int last = min(begin + a.seg, a.t);
    for (int t = max(begin, len) + tid / kCols; t < last; t += cc3d::kLinThreads / kCols) {
      const int e = tid % kCols;
      const int64_t place = o_at + int64_t(t) * o_row + e;
      if (e < width) {
        if (o_f32) reinterpret_cast<float*>(o_p)[place] = 0.f;
        else reinterpret_cast<T*>(o_p)[place] = T(0);
      }
    }
  }
  if constexpr (OUT && DEC) {
    if (keeps) {
      const float* dto = a.dto + nh * size;
      each_state([&](int mt, int nt, int c, int e) {
        const f32x4_s v = load_state(dto, c, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) decay += ((c + i < c_all) & (e < width)) ? double(v[i]) * double(st2[mt][nt][i]) : 0.0;
      });
    }
    double* box = reinterpret_cast<double*>(smem);  // (the last barrier above is behind every read of the tiles)
    __syncthreads();
    box[tid] = decay;
    __syncthreads();
    for (int half = cc3d::kLinThreads / 2; half > 0; half /= 2) {
      if (tid < half) box[tid] += box[tid + half];
      __syncthreads();
    }
    if (tid == 0) a.part[(nh * a.segs + s) * blocks + block] = box[0];
  }
}

template <class T, int DP, int KIND, bool OUT, bool DEC>
int start_run(const LinArgs& a, int64_t workgroups, hipStream_t s) {
  constexpr int lds = LinTiles<T, DP, OUT, DEC>::kBytes;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_run<T, DP, KIND, OUT, DEC>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return int(e);
    }
  }
  return launch(linear_run<T, DP, KIND, OUT, DEC>, workgroups, cc3d::kLinThreads, lds, s, a);
}

template <class T, int KIND>
int start_runs(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  const int starts = out ? a.segs : a.segs - 1;
  a.parts = 0;
  for (int i = 0; i < a.runs; ++i) a.parts += a.run[i].blocks = int(cc3d::linear_blocks(a.run[i].e, pad));
  a.units = unsigned(int64_t(a.n) * a.heads * starts);
  if (a.units == 0) return 0;
  const int64_t workgroups = (int64_t(a.units) + 7) / 8 * 8 * a.parts;
  auto go = [&](auto d) {
    constexpr int DP = decltype(d)::value;
    if (out)
      return dec ? start_run<T, DP, KIND, true, true>(a, workgroups, s) : start_run<T, DP, KIND, true, false>(a, workgroups, s);
    return dec ? start_run<T, DP, KIND, false, true>(a, workgroups, s) : start_run<T, DP, KIND, false, false>(a, workgroups, s);
  };
  if (pad == 64) return go(std::integral_constant<int, 64>());
  if (pad == 128) return go(std::integral_constant<int, 128>());
  return go(std::integral_constant<int, 256>());
}

}  // namespace
