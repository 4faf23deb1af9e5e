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
// A workgroup walks a segment of the time axis with the state of one head in
// registers, as the 32 by 32 results of matrix products (fp32): 32 columns of E and
// all of C a wave, or half of C (SPLIT).  What is multiplied again never passes through
// LDS on its way: the eight results of a lane in 16 rows are made neighbours by the
// order in which rows and columns are read (`place`), so that a lane's results,
// rounded, are its operand of the next product.  That holds for the state, which
// meets q from registers, and for the products q.k, which only go to LDS because
// all waves want those that one computed.  Operands whose tokens lie along the
// registers are read from LDS with the transposing load.  The next block's rows load
// while one is computed.
//
// Two waves with half of C each hand each other their sums over it (q S of a tile
// of 32 tokens, through LDS) and finish one tile of tokens each.  Both round f v, but
// with two waves a SIMD one computes while the other waits: 2048 tokens of 256 heads
// of 64 took 106 us with a wave for all of C and take 82; of 64 by 128 the decay's
// recurrences, 2 by 2049 tokens of 16 heads, 37 and 43 us and 32 each.  Heads of 128 by
// 128 do so where there is a workgroup a compute unit at most (8192 tokens of 16 heads in 77
// us instead of 79, 512 of 256 heads 46 instead of 50): two workgroups of four
// waves do better than one of eight (512 tokens of 1024 heads, 145 us and 181).
// Runs without outputs have nothing to hand over and little to wait for.
//
// With tiles of 16 by 16, the state's copy in LDS and each wave with 16 tokens of a
// block, a compute unit took 4.7 us for 64 tokens of a 128 by 128 head with its
// operands in cache: LDS, vector and matrix units one after the other, some 3 to
// 4 thousand cycles each.  Tiles of 32 by 32 read half as much from LDS.
//
// Few heads leave compute units idle, so the time axis is split: linear_run
// without outputs gives what each segment adds to the state, linear_join carries
// the states across, and linear_run starts each segment from its own.
//
// Rounding.  bf16 operands of a product are exact; what is computed and then
// multiplied again is rounded: f (q.k) to bf16 (half a step, 2^-8 at most, beside the
// result's own), the state to bf16 for the product with q (the same).  Outputs are so 0.0023
// from 64 bits where rounding them alone makes 0.0017, which they would be with both in
// two parts: 8192 tokens of 16 heads of 128 in 84 us instead of 77, 2048 tokens of 256 heads of
// 64 in 91 instead of 79, and 2 by 2049 tokens backward in 163 instead of 131 (a workgroup a
// compute unit less for LDS).  What is added
// to a state, f v, is kept whole, as three bf16: a state is an fp32 result and is
// carried (as two, 2^-18 each, 8192 tokens of 16 heads of 128 took 78
// instead of 83 us and a state was 1.6e-6 off).  The decay's gradient, fp32 too, takes
// the state as three bf16 as well and multiplies both products of its pairs in fp32.  fp32 tensors
// use the fp32 matrix products throughout.
//
// The decay's gradient is the sum over all blocks of what depends on g there, S the
// state before the block and G the gradient of the state behind it:
//
//   sum over i > j of (i-j) f[i-j] scale (q[i] . k[j]) (do[i] . v[j])  +
//   sum over i of (i+1) f[i+1] scale q[i] S do[i]  +  m f[m] <S, G>  +  sum over j of (m-1-j) f[m-1-j] k[j] G v[j]
//
// The first two fall out of dq's recurrence, the last out of dk's; for <S, G> dq's
// leaves every block's S behind, as its registers hold it, and dk's, which has the
// same rows of tokens in reverse, reads it.  (The derivative of the state carried
// along beside it, which needs neither, doubles the products and the registers: 170 of
// 240 us of a backward pass of 2 by 2049 tokens.)
#pragma once
#include <algorithm>

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
  const float* from;                         // state before the first token (reversed: behind the last), or null
  float* to;                                 // after the last valid one (reversed: before the first), or null
  float* segs;                               // [N][H][segments - 1]: states between segments
  // with the decay's gradient: rows that the part of the state that came in meets; whether pairs count here
  const void* x;
  int64_t xb, xr;
  int xper, pairs;
  float* put;        // each block's state before it, as registers hold it
  const float* get;  // the same of another recurrence, which meets this one's
  double* part;      // [N][H][segments][blocks]
};

struct LinArgs {
  LinRun run[3];
  int runs, parts;   // parts: workgroups of all runs that share a head and segment
  unsigned units;    // heads of all sequences times segments
  int n, heads, t, seg, segs;
  const float* log_decay;
  const int* lengths;
};

// Runs of one type and kind of widths (cc3d_heads_linear_*.hip).  out: with
// outputs, else what each segment adds to the state; dec: with the decay's
// gradient.
using LinStart = int(LinArgs& a, int pad, bool out, bool dec, hipStream_t s);
LinStart linear_bf16_eights, linear_bf16_rest, linear_bf16_less, linear_f32_eights, linear_f32_rest, linear_f32_less;

}  // namespace cc3d

namespace {

using cc3d::LinArgs;
using cc3d::LinRun;

typedef __bf16 bf16x8_h __attribute__((ext_vector_type(8)));
typedef short s16x4_h __attribute__((ext_vector_type(4)));
typedef float f32x16_h __attribute__((ext_vector_type(16)));

__device__ __forceinline__ int valid_tokens(const int* lengths, int n, int t) {
  return lengths ? min(max(lengths[n], 0), t) : t;
}

// exp(g d), 1 where d is zero even for g = -inf; g2 = g log2(e).
__device__ __forceinline__ float fade(float g2, int d) { return d == 0 ? 1.f : __builtin_amdgcn_exp2f(g2 * float(d)); }
// exp(g d) in 64 bits.
__device__ __forceinline__ double fade64(float g, int d) { return d == 0 ? 1.0 : exp(double(g) * d); }
// Whether an infinite state stays one: as long as a token's factor is more than zero, also where that of many is not.
__device__ __forceinline__ bool lasting(float g) { return __builtin_amdgcn_exp2f(g * kLog2e) > 0.f; }

// What a state is multiplied by at its blocks.  A factor of 32 bits is up to 2^-25 off, the
// same way at every block, so each takes back what those before it were off: together they
// are never off by more.  (S + S (exp(g d) - 1) is as good beside 1, but 2^-25 of S off whatever
// is left of it; a factor in two parts costs a multiplication more for each element, 4% of
// a prompt of 8192 tokens of 16 heads of 128.)  Where 32 bits hold none, the factor is the
// least number there is, which an infinite state survives (a choice for each element instead
// is a second copy of the state in registers: 4% there, 11% of a backward call of heads of 256).
struct Fades {
  float hi, lo, inverse;  // of a whole block, in two parts
  float last;             // of the block that may be less
  float drift = 0.f;      // of the factors so far, relative
  // (an exponential in 64 bits costs a short call's workgroups 1% and more: only those that are used)
  __device__ __forceinline__ Fades(float g, int whole, int rest, bool more) : hi(0.f), lo(0.f), inverse(0.f) {
    const float least = lasting(g) ? 0x1p-149f : 0.f;
    if (more || rest == whole) {
      const double f = fade64(g, whole);
      hi = float(f);
      if (hi < least) hi = least;
      if (f > 1e-30 && f < 1e30) {
        lo = float(f - double(hi));
        inverse = __builtin_amdgcn_rcpf(hi);
      }
    }
    last = rest == whole ? hi : float(fade64(g, rest));
    if (last < least) last = least;
  }
  __device__ __forceinline__ float next(bool is_whole) {
    if (!is_whole) return last;
    const float f = hi + fmaf(-hi, drift, lo);
    drift = fmaf((f - hi) - lo, inverse, drift);
    return f;
  }
};

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
__device__ __forceinline__ f32x16_h zero16() { return f32x16_h(0.f); }

// Two values rounded in one instruction.
typedef __bf16 bf16x2_h __attribute__((ext_vector_type(2)));
typedef float f32x2_h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2_h{lo, hi}, bf16x2_h));
}

// What rounding v to hi leaves; nothing where that is an infinity (the median of
// r, 0 and r is r, but 0 where r is no number).
__device__ __forceinline__ float rest(float v, float hi) { return __builtin_amdgcn_fmed3f(v - hi, 0.f, v - hi); }

// Two values as sums of three bf16 each: rounded, the rest rounded, and what that
// leaves (24 bits hold three times eight).
__device__ __forceinline__ void split2(float v, float w, unsigned (&part)[3]) {
  part[0] = pack2(v, w);
  v = rest(v, __uint_as_float(part[0] << 16));
  w = rest(w, __uint_as_float(part[0] & 0xffff0000u));
  part[1] = pack2(v, w);
  part[2] = pack2(v - __uint_as_float(part[1] << 16), w - __uint_as_float(part[1] & 0xffff0000u));
}

// Row (or column) m of 32 of a product's result holds place(m) of what it is
// computed from.  A lane has the results m = 8 (r / 4) + 4 h + r % 4 of its column
// (r of 16 registers, h its half of the wave), so place(m) = 16 (r / 8) + 8 h + r % 8:
// eight neighbours in registers 0..7, the eight 16 on in 8..15.
__device__ __forceinline__ int place(int m) { return m / 16 * 16 + m % 8 / 4 * 8 + m % 16 / 8 * 4 + m % 4; }

// Operands of the matrix products: 16 terms of a sum for 32 rows, eight a lane
// (row lane % 32, terms 8 (lane / 32) .. + 7).
template <class T>
struct Mat;

template <>
struct Mat<bf16_s> {
  using Frag = bf16x8_h;
  // Elements between rows beside their own.  Rows of 16 bytes for 16 lanes meet all 64 banks where rows
  // are an odd number of 16 bytes apart, and the transposing loads (four rows of 64 bytes) meet no bank
  // more than twice where that is 12 or 36 words (of 64).
  static constexpr int kPad = 8;
  static constexpr int pad_both(int width) { return width % 128 == 0 ? 24 : 8; }
  static constexpr int kParts = 3;  // of what is rounded on its way into a state
  static __device__ __forceinline__ f32x16_h mma(Frag a, Frag b, f32x16_h c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Frag row(const bf16_s* p) {
    return __builtin_bit_cast(Frag, *reinterpret_cast<const u32x4_s*>(p));
  }
  // eight rows from 8 h on of column place(lane % 32): p is the lane's place among the four rows of 16
  // columns that its 16 lanes read together
  static __device__ __forceinline__ const bf16_s* col_at(const bf16_s* tile, int stride, int lane) {
    const int chunk = lane % 4;  // of four columns: the middle ones change places
    return tile + (lane / 32 * 8 + lane % 16 / 4) * stride + lane % 32 / 16 * 16 + 4 * (chunk % 2 * 2 + chunk / 2);
  }
  static __device__ __forceinline__ s16x4_h col4(const bf16_s* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4_h*)(const_cast<bf16_s*>(p)));
  }
  static __device__ __forceinline__ Frag col(const bf16_s* p, int stride) {
    const s16x4_h a = col4(p), b = col4(p + 4 * stride);
    return __builtin_bit_cast(Frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // results 8 g .. 8 g + 7, rounded
  template <int g>
  static __device__ __forceinline__ Frag of(const f32x16_h& v) {
    return __builtin_bit_cast(Frag, u32x4_s{pack2(v[8 * g], v[8 * g + 1]), pack2(v[8 * g + 2], v[8 * g + 3]),
                                            pack2(v[8 * g + 4], v[8 * g + 5]), pack2(v[8 * g + 6], v[8 * g + 7])});
  }
  template <int g>
  static __device__ __forceinline__ void split(const f32x16_h& v, Frag (&out)[kParts]) {
    u32x4_s part[kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned w[kParts];
      split2(v[8 * g + 2 * i], v[8 * g + 2 * i + 1], w);
#pragma unroll
      for (int x = 0; x < kParts; ++x) part[x][i] = w[x];
    }
#pragma unroll
    for (int x = 0; x < kParts; ++x) out[x] = __builtin_bit_cast(Frag, part[x]);
  }
  // f[i] times the eight terms, in kParts
  static __device__ __forceinline__ void scaled(Frag v, const float (&f)[8], Frag (&out)[kParts]) {
    const u32x4_s w = __builtin_bit_cast(u32x4_s, v);
    u32x4_s part[kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned u[kParts];
      split2(__uint_as_float(w[i] << 16) * f[2 * i], __uint_as_float(w[i] & 0xffff0000u) * f[2 * i + 1], u);
#pragma unroll
      for (int x = 0; x < kParts; ++x) part[x][i] = u[x];
    }
#pragma unroll
    for (int x = 0; x < kParts; ++x) out[x] = __builtin_bit_cast(Frag, part[x]);
  }
  static __device__ __forceinline__ void put(bf16_s* p, Frag v) { *reinterpret_cast<u32x4_s*>(p) = __builtin_bit_cast(u32x4_s, v); }
  static __device__ __forceinline__ void put(bf16_s* p, const Raw8<bf16_s>& r) { *reinterpret_cast<u32x4_s*>(p) = r.q[0]; }
  // not zero where an element's exponent is full: an infinity or no number
  static __device__ __forceinline__ unsigned full(const Raw8<bf16_s>& r) {
    unsigned v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) v |= (r.q[0][i] & 0x7f807f80u) + 0x00800080u;
    return v & 0x80008000u;
  }
  // zeros in the place of those
  static __device__ __forceinline__ Frag finite(Frag v) {
    u32x4_s w = __builtin_bit_cast(u32x4_s, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~((((w[i] & 0x7f807f80u) + 0x00800080u) >> 15 & 0x00010001u) * 0xffffu);
    return __builtin_bit_cast(Frag, w);
  }
};

template <>
struct Mat<float> {
  struct Frag {
    float x[8];
  };
  static constexpr int kPad = 4;
  static constexpr int pad_both(int) { return 4; }
  static constexpr int kParts = 1;
  // (the eight products take the lanes' terms one after another: any order of the 16 does)
  static __device__ __forceinline__ f32x16_h mma(const Frag& a, const Frag& b, f32x16_h c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x[i], b.x[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag row(const float* p) {
    Raw8<float> r;
    r.q[0] = reinterpret_cast<const u32x4_s*>(p)[0];
    r.q[1] = reinterpret_cast<const u32x4_s*>(p)[1];
    return __builtin_bit_cast(Frag, r);
  }
  static __device__ __forceinline__ const float* col_at(const float* tile, int stride, int lane) {
    return tile + lane / 32 * 8 * stride + place(lane % 32);
  }
  static __device__ __forceinline__ Frag col(const float* p, int stride) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.x[i] = p[i * stride];
    return f;
  }
  template <int g>
  static __device__ __forceinline__ Frag of(const f32x16_h& v) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.x[i] = v[8 * g + i];
    return f;
  }
  template <int g>
  static __device__ __forceinline__ void split(const f32x16_h& v, Frag (&out)[kParts]) {
    out[0] = of<g>(v);
  }
  static __device__ __forceinline__ void scaled(const Frag& v, const float (&f)[8], Frag (&out)[kParts]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[0].x[i] = v.x[i] * f[i];
  }
  static __device__ __forceinline__ void put(float* p, const Frag& v) { put(p, __builtin_bit_cast(Raw8<float>, v)); }
  static __device__ __forceinline__ void put(float* p, const Raw8<float>& r) {
    reinterpret_cast<u32x4_s*>(p)[0] = r.q[0];
    reinterpret_cast<u32x4_s*>(p)[1] = r.q[1];
  }
  static __device__ __forceinline__ unsigned full(const Raw8<float>& r) {
    unsigned v = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v |= (r.q[i / 4][i % 4] & 0x7f800000u) + 0x00800000u;
    return v & 0x80000000u;
  }
  static __device__ __forceinline__ Frag finite(Frag v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[i] = __builtin_fabsf(v.x[i]) < __builtin_inff() ? v.x[i] : 0.f;
    return v;
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
  __device__ __forceinline__ Raw8<T> load(const T* p, int width) const {  // p: at column c of a row
    if constexpr (KIND == kLess) {
      Raw8<T> r;
#pragma unroll
      for (int j = 0; j < 8; ++j) set8(r, j, p[min(c + j, width - 1) - c]);
      return r;
    } else {
      return load8(p);
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

// Eight columns of a result.
template <class T, int KIND>
__device__ __forceinline__ void store_cols(T* row, int col, int width, const float* v) {
  if (KIND == kEights ? col < width : col + 8 <= width) {
    using Q = typename Quad<T>::type;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<Q*>(row + col) = u32x4_s{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    } else {
      store8(row + col, v);
    }
  } else if (KIND != kEights && col < width) {
    store_some(row + col, width - col, v);
  }
}

// LDS of a workgroup, in elements of T: rows of q, of k and of v, the products q.k
// as operands; with the decay's gradient, rows of x.
template <class T, int DP, int CB, int TOK, int SPLIT, bool OUT, bool DEC>
struct LinTiles {
  using M = Mat<T>;
  static constexpr int kRowQ = DP + M::kPad, kRowK = DP + M::pad_both(DP), kRowV = CB + M::pad_both(CB);
  static constexpr int kK = 0, kV = kK + TOK * kRowK, kQ = kV + TOK * kRowV, kP = kQ + (OUT ? TOK * kRowQ : 0);
  static constexpr int kPairs = TOK == 64 ? 3 : 1;  // tiles of 32 by 32 pairs of tokens
  static constexpr int kX = kP + (OUT ? kPairs * 2 * 64 * 8 : 0);
  static constexpr int kE = kX + (DEC ? TOK * kRowV : 0);  // tiles that two waves hand each other
  static constexpr int kTotal = kE + (SPLIT > 1 ? CB / 32 * SPLIT * 1024 * 4 / int(sizeof(T)) : 0);
  static constexpr int kBytes = kTotal * int(sizeof(T)) > 4096 ? kTotal * int(sizeof(T)) : 4096;
};

template <class T, int DP, int CB, int TOK, int KIND, int SPLIT, bool OUT, bool DEC>
__global__ __launch_bounds__(2 * CB * SPLIT, (sizeof(T) == 2 ? 2 : 1)) void linear_run(LinArgs a) {
  using M = Mat<T>;
  using Frag = typename M::Frag;
  using L = LinTiles<T, DP, CB, TOK, SPLIT, OUT, DEC>;
  constexpr int kThreads = 2 * CB * SPLIT, kWaves = CB / 32 * SPLIT, kRowQ = L::kRowQ, kRowK = L::kRowK, kRowV = L::kRowV;
  constexpr int kSteps = DP / 16, kMt = DP / 32 / SPLIT, kIt = TOK / 32, kTs = TOK / 16;  // steps of C, a wave's tiles; of the tokens
  constexpr int kOwn = SPLIT == 1 ? kIt : 1;  // tiles of tokens whose results are the wave's
  constexpr int kVecK = TOK * DP / 8 / kThreads, kVecV = TOK * CB / 8 / kThreads;  // eights that a thread stages
  constexpr int kStepK = kThreads / (DP / 8), kStepV = kThreads / (CB / 8);
  static_assert(kVecK * kThreads * 8 == TOK * DP && kVecV * kThreads * 8 == TOK * CB, "threads");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int odd[2];  // a block of v holds an infinity or NaN
  T* lds = reinterpret_cast<T*>(smem);
  const int tid = threadIdx.x, lane = tid % 64, wave = pin(tid / 64), il = lane % 32, hh = lane / 32;
  const int cw = wave / SPLIT, half = wave % SPLIT, c_half = half * (kMt * 32);  // its columns, its part of C
  const bool own = SPLIT == 1 || kIt > 1 || half == 0;
  auto tile = [&](int x) { return SPLIT == 1 ? x : kIt > 1 ? half : 0; };

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
  const int s = pin(int(unit % starts) + (!OUT && r.rev ? 1 : 0));
  unit /= starts;
  const int h = pin(int(unit % a.heads)), n = pin(int(unit / a.heads));
  const int64_t nh = int64_t(n) * a.heads + h;
  const int e0 = block * CB;
  const float g = a.log_decay ? a.log_decay[h] : 0.f;  // (in flight beside the length: the first rows wait for both)
  const int len = pin(valid_tokens(a.lengths, n, a.t));
  const int begin = s * a.seg, end = pin(min(begin + a.seg, len));
  const int c_all = pin(r.c), width = pin(min(CB, r.e - e0));
  const int sc = pin(r.sc), se = pin(r.se), rev = pin(r.rev), r_lead = pin(r.lead);

  // Rows of a block are at 32-bit offsets from its first token; a place may be up to
  // seven elements before a row's (Cols8), so offsets count from eight before.
  constexpr unsigned kBias = KIND == kRest ? 8 : 0, kSize = sizeof(T);
  const T* q = pin(static_cast<const T*>(r.q) + n * r.qb + int64_t(h / r.qper) * r.c - kBias);
  const T* k = pin(static_cast<const T*>(r.k) + n * r.kb + int64_t(h / r.kper) * r.c - kBias);
  const T* v = pin(static_cast<const T*>(r.v) + n * r.vb + int64_t(h / r.vper) * r.e + e0 - kBias);
  const T* x = nullptr;
  if constexpr (DEC) x = pin(static_cast<const T*>(r.x) + n * r.xb + int64_t(h / r.xper) * r.e + e0 - kBias);
  const int qr = pin(int(r.qr)), kr = pin(int(r.kr)), vr = pin(int(r.vr)), o_row = pin(int(r.orow)), xr = DEC ? pin(int(r.xr)) : 0;
  char* o_p = pin(static_cast<char*>(r.o));
  const int64_t o_at = pin(n * r.ob + int64_t(h) * r.e + e0);
  const int o_f32 = pin(r.o_f32), pairs = DEC ? pin(r.pairs) : 0;
  float* put = DEC ? pin(r.put) : nullptr;
  const float* get = DEC ? pin(r.get) : nullptr;
  auto by = [](const T* p, unsigned bytes) { return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + bytes); };

  // ---- rows of a block in flight.  A block of m < TOK tokens has them as its last rows, behind rows of zeros.
  Raw8<T> kn[kVecK], vn[kVecV], qn[OUT ? kVecK : 1], xn[DEC ? kVecV : 1];
  const int krow = tid / (DP / 8), kcol = tid % (DP / 8) * 8, vrow = tid / (CB / 8), vcol = tid % (CB / 8) * 8;
  const Cols8<T, KIND> kc(kcol, c_all), vc(vcol, width);
  auto fetch = [&](int p0, int blk) {
    const int m = min(blk, end - p0);
    const int64_t t = p0;
    const T *kb = k + t * kr, *vb = v + t * vr;
    auto place_of = [&](int j, int stride, const Cols8<T, KIND>& c) {
      const int tok = max(j - (TOK - m), 0);
      return (unsigned(rev ? m - 1 - tok : tok) * unsigned(stride) + unsigned(c.c) + kBias) * kSize;
    };
#pragma unroll
    for (int y = 0; y < kVecK; ++y) kn[y] = kc.load(by(kb, place_of(krow + y * kStepK, kr, kc)), c_all);
#pragma unroll
    for (int y = 0; y < kVecV; ++y) vn[y] = vc.load(by(vb, place_of(vrow + y * kStepV, vr, vc)), width);
    if constexpr (OUT) {
      const T* qb = q + t * qr;
#pragma unroll
      for (int y = 0; y < kVecK; ++y) qn[y] = kc.load(by(qb, place_of(krow + y * kStepK, qr, kc)), c_all);
    }
    if constexpr (DEC) {
      const T* xb = x + t * xr;
#pragma unroll
      for (int y = 0; y < kVecV; ++y) xn[y] = vc.load(by(xb, place_of(vrow + y * kStepV, xr, vc)), width);
    }
  };
  // Blocks of the segment's tokens, from the last one where time is reversed.  Where states grow so fast that
  // products of three factors over 64 tokens may be no fp32 numbers, a block has fewer tokens (and `apart` is the
  // farthest that two of them are): rows of zeros in front of them are to stay zeros, whatever they are multiplied
  // by.  With the decay's gradient, whose states lie TOK tokens apart, those products are held at `top`
  // instead where those of valid tokens are within it.
  const float g2 = g * kLog2e;
  const int all = max(end - begin, 0);
  int blk = TOK, apart = TOK;
  float top = __builtin_inff();
  if constexpr (DEC) {
    if (g2 * float(min(all, TOK)) < 126.f) top = 0x1.fffffep127f;
    if (g2 != g2) top = g2;
  } else if (g2 * float(TOK) > 36.f) {
    blk = pin(max(int(36.f / g2), 1));
    apart = blk - 1;
  }
  auto held = [&](float f) { return DEC ? __builtin_amdgcn_fmed3f(f, -top, top) : f; };
  const int count = blk == TOK ? (all + TOK - 1) / TOK : (all + blk - 1) / blk;
  const int first = begin + (rev ? (count - 1) * blk : 0), step = rev ? -blk : blk;
  if (count > 0) fetch(first, blk);

  // ---- the state before the segment: result i of tile mt is c = 32 mt + 16 (i / 8) + 8 hh + i % 8 of the lane's column
  f32x16_h st[kMt];
  const int col = 32 * cw + place(il);  // of the lane
  const bool has = 32 * cw < width;     // the wave has columns
  // (unconditional loads, for the same reason as those of the rows)
  auto load_state = [&](const float* p, f32x16_h (&v)[kMt]) {
    const bool in = col < width;
    p += (e0 + min(col, width - 1)) * se;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int c = c_half + 32 * mt + 16 * g + 8 * hh;
        if (KIND == kEights && sc == 1) {
          const u32x4_by4* w = reinterpret_cast<const u32x4_by4*>(p + min(c, c_all - 8));
          const f32x4_s lo = __builtin_bit_cast(f32x4_s, w[0]), hi = __builtin_bit_cast(f32x4_s, w[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[mt][8 * g + i] = (in & (c < c_all)) ? lo[i] : 0.f;
            v[mt][8 * g + 4 + i] = (in & (c < c_all)) ? hi[i] : 0.f;
          }
        } else {
          float u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = p[min(c + i, c_all - 1) * sc];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[mt][8 * g + i] = (in & (c + i < c_all)) ? u[i] : 0.f;
        }
      }
  };
  auto store_state = [&](float* p, const f32x16_h (&v)[kMt]) {
    if (col >= width) return;
    p += (e0 + col) * se;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int c = c_half + 32 * mt + 16 * g + 8 * hh;
        if (KIND == kEights) {
          if (c >= c_all) continue;
          if (sc == 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              reinterpret_cast<u32x4_by4*>(p + c)[i] =
                  __builtin_bit_cast(u32x4_s, f32x4_s{v[mt][8 * g + 4 * i], v[mt][8 * g + 4 * i + 1], v[mt][8 * g + 4 * i + 2],
                                                      v[mt][8 * g + 4 * i + 3]});
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[(c + i) * sc] = v[mt][8 * g + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < c_all) p[(c + i) * sc] = v[mt][8 * g + i];
        }
      }
  };
  const int64_t size = int64_t(r.c) * r.e;
  const float* from = nullptr;
  const int slot = rev ? s : s - 1;  // of the state before the segment
  if constexpr (OUT)
    from = slot >= 0 && slot < a.segs - 1 ? r.segs + (nh * (a.segs - 1) + slot) * size : r.from ? r.from + nh * size : nullptr;
  if (from && has) {
    load_state(from, st);
  } else {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) st[mt] = zero16();
  }

  // ---- factors, all of them f of a number of tokens, never of less than none.  Token j of a block (from its end)
  // adds f[TOK-1-j] = f[16 (TOK/16-1-j/16)] f[15-j%16], and tokens i of the second tile and j of the first are
  // f[il+1] f[31-jl] apart: a few by step, in scalar registers, times a few by lane.
  Fades fades(g, blk, count > 0 ? all - (count - 1) * blk : 0, count > 1);
  fades.hi = pin(fades.hi);
  fades.lo = pin(fades.lo);
  fades.inverse = pin(fades.inverse);
  fades.last = pin(fades.last);
  float fq[8], diag[OUT ? 16 : 1], f_lane = 0.f, f_step[kTs];
#pragma unroll
  for (int b = 0; b < 8; ++b) fq[b] = fade(g2, min(15 - 8 * hh - b, apart));
#pragma unroll
  for (int y = 0; y < kTs; ++y) f_step[y] = pin(fade(g2, min(16 * y, apart)));
  const float f_last = pin(r.update) * fade(g2, 1 - r_lead), inter = pin(r.inter), score = pin(r.score);
  if constexpr (OUT) {
#pragma unroll
    for (int b = 0; b < 16; ++b) diag[b] = held(score * fade(g2, min(max(il - (16 * (b / 8) + 8 * hh + b % 8), 0), apart)));
    f_lane = score * fade(g2, min(il + 1, apart));
  }
  if (tid < 2) odd[tid] = 0;
  __syncthreads();

  double decay = 0.0;
  const bool keeps = OUT ? (rev ? s == 0 : s + 1 == a.segs) && r.to : true;  // the state after the segment is asked for
  int turn = 0;
  for (int b0 = 0, p0 = first; b0 < count; ++b0, p0 += step, turn ^= 1) {
    const int m = min(blk, end - p0), none = TOK - m;
    const bool more = b0 + 1 < count;
    // (what follows from these is cheap, and would be kept in registers over all blocks)
    asm volatile("" : "+v"(fq[0]), "+v"(fq[1]), "+v"(fq[2]), "+v"(fq[3]), "+v"(fq[4]), "+v"(fq[5]), "+v"(fq[6]), "+v"(fq[7]));
    // ---- stage the rows
    const bool whole = m == TOK && c_all == DP && width == CB;  // nothing to put right
    unsigned full = 0;
#pragma unroll
    for (int y = 0; y < kVecK; ++y) {
      const int j = krow + y * kStepK;
      if (!whole) kn[y] = kc.finish(kn[y], j >= none, c_all);
      M::put(lds + L::kK + j * kRowK + kcol, kn[y]);
      if constexpr (OUT) {
        if (!whole) qn[y] = kc.finish(qn[y], j >= none, c_all);
        M::put(lds + L::kQ + j * kRowQ + kcol, qn[y]);
      }
    }
#pragma unroll
    for (int y = 0; y < kVecV; ++y) {
      const int j = vrow + y * kStepV;
      if (!whole) vn[y] = vc.finish(vn[y], j >= none, width);
      if constexpr (OUT) full |= M::full(vn[y]);
      M::put(lds + L::kV + j * kRowV + vcol, vn[y]);
      if constexpr (DEC) {
        if (!whole) xn[y] = vc.finish(xn[y], j >= none, width);
        M::put(lds + L::kX + j * kRowV + vcol, xn[y]);
      }
    }
    if (OUT && full) odd[turn] = 1;
    __syncthreads();
    if (more) fetch(p0 + step, blk);
    const bool strange = pin(odd[turn]) != 0;

    const T* q_row = lds + L::kQ + il * kRowQ + 8 * hh;
    if constexpr (OUT) {
      // ---- products q.k of 32 by 32 tokens (second tile by first, and both by themselves), transposed, a wave each in turn:
      // result b is token j = 16 (b / 8) + 8 hh + b % 8 of its tile, of the lane's token
      float sum = 0.f;
#pragma unroll
      for (int p = 0; p < (L::kPairs + kWaves - 1) / kWaves; ++p) {
        const int pair = p * kWaves + wave, it = pair > 0, jt = pair > 1;
        if (pair >= L::kPairs) break;
        f32x16_h pr = zero16();
        const T *kp = lds + L::kK + (32 * jt + place(il)) * kRowK + 8 * hh, *qp = q_row + 32 * it * kRowQ;
#pragma unroll
        for (int y = 0; y < kSteps; ++y) pr = M::mma(M::row(kp + 16 * y), M::row(qp + 16 * y), pr);
        if (pair == 1) {
#pragma unroll
          for (int b = 0; b < 16; ++b) pr[b] *= held(f_lane * f_step[1 - b / 8] * fq[b % 8]);
        } else {
#pragma unroll
          for (int b = 0; b < 16; ++b) pr[b] = 16 * (b / 8) + 8 * hh + b % 8 <= il ? pr[b] * diag[b] : 0.f;
        }
        T* at = lds + L::kP + (pair * 128 + lane) * 8;
        M::put(at, M::template of<0>(pr));
        M::put(at + 512, M::template of<1>(pr));
        if constexpr (DEC) {
          // the decay's gradient: (i - j) f[i-j] (q[i] . k[j]) (x[i] . v[j]) of every pair (of these columns of x and v)
          if (pairs) {
            f32x16_h xv = zero16();
            const T *vp = lds + L::kV + (32 * jt + place(il)) * kRowV + 8 * hh, *xp = lds + L::kX + (32 * it + il) * kRowV + 8 * hh;
#pragma unroll
            for (int y = 0; y < CB / 16; ++y) xv = M::mma(M::row(vp + 16 * y), M::row(xp + 16 * y), xv);
#pragma unroll
            for (int b = 0; b < 16; ++b) {
              const int d = 32 * (it - jt) + il - (16 * (b / 8) + 8 * hh + b % 8);
              const float term = float(d) * pr[b] * xv[b];
              sum += d > 0 ? term : 0.f;
            }
          }
        }
      }
      // ---- f[i+1] q S
      // (a wave's part of C, of its own tile of tokens and of the other one's, which the other wave of its columns gets)
      f32x16_h o[kOwn], give;
      float* box = reinterpret_cast<float*>(lds + L::kE);
      if (has) {
#pragma unroll
        for (int x = 0; x < kOwn; ++x) o[x] = zero16();
        give = zero16();
#pragma unroll
        for (int y = 0; y < kSteps / SPLIT; ++y) {
          Frag sf[M::kParts];
          if constexpr (DEC) {
            if (y % 2) M::template split<1>(st[y / 2], sf);
            else M::template split<0>(st[y / 2], sf);
          } else {
            sf[0] = y % 2 ? M::template of<1>(st[y / 2]) : M::template of<0>(st[y / 2]);
          }
          const T* qp = q_row + c_half + 16 * y;
#pragma unroll
          for (int part = 0; part < (DEC ? M::kParts : 1); ++part) {
#pragma unroll
            for (int x = 0; x < kOwn; ++x) o[x] = M::mma(sf[part], M::row(qp + 32 * tile(x) * kRowQ), o[x]);
            if constexpr (SPLIT > 1 && kIt > 1) give = M::mma(sf[part], M::row(qp + 32 * (1 - half) * kRowQ), give);
          }
        }
        if (SPLIT > 1 && (kIt > 1 || half == 1)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x16_h& g = kIt > 1 ? give : o[0];
            *reinterpret_cast<f32x4_s*>(box + wave * 1024 + (i * 64 + lane) * 4) = f32x4_s{g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]};
          }
        }
      }
      if constexpr (DEC) {
        // the state that another recurrence had here
        if (has) {
          const int64_t at = (((nh * ((a.t + TOK - 1) / TOK) + p0 / TOK) * blocks + block) * kWaves + wave) * (kMt * 1024) + lane * 4;
          if (put) {
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4_s*>(put + at + (mt * 4 + i) * 256) =
                    f32x4_s{st[mt][4 * i], st[mt][4 * i + 1], st[mt][4 * i + 2], st[mt][4 * i + 3]};
          }
          if (get) {
            float met = 0.f;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const f32x4_s u = *reinterpret_cast<const f32x4_s*>(get + at + (mt * 4 + i) * 256);
#pragma unroll
                for (int j = 0; j < 4; ++j) met = fmaf(u[j], st[mt][4 * i + j], met);
              }
            sum += float(m) * (m == TOK ? fades.hi : fades.last) * met;
          }
        }
      }
      __syncthreads();
      if (tid == 0) odd[turn ^ 1] = 0;
      if (has && own) {
        if constexpr (SPLIT > 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4_s u = *reinterpret_cast<const f32x4_s*>(box + (wave ^ 1) * 1024 + (i * 64 + lane) * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[0][4 * i + j] += u[j];
          }
        }
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
          const float lead = inter * fade(g2, max(32 * tile(x) + il - none + r_lead, 0));
#pragma unroll
          for (int b = 0; b < 16; ++b) o[x][b] *= lead;
        }
        if constexpr (DEC) {
          // the decay's gradient: what came in, by the tokens since
#pragma unroll
          for (int x = 0; x < kOwn; ++x) {
            const int it = tile(x);
            const T* xrow = lds + L::kX + (32 * it + il) * kRowV + 32 * cw + 8 * hh;
            const int tok = 32 * it + il - none;
            float met = 0.f;
#pragma unroll
            for (int b = 0; b < 16; ++b) met = fmaf(o[x][b], to_f32(xrow[16 * (b / 8) + b % 8]), met);
            sum += tok >= 0 ? float(tok + r_lead) * met : 0.f;
          }
        }
      }
      if constexpr (DEC) decay += double(sum);
      if (has && own && o_p) {
        // ---- the products meet v
        const T* vt = M::col_at(lds + L::kV, kRowV, lane) + 32 * cw;
        const T* pp = lds + L::kP + lane * 8;
        auto meet = [&](auto&& get) {
#pragma unroll
          for (int y = 0; y < kTs; ++y) {
            if (SPLIT > 1 && y >= 2 && half == 0) break;
            const Frag vf = get(M::col(vt + 16 * y * kRowV, kRowV));
#pragma unroll
            for (int x = 0; x < kOwn; ++x)
              if (y < 2 || tile(x)) o[x] = M::mma(vf, M::row(pp + (y + 2 * tile(x)) * 512), o[x]);
          }
        };
        if (!strange) {
          meet([](Frag f) { return f; });
        } else {
          // An infinity or NaN among the block's v meets no product of an earlier token, not even a zero one: zero in the
          // sums for all, and added by itself to the tokens from its own on.
          meet([](Frag f) { return M::finite(f); });
#pragma unroll
          for (int x = 0; x < kOwn; ++x)
            for (int j = 0; j < 32 * tile(x) + 32; ++j) {
              const int it = tile(x);
              const int jl = j % 32, pair = it + j / 32;
              if (j > 32 * it + il) continue;
              const float p = to_f32(lds[L::kP + ((pair * 2 + jl / 16) * 64 + jl % 16 / 8 * 32 + il) * 8 + j % 8]);
              const T* row = lds + L::kV + j * kRowV + 32 * cw + 8 * hh;
#pragma unroll
              for (int b = 0; b < 16; ++b) {
                const float u = to_f32(row[16 * (b / 8) + b % 8]);
                if (!(__builtin_fabsf(u) < __builtin_inff())) o[x][b] = fmaf(p, u, o[x][b]);
              }
            }
        }
        const int64_t t = o_at + int64_t(p0) * o_row;
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
          const int it = tile(x);
          const int tok = 32 * it + il - none;
          if (tok < 0) continue;
          const int64_t at = t + int64_t(unsigned(rev ? m - 1 - tok : tok) * uint64_t(o_row));
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = o[x][8 * g + i];
            const int e = 32 * cw + 16 * g + 8 * hh;
            if (o_f32) store_cols<float, KIND>(reinterpret_cast<float*>(o_p) + at, e, width, u);
            else store_cols<T, KIND>(reinterpret_cast<T*>(o_p) + at, e, width, u);
          }
        }
      }
    }
    if (!(more || keeps)) break;  // (for all threads of the workgroup)

    // ---- the state after the block, 16 tokens at a time
    if (has) {
      const float fade_st = pin(fades.next(m == blk));
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int b = 0; b < 16; ++b) st[mt][b] *= fade_st;
      const T* kt = M::col_at(lds + L::kK, kRowK, lane) + c_half;
      const T* vt = M::col_at(lds + L::kV, kRowV, lane) + 32 * cw;
#pragma unroll
      for (int y = 0; y < kTs; ++y) {
        const Frag vf = M::col(vt + 16 * y * kRowV, kRowV);
        float fy[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) fy[i] = held(fq[i] * (f_step[kTs - 1 - y] * f_last));
        Frag f[M::kParts];
        M::scaled(vf, fy, f);
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          const Frag kf = M::col(kt + 16 * y * kRowK + 32 * mt, kRowK);
#pragma unroll
          for (int part = 0; part < M::kParts; ++part) st[mt] = M::mma(kf, f[part], st[mt]);
        }
      }
    }
    __syncthreads();
  }

  // ---- what is left behind: the state, zeros for the tokens that are not valid, the decay's sum
  float* to = nullptr;
  if constexpr (OUT) to = keeps && r.to ? r.to + nh * size : nullptr;
  else to = r.segs + (nh * (a.segs - 1) + (rev ? s - 1 : s)) * size;
  if (to && has) store_state(to, st);
  if (OUT && o_p) {
    const int last = min(begin + a.seg, a.t);
    for (int t = max(begin, len) + tid / CB; t < last; t += kThreads / CB) {
      const int e = tid % CB;
      const int64_t place = o_at + int64_t(t) * o_row + e;
      if (e < width) {
        if (o_f32) reinterpret_cast<float*>(o_p)[place] = 0.f;
        else reinterpret_cast<T*>(o_p)[place] = T(0);
      }
    }
  }
  if constexpr (DEC) {
    double* box = reinterpret_cast<double*>(smem);
    __syncthreads();
    box[tid] = decay;
    __syncthreads();
    for (int half = kThreads / 2; half > 0; half /= 2) {
      if (tid < half) box[tid] += box[tid + half];
      __syncthreads();
    }
    if (tid == 0) r.part[(nh * a.segs + s) * blocks + block] = box[0];
  }
}

template <class T, int DP, int CB, int TOK, int KIND, int SPLIT, bool OUT, bool DEC>
int start_run(const LinArgs& a, int64_t workgroups, hipStream_t s) {
  constexpr int lds = LinTiles<T, DP, CB, TOK, SPLIT, OUT, DEC>::kBytes;
  static_assert(lds + 8 <= 160 * 1024, "LDS of a compute unit");
  constexpr auto kernel = linear_run<T, DP, CB, TOK, KIND, SPLIT, OUT, DEC>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return int(e);
    }
  }
  return launch(kernel, workgroups, 2 * CB * SPLIT, lds, s, a);
}

template <class T, int KIND>
int start_runs(LinArgs& a, int pad, bool out, bool dec, hipStream_t s) {
  const int starts = out ? a.segs : a.segs - 1;
  int widest = 0;
  for (int i = 0; i < a.runs; ++i) widest = std::max(widest, a.run[i].e);
  const int cols = cc3d::linear_cols(widest);
  a.parts = 0;
  for (int i = 0; i < a.runs; ++i) a.parts += a.run[i].blocks = (a.run[i].e + cols - 1) / cols;
  a.units = unsigned(int64_t(a.n) * a.heads * starts);
  if (a.units == 0) return 0;
  const int64_t workgroups = (int64_t(a.units) + 7) / 8 * 8 * a.parts;
  auto go = [&](auto d, auto c) {
    constexpr int DP = decltype(d)::value, CB = decltype(c)::value, TOK = cc3d::linear_tokens(sizeof(T), DP);
    if (!out) return start_run<T, DP, CB, TOK, KIND, 1, false, false>(a, workgroups, s);
    // (a block of 32 tokens in place of one of 64: 17 tokens of 1560 sequences, 6 heads of 64, in 87 us instead
    // of 109; of 128 sequences, 16 heads of 128, in 68 instead of 75; with the decay's gradient 6 of 977, 6 heads of 16
    // by 50, in 174 instead of 258, 4 of 1541, 6 heads of 16 by 64 in fp32, in 491 instead of 972)
    if constexpr (DP <= 128) {
      if (a.t <= cc3d::kLinFew)
        return dec ? start_run<T, DP, CB, 32, KIND, 1, true, true>(a, workgroups, s)
                   : start_run<T, DP, CB, 32, KIND, 1, true, false>(a, workgroups, s);
    }
    if (dec) {
      // (128 by 128 in fp32 leave no room for the handed tiles)
      constexpr int kSplit = LinTiles<T, DP, CB, TOK, 2, true, true>::kBytes + 8 <= 160 * 1024 ? 2 : 1;
      return start_run<T, DP, CB, TOK, KIND, kSplit, true, true>(a, workgroups, s);
    }
    if constexpr (sizeof(T) == 2 && DP == 128 && CB == 128) {
      if (workgroups > cc3d::kLinUnits) return start_run<T, DP, CB, TOK, KIND, 1, true, false>(a, workgroups, s);
    }
    return start_run<T, DP, CB, TOK, KIND, 2, true, false>(a, workgroups, s);
  };
  const std::integral_constant<int, 64> c64;
  const std::integral_constant<int, 128> c128;
  const std::integral_constant<int, 256> c256;
  if (pad == 64) return cols == 64 ? go(c64, c64) : go(c64, c128);
  if (pad == 128) return cols == 64 ? go(c128, c64) : go(c128, c128);
  return cols == 64 ? go(c256, c64) : go(c256, c128);
}

}  // namespace
