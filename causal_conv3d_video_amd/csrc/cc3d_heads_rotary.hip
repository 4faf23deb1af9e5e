// Rotary positions of the heads of q and k.
//
//   a' = A (a cos - b sin);  b' = A (a sin + b cos)      by position * f[j] for pair j
//
// One read and one write of everything and a few operations an element: bound by
// memory (8192 tokens of 20 heads of 128, bf16, 84 MB, in 18 us).  A workgroup takes a few tokens.  The angles of a token are those of all
// its heads, so they are computed once, in LDS: in turns, position * (f / 2 pi) in
// 64 bits, of which the whole part is dropped before anything is rounded to 32.
#include <algorithm>

#include "cc3d_heads_internal.h"
#include "cc3d_seq_device.h"

namespace {

struct RotaryArgs {
  const void* in[2];
  void* out[2];
  int64_t ib[2], ir[2], ob[2], orow[2];
  int heads[2];
  const int *positions, *offsets, *lengths;
  int64_t all;  // N T
  int t, d, rot, first, tokens, interleaved;
  float amplitude, sign;
  double turns[128];
};

// The angles of a workgroup's tokens, [tokens][rot / 2].  What rounding a half turn to 32 bits
// leaves, up to pi 2^-25 of an angle, is added back to its sine and cosine for fp32 heads (results 3.9e-8 off 64 bits without).
template <class T>
__device__ __forceinline__ void angles(const RotaryArgs& a, float2* table, int64_t tok0, int tokens) {
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < tokens * half; i += cc3d::kRotaryThreads) {
    const int x = i / half, j = i - x * half;
    const int64_t tok = tok0 + x, n = tok / a.t, t = tok - n * a.t;
    const int64_t pos = a.positions ? int64_t(a.positions[tok]) : (a.offsets ? int64_t(a.offsets[n]) : 0) + t;
    double turns = double(pos) * a.turns[j];
    turns -= rint(turns);
    float s, c;
    const float half_turns = float(2.0 * turns);
    sincospif(half_turns, &s, &c);
    if constexpr (sizeof(T) == 4) {
      const float left = 3.14159265f * float(2.0 * turns - double(half_turns)), near = s;
      s = fmaf(c, left, s);
      c = fmaf(-near, left, c);
    }
    table[i] = float2{c * a.amplitude, s * a.amplitude * a.sign};
  }
  __syncthreads();
}

// All borders at multiples of eight channels: a thread takes eight channels that
// are passed on, eight pairs of the half layout or four of the interleaved one.
template <class T>
__global__ __launch_bounds__(cc3d::kRotaryThreads) void rotary_wide(RotaryArgs a) {
  extern __shared__ __attribute__((aligned(16))) float2 table[];
  const int half = a.rot / 2, tid = threadIdx.x;
  const int64_t tok0 = int64_t(blockIdx.x) * a.tokens;
  const int tokens = int(min(int64_t(a.tokens), a.all - tok0));
  angles<T>(a, table, tok0, tokens);
  const int turned = a.interleaved ? a.rot / 8 : a.rot / 16;
  const int per = turned + (a.d - a.rot) / 8;
  const int each = per * (a.heads[0] + a.heads[1]);
  const int step_head = cc3d::kRotaryThreads / per, step_piece = cc3d::kRotaryThreads - step_head * per;
  for (int x = 0; x < tokens; ++x) {
    const int64_t tok = tok0 + x, n = tok / a.t, t = tok - n * a.t;
    const bool on = !a.lengths || t < a.lengths[n];
    const float2* cs = table + x * half;
    int head = tid / per, piece = tid - head * per;
    for (int i = tid; i < each; i += cc3d::kRotaryThreads) {
      const int w = head >= a.heads[0], h = w ? head - a.heads[0] : head;
      const T* p = static_cast<const T*>(a.in[w]) + n * a.ib[w] + t * a.ir[w] + int64_t(h) * a.d;
      T* q = static_cast<T*>(a.out[w]) + n * a.ob[w] + t * a.orow[w] + int64_t(h) * a.d;
      if (piece >= turned) {
        int c = (piece - turned) * 8;
        if (c >= a.first) c += a.rot;
        Raw8<T> v = on ? load8(p + c) : zero8<T>();
        using Q = typename Quad<T>::type;
#pragma unroll
        for (int k = 0; k < int(sizeof(T) / 2); ++k) reinterpret_cast<Q*>(q + c)[k] = v.q[k];
      } else if (a.interleaved) {
        const int c = a.first + piece * 8;
        const Raw8<T> v = on ? load8(p + c) : zero8<T>();
        float o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = cs[piece * 4 + k];
          const float u = get8(v, 2 * k), z = get8(v, 2 * k + 1);
          o[2 * k] = on ? u * f.x - z * f.y : 0.f;
          o[2 * k + 1] = on ? u * f.y + z * f.x : 0.f;
        }
        store8(q + c, o);
      } else {
        const int c = a.first + piece * 8;
        const Raw8<T> v = on ? load8(p + c) : zero8<T>(), y = on ? load8(p + c + half) : zero8<T>();
        float o[8], r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = cs[piece * 8 + k];
          const float u = get8(v, k), z = get8(y, k);
          o[k] = on ? u * f.x - z * f.y : 0.f;
          r[k] = on ? u * f.y + z * f.x : 0.f;
        }
        store8(q + c, o);
        store8(q + c + half, r);
      }
      head += step_head;
      piece += step_piece;
      if (piece >= per) {
        piece -= per;
        ++head;
      }
    }
  }
}

// Any borders: whole heads, kRotaryRow channels of them and fewer, pass through LDS
// on their way, so that memory is read and written eight channels at a time wherever
// pairs lie.  (Everything of a piece is read before any of it is written: an output
// may be its input.)  2 by 2049 tokens of 40 fp32 heads of 100, half of each turned:
// 4-byte accesses, pair by pair, took 54 us where this takes 32 us (a whole pass).
template <class T>
__global__ __launch_bounds__(cc3d::kRotaryThreads) void rotary_odd(RotaryArgs a) {
  extern __shared__ __attribute__((aligned(16))) float2 table[];
  __shared__ __attribute__((aligned(16))) float row[cc3d::kRotaryRow];
  const int half = a.rot / 2, tid = threadIdx.x;
  const int64_t tok0 = int64_t(blockIdx.x) * a.tokens;
  const int tokens = int(min(int64_t(a.tokens), a.all - tok0));
  angles<T>(a, table, tok0, tokens);
  const int at_once = cc3d::kRotaryRow / a.d;  // heads
  for (int x = 0; x < tokens; ++x) {
    const int64_t tok = tok0 + x, n = tok / a.t, t = tok - n * a.t;
    const bool on = !a.lengths || t < a.lengths[n];
    const float2* cs = table + x * half;
    for (int w = 0; w < 2; ++w)
      for (int h0 = 0; h0 < a.heads[w]; h0 += at_once) {
        const int el = min(at_once, a.heads[w] - h0) * a.d;
        const T* p = static_cast<const T*>(a.in[w]) + n * a.ib[w] + t * a.ir[w] + int64_t(h0) * a.d;
        T* q = static_cast<T*>(a.out[w]) + n * a.ob[w] + t * a.orow[w] + int64_t(h0) * a.d;
        if (on)
          for (int i = tid * 8; i < el; i += cc3d::kRotaryThreads * 8) {
            const Raw8<T> v = i + 8 <= el ? load8(p + i) : load_some(p + i, el - i);
#pragma unroll
            for (int j = 0; j < 8; ++j) row[i + j] = get8(v, j);
          }
        __syncthreads();
        for (int i = tid * 8; i < el; i += cc3d::kRotaryThreads * 8) {
          const int h = i / a.d;
          int c = i - h * a.d, base = i - c;
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = c - a.first;  // of the turned channels
            const bool turns = (r >= 0) & (r < a.rot);
            const bool second = a.interleaved ? r & 1 : r >= half;
            const int pair = a.interleaved ? r >> 1 : second ? r - half : r;
            const int apart = a.interleaved ? 1 : half;
            const float2 f = cs[turns ? pair : 0];
            // (past the piece's end: whatever the row's last elements are)
            const float own = row[min(base + c, cc3d::kRotaryRow - 1)];
            const float other = row[turns ? min(base + c + (second ? -apart : apart), cc3d::kRotaryRow - 1) : 0];
            const float turned = second ? other * f.y + own * f.x : own * f.x - other * f.y;
            o[j] = on ? (turns ? turned : own) : 0.f;
            if (++c == a.d) {
              c = 0;
              base += a.d;
            }
          }
          if (i + 8 <= el) store8(q + i, o);
          else store_some(q + i, el - i, o);
        }
        __syncthreads();
      }
  }
}

}  // namespace

namespace cc3d {

int launch_rotary(const cc3d_rotary_plan& p, const cc3d_rotary_args_t& c, bool backward, void* stream) {
  const auto& d = p.d;
  RotaryArgs a{};
  const cc3d_rows_t in[2] = {c.q, c.k}, out[2] = {c.q_out, c.k_out};
  for (int w = 0; w < 2; ++w) {
    a.in[w] = in[w].p;
    a.out[w] = out[w].p;
    a.ib[w] = in[w].batch;
    a.ir[w] = in[w].row;
    a.ob[w] = out[w].batch;
    a.orow[w] = out[w].row;
  }
  a.heads[0] = d.q_heads;
  a.heads[1] = d.k_heads;
  a.positions = c.positions;
  a.offsets = c.offsets;
  a.lengths = c.lengths;
  a.all = int64_t(d.n) * d.t;
  a.t = d.t;
  a.d = d.d;
  a.rot = d.rot;
  a.first = d.first;
  a.tokens = p.tokens;
  a.interleaved = d.layout == CC3D_ROTARY_INTERLEAVED;
  a.amplitude = float(d.amplitude);
  a.sign = backward ? -1.f : 1.f;
  std::copy(p.turns, p.turns + d.rot / 2, a.turns);
  const bool wide = d.d % 8 == 0 && d.first % 8 == 0 && d.rot % (a.interleaved ? 8 : 16) == 0;
  const int64_t workgroups = (a.all + p.tokens - 1) / p.tokens;
  const int lds = p.tokens * d.rot / 2 * int(sizeof(float2));
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto* kernel) { return launch(kernel, workgroups, kRotaryThreads, lds, s, a); };
  if (d.dtype == CC3D_BF16) return wide ? go(&rotary_wide<bf16_s>) : go(&rotary_odd<bf16_s>);
  return wide ? go(&rotary_wide<float>) : go(&rotary_odd<float>);
}

}  // namespace cc3d
