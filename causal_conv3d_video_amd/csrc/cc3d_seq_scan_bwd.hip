// Selective state space scan, backward.
//
//   g[t] = C gy[t] + exp(delta[t+1] A) g[t+1],  gy = dy silu(z)
//   du = D gy + delta sum g B;   ddelta = sum g (A exp(delta A) h[t-1] + u B)
//   dA = sum g delta exp(delta A) h[t-1];  dB = sum_channels g delta u;  dC = sum_channels gy h
//
// The states are not kept by the forward pass: the time axis is cut into
// chunks of 64 tokens, the forward and the reverse recurrence are carried
// across them as in the forward pass, and a workgroup then takes one chunk of
// its channels at a time, independent of every other.  It walks the chunk
// forward, leaving the state before every eight tokens in LDS, and then back,
// eight tokens at a time: the eight decays and decayed states are made again
// into registers and the gradient walks over them.
//
// Two kinds of sums cross: over states (du, ddelta, dz) and over channels (dB,
// dC).  A lane holds two channels by four states, so most of either is added
// inside it; four groups of 16 lanes hold different states.  What is left goes
// across lanes by halving, each step adding two registers' halves into one:
// the sums over states of four tokens end in the four lane groups, one token
// each (which is also the group that loads that token's inputs and stores its
// results), those over channels one value a lane.  Waves of other channels add
// their dB and dC in LDS, and each workgroup writes one row of partial sums a
// token, added in the tiles' order by a last small kernel.
//
// Measured, bf16, 2 x 2049 tokens of 2048 channels, 16 states: 247 us (in a
// kernel trace, whose durations add up to more: scan_carry 63, scan_join 11, this
// kernel 178, bc_sum and sum_rows 6 each).
// 31 vector instructions a channel, token and state bound it: vector units busy
// 69% at the two waves a SIMD that its 256 registers allow (some still spill).
// The bytes alone would take 25 us at a large copy's rate.  One channel and eight
// states a lane, every decay of eight tokens kept, spilled and took 1707 us.
#include "cc3d_seq_scan.h"

#include <algorithm>

namespace {

__device__ __forceinline__ float swap32_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Lanes without `bit` keep x and receive the partner's x, the others y.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x, float y, bool bit) {
  const float keep = bit ? y : x, send = bit ? x : y;
  return keep + dpp<CTRL>(send);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kRor8 = 0x128;

// The sums of eight values over aligned groups of LC lanes.  Lane bits say
// which value a lane ends with, highest bit of the value first: bits 5, 4, 3
// (LC = 64), 4, 3, 2 (32) or 3, 2, 1 (16); the lower ones hold copies.
// (Mirroring eight lanes pairs lanes of different bit 2; it also turns the
// bits below, over which everything is summed afterwards.)
template <int LC>
__device__ __forceinline__ float reduce8(const float (&in)[8], int lane) {
  float v[4], w[2], r;
  if constexpr (LC == 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = swap32_add(in[i], in[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = swap16_add(v[i], v[i + 2]);
    r = dpp_add<kRor8>(w[0], w[1], lane & 8);
    r += dpp<kMirror8>(r);
    r += dpp<kXor1>(r);
    r += dpp<kXor2>(r);
  } else if constexpr (LC == 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = swap16_add(in[i], in[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = dpp_add<kRor8>(v[i], v[i + 2], lane & 8);
    r = dpp_add<kMirror8>(w[0], w[1], lane & 4);
    r += dpp<kXor1>(r);
    r += dpp<kXor2>(r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = dpp_add<kRor8>(in[i], in[i + 4], lane & 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = dpp_add<kMirror8>(v[i], v[i + 2], lane & 4);
    r = dpp_add<kXor2>(w[0], w[1], lane & 2);
    r += dpp<kXor1>(r);
  }
  return r;
}

// Sums over the SG lane groups of one value of each of SG tokens: group q
// ends with token q's.
template <int SG>
__device__ __forceinline__ float sum_groups(const float (&v)[SG]) {
  if constexpr (SG == 4) return swap16_add(swap32_add(v[0], v[2]), swap32_add(v[1], v[3]));
  else if constexpr (SG == 2) return swap32_add(v[0], v[1]);
  else return v[0];
}

// Two neighbouring channels as they are stored; aligned to one (as 16-byte
// accesses, 4- and 8-byte ones lose little off their alignment).
typedef unsigned unsigned_by2 __attribute__((aligned(2)));
typedef unsigned long long ulong_by4 __attribute__((aligned(4)));

template <class T>
struct Pair {
  using U = std::conditional_t<sizeof(T) == 4, unsigned long long, unsigned>;
  using Mem = std::conditional_t<sizeof(T) == 4, ulong_by4, unsigned_by2>;
  U v;
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(unsigned(v >> (32 * i)));
    else return __uint_as_float(i ? v & 0xffff0000u : v << 16);
  }
};

// DUO: there are two channels; otherwise the one stands for both.
template <class T, bool DUO>
__device__ __forceinline__ Pair<T> load_pair(const T* p) {
  using P = Pair<T>;
  P r;
  if constexpr (DUO) {
    r.v = *reinterpret_cast<const typename P::Mem*>(p);
  } else if constexpr (sizeof(T) == 4) {
    r.v = __float_as_uint(*p) * 0x100000001ull;
  } else {
    r.v = *p * 0x10001u;
  }
  return r;
}

// Stores the channels that are this lane's own: both, the second, or none
// (DUO); the first or none.
template <class T, bool DUO>
__device__ __forceinline__ void store_pair(T* p, float x, float y, bool own0, bool own1) {
  using P = Pair<T>;
  if constexpr (!DUO) {
    if (own0) p[0] = from_f32<T>(x);
  } else if (own0) {
    typename P::U v;
    if constexpr (sizeof(T) == 4) v = __float_as_uint(x) | typename P::U(__float_as_uint(y)) << 32;
    else v = pack_bf16(x, y);
    *reinterpret_cast<typename P::Mem*>(p) = v;
  } else if (own1) {
    p[1] = from_f32<T>(y);
  }
}

// LDS of a workgroup, in floats.
template <int SG, int SUB>
struct BwdLds {
  static constexpr int kChan = 128 / SG;                // channels of a wave
  static constexpr int kTok = 3 * SUB * kChan;          // delta, delta u, gy of SUB tokens
  static constexpr int kBc = 2 * SUB * 4 * SG;          // B and C of SUB tokens
  static constexpr int kComb = SUB * 8 * SG;            // dB and dC of SUB tokens
  static constexpr int kMeet = 6 * 64 * (SUB / SG);     // sums over states, when waves share channels
  int kept, per_wave, comb, meet, total;
  __host__ __device__ BwdLds(int chunk, int waves, int wc) {
    kept = (chunk / SUB - 1) * 8 * 64;  // states before every SUB tokens but the last
    per_wave = kept + kTok + kBc;
    comb = waves * wc * per_wave;
    meet = comb + 2 * waves * wc * kComb;
    total = meet + (waves > 1 ? 2 * waves * wc * kMeet : 0);
  }
};

// A view of the kernel's arguments, read again from where they lie: kept in
// scalar registers the ten views spill into lanes of vector registers, and
// some 200 of a walk's 2100 vector instructions only moved them.
struct FreshRows {
  uintptr_t p;
  int64_t batch, row;
};
__device__ __forceinline__ FreshRows fresh(unsigned offset) {
  auto base = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(base));  // not the same address as before, for all the compiler knows
  auto q = (const __attribute__((address_space(4))) int64_t*)(base + offset);
  return {uintptr_t(q[0]), q[1], q[2]};
}

template <class T, int SG, int SUB, bool MULTI, bool DUO>
__global__ __launch_bounds__(256, 2) void scan_bwd(ScanArgs a, int wc) {
  using L = BwdLds<SG, SUB>;
  constexpr int LC = 64 / SG, CT = 2 * LC, NB = SUB / SG, kDup = LC / 8, kVal = 8 * SG;
  constexpr int kBcEach = (L::kBc + 63) / 64;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int waves = MULTI ? a.waves : 1;
  const L at(a.chunk, waves, wc);
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int sw = MULTI ? wave % waves : 0, cw = MULTI ? wave / waves : wave;
  const int q = lane / LC, l = lane % LC;
  const int tiles = a.tiles_per_group * a.groups, tile = blockIdx.x % tiles, worker = blockIdx.x / tiles;
  const int group = tile / a.tiles_per_group;
  // Channels chan and chan + 1.  In a group of odd width the last lane's first
  // channel is also the lane's before it, and not its own; lanes past the
  // group own none.
  const int in_group = ((tile - group * a.tiles_per_group) * wc + cw) * CT + 2 * l;
  const int chan = group * a.wide + (DUO ? min(in_group, a.wide - 2) : 0), other = DUO ? 1 : 0;
  const bool own[2] = {in_group < a.wide && (!DUO || in_group + 1 < a.wide), DUO && in_group < a.wide};
  const int channels = a.groups * a.wide;
  const int s0 = sw * 4 * SG + q * 4;  // this lane's first state
  f32x4_s* kept = reinterpret_cast<f32x4_s*>(lds + wave * at.per_wave) + lane;
  float* tok = lds + wave * at.per_wave + at.kept;
  float* bc = tok + L::kTok;
  // where this lane's sums over channels go: kDup tokens a store, one for each
  // copy; [channel wave][token][state wave][which][4 SG]
  const int copy = lane & (kDup - 1), value = l / kDup;
  const int comb_at = (cw * SUB + copy) * waves * kVal + sw * kVal + (value >> 2) * (4 * SG) + q * 4 + (value & 3);

  float bias[2], skip[2], a2[2][4], da[2][4] = {}, dd[2] = {}, dbias[2] = {};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    bias[c] = a.bias ? a.bias[chan + c * other] : 0.f;
    skip[c] = a.d ? a.d[chan + c * other] : 0.f;
    const float* p = a.a + int64_t(chan + c * other) * a.s + s0;
    if (a.s % 4 == 0 && reinterpret_cast<uintptr_t>(a.a) % 16 == 0) {
      const f32x4_s v = s0 < a.s ? *reinterpret_cast<const f32x4_s*>(p) : f32x4_s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) a2[c][i] = rate_of(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) a2[c][i] = s0 + i < a.s ? rate_of(p[i]) : 0.f;
    }
  }
  // (a branch costs more here than what it saves: flags select)
  const bool soft = a.softplus, gated = a.z.p != nullptr;
  const bool has_du = a.du.p != nullptr, has_ddt = a.ddt.p != nullptr, has_dz = a.dz.p != nullptr;
  const ScanRows& zrows = gated ? a.z : a.dy;
  // this lane's places behind a walk's first token: its own tokens' channel
  // pair in every stream (token q of each SG), and its share of B and C
  auto own_at = [&](const ScanRows& v) { return unsigned(q) * unsigned(v.row) + unsigned(chan); };
  const unsigned o_dt = own_at(a.dt), o_u = own_at(a.u), o_z = own_at(zrows), o_dy = own_at(a.dy);
  const unsigned o_du = own_at(a.du), o_ddt = own_at(a.ddt), o_dz = own_at(a.dz);
  unsigned o_bc[kBcEach];
  int t_bc[kBcEach];  // its token of the walk; none of it where there is no such state
#pragma unroll
  for (int r = 0; r < kBcEach; ++r) {
    const int i = lane + 64 * r, which = i / (L::kBc / 2), t = i / (4 * SG) % SUB, s = i % (4 * SG);
    const bool in = i < L::kBc && sw * 4 * SG + s < a.s;
    o_bc[r] = in ? unsigned(t) * unsigned(which ? a.c.row : a.b.row) + unsigned(s) : 0;
    t_bc[r] = in ? t : SUB;
  }
  int turn = 0;

  for (int64_t item = worker; item < int64_t(a.n) * a.chunks; item += a.workers) {
    const int n = int(item / a.chunks), ch = int(item - int64_t(n) * a.chunks);
    const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
    const int subs = te > t0 ? (te - t0 + SUB - 1) / SUB : 0;
    // a walk's first token: the same address for the whole wave
    struct Walk {
      T* p;
      int64_t row;
    };
    auto walk = [&](unsigned offset, int k) -> Walk {
      const FreshRows v = fresh(offset);
      return {reinterpret_cast<T*>(v.p) + int64_t(n) * v.batch + int64_t(t0 + k * SUB) * v.row, v.row};
    };
    float* pbc = a.part_bc + (int64_t(tile) * a.n + n) * a.t * waves * kVal;

    // Inputs of the tokens of one walk: this lane group's tokens, and this
    // lane's share of B and C.  For tokens past the valid ones the walk's first
    // is read (and not used).
    Pair<T> rdt[NB], ru[NB], rz[NB], rdy[NB];
    T rbc[kBcEach];
    auto fetch = [&](int k, auto back) {
      const int there = te - t0 - k * SUB;  // at least one
      const Walk dt = walk(offsetof(ScanArgs, dt), k), u = walk(offsetof(ScanArgs, u), k);
      const T* bp = walk(offsetof(ScanArgs, b), k).p + group * a.s + sw * 4 * SG;
      const T* cp = walk(offsetof(ScanArgs, c), k).p + group * a.s + sw * 4 * SG;
      Walk z{}, dy{};
      if constexpr (back.value) {
        dy = walk(offsetof(ScanArgs, dy), k);
        z = walk(gated ? offsetof(ScanArgs, z) : offsetof(ScanArgs, dy), k);
      }
      auto at_token = [&](const Walk& v, unsigned o, int b) { return load_pair<T, DUO>(v.p + int64_t(b * SG) * v.row + o); };
      if (there >= SUB) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          rdt[b] = at_token(dt, o_dt, b);
          ru[b] = at_token(u, o_u, b);
          if constexpr (back.value) {
            rz[b] = at_token(z, o_z, b);
            rdy[b] = at_token(dy, o_dy, b);
          }
        }
#pragma unroll
        for (int r = 0; r < kBcEach; ++r) {
          // (whole rows of 64 lanes are B or C alike, but for a single one)
          const bool which = kBcEach == 1 ? lane >= L::kBc / 2 : 64 * r >= L::kBc / 2;
          if (back.value || kBcEach == 1 || !which) rbc[r] = (which ? cp : bp)[o_bc[r]];
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bool in = b * SG + q < there;
          auto clamped = [&](const Walk& v, unsigned o) {
            return load_pair<T, DUO>(v.p + (in ? int64_t(b * SG) * v.row + o : int64_t(chan)));
          };
          rdt[b] = clamped(dt, o_dt);
          ru[b] = clamped(u, o_u);
          if constexpr (back.value) {
            rz[b] = clamped(z, o_z);
            rdy[b] = clamped(dy, o_dy);
          }
        }
#pragma unroll
        for (int r = 0; r < kBcEach; ++r) {
          const bool which = kBcEach == 1 ? lane >= L::kBc / 2 : 64 * r >= L::kBc / 2;
          rbc[r] = (which ? cp : bp)[t_bc[r] < there ? o_bc[r] : 0];
        }
      }
    };
    // what every lane group needs of them, into LDS
    auto spread = [&](int k, auto back) {
      const int left = te - t0 - k * SUB;
      wave_fence();
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = b * SG + q;
        const bool in = j < left;
        float delta[2], x[2], gy[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float raw = rdt[b].get(c) + bias[c], plus = softplus_f32(raw);
          const bool real = in && own[c];
          delta[c] = real ? (soft ? plus : raw) : 0.f;
          x[c] = real ? delta[c] * ru[b].get(c) : 0.f;
          if constexpr (back.value) {
            const float zz = rz[b].get(c), gate = zz * sigmoid_f32(zz);
            gy[c] = real ? rdy[b].get(c) * (gated ? gate : 1.f) : 0.f;
          }
        }
        *reinterpret_cast<float2*>(tok + j * CT + 2 * l) = make_float2(delta[0], delta[1]);
        *reinterpret_cast<float2*>(tok + (SUB + j) * CT + 2 * l) = make_float2(x[0], x[1]);
        if constexpr (back.value) *reinterpret_cast<float2*>(tok + (2 * SUB + j) * CT + 2 * l) = make_float2(gy[0], gy[1]);
      }
#pragma unroll
      for (int r = 0; r < kBcEach; ++r) {
        const float v = t_bc[r] < min(left, SUB) ? to_f32(rbc[r]) : 0.f;
        if (L::kBc % 64 == 0 || lane + 64 * r < L::kBc) bc[lane + 64 * r] = v;
      }
      wave_fence();
    };
    auto pair_at = [&](int kind, int j) {
      return *reinterpret_cast<const float2*>(tok + (kind * SUB + j) * CT + 2 * l);
    };
    auto states_at = [&](int which, int j) {
      return *reinterpret_cast<const f32x4_s*>(bc + (which * SUB + j) * (4 * SG) + 4 * q);
    };
    const std::true_type yes{};
    const std::false_type no{};

    if (subs == 1) fetch(0, yes);
    else if (subs > 1) fetch(0, no);
    float h[2][4] = {}, g[2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!own[c] || s0 + i >= a.s) continue;
        if (a.chunks > 1) {
          const int64_t k = (item * a.s + s0 + i) * channels + chan + c;
          h[c][i] = a.carry[k];
          g[c][i] = a.gcarry[k];
        } else {
          const int64_t k = (int64_t(n) * channels + chan + c) * a.s + s0 + i;
          if (a.h_in) h[c][i] = a.h_in[k];
          if (a.dh_out) g[c][i] = a.dh_out[k];
        }
      }

    // forward, to the states before every SUB tokens
    for (int k = 0; k < subs - 1; ++k) {
      kept[(2 * k) * 64] = f32x4_s{h[0][0], h[0][1], h[0][2], h[0][3]};
      kept[(2 * k + 1) * 64] = f32x4_s{h[1][0], h[1][1], h[1][2], h[1][3]};
      spread(k, no);
      if (k + 1 == subs - 1) fetch(k + 1, yes);
      else fetch(k + 1, no);
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        const float2 delta = pair_at(0, j), x = pair_at(1, j);
        const f32x4_s b = states_at(0, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[0][i] = fmaf(__builtin_amdgcn_exp2f(delta.x * a2[0][i]), h[0][i], x.x * b[i]);
          h[1][i] = fmaf(__builtin_amdgcn_exp2f(delta.y * a2[1][i]), h[1][i], x.y * b[i]);
        }
      }
    }

    // and back
    for (int k = subs - 1; k >= 0; --k) {
      const int tb = t0 + k * SUB;
      spread(k, yes);
      Pair<T> mdt[NB], mu[NB], mz[NB], mdy[NB];  // this walk's, while the next one's load
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mdt[b] = rdt[b];
        mu[b] = ru[b];
        mz[b] = rz[b];
        mdy[b] = rdy[b];
      }
      if (k < subs - 1) {
        const f32x4_s x = kept[(2 * k) * 64], y = kept[(2 * k + 1) * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[0][i] = x[i];
          h[1][i] = y[i];
        }
      }
      float old[SUB][2][4];
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        const float2 delta = pair_at(0, j), x = pair_at(1, j);
        const f32x4_s b = states_at(0, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          old[j][0][i] = __builtin_amdgcn_exp2f(delta.x * a2[0][i]) * h[0][i];
          old[j][1][i] = __builtin_amdgcn_exp2f(delta.y * a2[1][i]) * h[1][i];
          h[0][i] = fmaf(x.x, b[i], old[j][0][i]);
          h[1][i] = fmaf(x.y, b[i], old[j][1][i]);
        }
      }
      wave_fence();  // what follows reads LDS again rather than hold eight tokens' values
      if (k > 0) fetch(k - 1, yes);
      float* comb = lds + at.comb + turn * waves * wc * L::kComb;
      float* meet = lds + at.meet + turn * waves * wc * L::kMeet;
      // results of this lane group's token of the b-th SG, from its sums over states
      auto finish = [&](int b, const float (&sum)[6]) {
        const Walk du_o = walk(offsetof(ScanArgs, du), k), ddt_o = walk(offsetof(ScanArgs, ddt), k),
                   dz_o = walk(offsetof(ScanArgs, dz), k);
        const int j = b * SG + q;
        const bool in = j < te - tb;
        const float2 delta2 = pair_at(0, j), gy2 = pair_at(2, j);
        const float delta[2] = {delta2.x, delta2.y}, gy[2] = {gy2.x, gy2.y};
        float du[2], ddt[2], dz[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float raw = mdt[b].get(c) + bias[c], uu = mu[b].get(c), zz = mz[b].get(c);
          const bool real = in && own[c];
          const float slope = sigmoid_f32(raw), sg = sigmoid_f32(zz);
          const float d = fmaf(sum[4 + c], kLn2, uu * sum[2 + c]);
          ddt[c] = real ? d * (soft && !(raw > 20.f) ? slope : 1.f) : 0.f;
          du[c] = real ? fmaf(skip[c], gy[c], delta[c] * sum[2 + c]) : 0.f;
          dd[c] = real ? fmaf(gy[c], uu, dd[c]) : dd[c];
          dbias[c] += ddt[c];
          const float y_all = fmaf(skip[c], uu, sum[c]);
          dz[c] = real ? mdy[b].get(c) * y_all * (sg * (1.f + zz * (1.f - sg))) : 0.f;
        }
        if (j < t1 - tb) {
          if (has_du) store_pair<T, DUO>(du_o.p + int64_t(b * SG) * du_o.row + o_du, du[0], du[1], own[0], own[1]);
          if (has_ddt) store_pair<T, DUO>(ddt_o.p + int64_t(b * SG) * ddt_o.row + o_ddt, ddt[0], ddt[1], own[0], own[1]);
          if (has_dz) store_pair<T, DUO>(dz_o.p + int64_t(b * SG) * dz_o.row + o_dz, dz[0], dz[1], own[0], own[1]);
        }
      };
      float bcsum[SUB];
#pragma unroll
      for (int b = NB - 1; b >= 0; --b) {
        float y0[2][SG], gb[2][SG], ca[2][SG];
#pragma unroll
        for (int jj = SG - 1; jj >= 0; --jj) {
          const int j = b * SG + jj;
          const float2 delta2 = pair_at(0, j), x2 = pair_at(1, j), gy2 = pair_at(2, j);
          const f32x4_s bb = states_at(0, j), cc = states_at(1, j);
          const float delta[2] = {delta2.x, delta2.y}, x[2] = {x2.x, x2.y}, gy[2] = {gy2.x, gy2.y};
          float v[8] = {};  // dB of four states, dC of four states
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            y0[c][jj] = gb[c][jj] = ca[c][jj] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float hh = fmaf(x[c], bb[i], old[j][c][i]);
              g[c][i] = fmaf(cc[i], gy[c], g[c][i]);
              y0[c][jj] = fmaf(hh, cc[i], y0[c][jj]);
              gb[c][jj] = fmaf(g[c][i], bb[i], gb[c][jj]);
              v[i] = fmaf(g[c][i], x[c], v[i]);
              v[4 + i] = fmaf(hh, gy[c], v[4 + i]);
              const float through = g[c][i] * old[j][c][i];
              ca[c][jj] = fmaf(through, a2[c][i], ca[c][jj]);
              da[c][i] = fmaf(through, delta[c], da[c][i]);
              g[c][i] *= __builtin_amdgcn_exp2f(delta[c] * a2[c][i]);
            }
          }
          bcsum[j] = reduce8<LC>(v, lane);
          if (j % kDup == 0) {  // kDup tokens a store, one for each copy
            float w = bcsum[j];
#pragma unroll
            for (int i = 1; i < kDup && j + i < SUB; ++i) w = copy == i ? bcsum[j + i] : w;
            if (SUB >= kDup || copy < SUB) comb[j * waves * kVal + comb_at] = w;
          }
        }
        float sum[6];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sum[c] = sum_groups<SG>(y0[c]);
          sum[2 + c] = sum_groups<SG>(gb[c]);
          sum[4 + c] = sum_groups<SG>(ca[c]);
        }
        if constexpr (MULTI) {
#pragma unroll
          for (int i = 0; i < 6; ++i) meet[((wave * NB + b) * 6 + i) * 64 + lane] = sum[i];
        } else {
          finish(b, sum);
        }
      }

      __syncthreads();
      // (a token past the valid ones has zeros here, unless a state or gradient is infinite)
      const int more = waves * L::kComb, held = (te - tb) * waves * kVal;
      for (int i = threadIdx.x; i < more; i += 64 * waves * wc) {
        float s = comb[i];
        if (wc == 4) s += comb[more + i] + comb[2 * more + i] + comb[3 * more + i];
        else if (wc == 2) s += comb[more + i];
        if (i < (t1 - tb) * waves * kVal) pbc[int64_t(tb) * waves * kVal + i] = i < held ? s : 0.f;
      }
      if constexpr (MULTI) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (b % waves != sw) continue;
          float total[6];
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            total[i] = 0.f;
            for (int w = 0; w < waves; ++w) total[i] += meet[(((cw * waves + w) * NB + b) * 6 + i) * 64 + lane];
          }
          finish(b, total);
        }
      }
      turn ^= 1;
    }

    // tokens after the valid ones that no walk held
    if (subs * SUB < t1 - t0) {
      const Walk du_o = walk(offsetof(ScanArgs, du), subs), ddt_o = walk(offsetof(ScanArgs, ddt), subs),
                 dz_o = walk(offsetof(ScanArgs, dz), subs);
      for (int j = q; j < t1 - t0 - subs * SUB; j += SG) {
        if (sw != 0) continue;
        const unsigned on = unsigned(j - q);
        if (has_du) store_pair<T, DUO>(du_o.p + (o_du + on * unsigned(du_o.row)), 0.f, 0.f, own[0], own[1]);
        if (has_ddt) store_pair<T, DUO>(ddt_o.p + (o_ddt + on * unsigned(ddt_o.row)), 0.f, 0.f, own[0], own[1]);
        if (has_dz) store_pair<T, DUO>(dz_o.p + (o_dz + on * unsigned(dz_o.row)), 0.f, 0.f, own[0], own[1]);
      }
      const int64_t first = int64_t(t0 + subs * SUB) * waves * kVal, last = int64_t(t1) * waves * kVal;
      for (int64_t i = first + threadIdx.x; i < last; i += 64 * waves * wc) pbc[i] = 0.f;
    }
    if (ch == 0 && a.dh_in) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (own[c] && s0 + i < a.s) a.dh_in[(int64_t(n) * channels + chan + c) * a.s + s0 + i] = g[c][i];
    }
  }

#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float s[SG], w[SG];
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      s[i] = dd[c];
      w[i] = dbias[c];
    }
    const float sum_d = sum_groups<SG>(s), sum_b = sum_groups<SG>(w);
    if (!own[c]) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s0 + i < a.s) a.part_a[(int64_t(worker) * channels + chan + c) * a.s + s0 + i] = da[c][i];
    if (q == 0) {
      a.part_d[(int64_t(worker) * waves + sw) * channels + chan + c] = sum_d;
      a.part_bias[(int64_t(worker) * waves + sw) * channels + chan + c] = sum_b;
    }
  }
}

// dB and dC: the sum over the group's tiles of the partial sums [tile][n][t][waves][2][each].
// A grid of up to kBcGrid workgroups takes all values in turns: a long call has
// more of them than a launch has threads.
constexpr int64_t kBcGrid = 1 << 16;

template <class T>
__global__ __launch_bounds__(256) void bc_sum(ScanArgs a, ScanRows db, ScanRows dc, int each) {
  const int64_t per = int64_t(2) * a.groups * a.s;  // values a token
  const int64_t values = int64_t(a.n) * a.t * per, step = int64_t(gridDim.x) * 256;
  const int64_t token = int64_t(a.waves) * 2 * each, tile = int64_t(a.n) * a.t * token;
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < values; id += step) {
    const int64_t tok = id / per;
    const int v = int(id - tok * per), which = v / (a.groups * a.s), gs = v - which * a.groups * a.s;
    const int group = gs / a.s, s = gs - group * a.s;
    const ScanRows& out = which ? dc : db;
    if (!out.p) continue;
    const float* p = a.part_bc + group * a.tiles_per_group * tile + tok * token + (s / each * 2 + which) * each + s % each;
    float sum = 0.f;
    for (int i = 0; i < a.tiles_per_group; ++i) sum += p[i * tile];
    const int64_t n = tok / a.t, t = tok - n * a.t;
    static_cast<T*>(out.p)[n * out.batch + t * out.row + gs] = from_f32<T>(sum);
  }
}

template <class T, int SG, int SUB, bool MULTI, bool DUO>
int launch_main(const ScanArgs& a, const cc3d::ScanBwdShape& v, hipStream_t s) {
  const int lds = 4 * BwdLds<SG, SUB>(a.chunk, v.waves, v.wc).total;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_bwd<T, SG, SUB, MULTI, DUO>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();  // leave no error for the caller's next runtime call
      return int(e);
    }
  }
  const int64_t tiles = int64_t(a.groups) * a.tiles_per_group;
  return launch(scan_bwd<T, SG, SUB, MULTI, DUO>, tiles * a.workers, 64 * v.waves * v.wc, lds, s, a, v.wc);
}

template <class T, int SG, int SUB, bool MULTI>
int run_main(const ScanArgs& a, const cc3d::ScanBwdShape& v, hipStream_t s) {
  return a.wide > 1 ? launch_main<T, SG, SUB, MULTI, true>(a, v, s) : launch_main<T, SG, SUB, MULTI, false>(a, v, s);
}

template <class T, int NS>
int run_carries(const cc3d_scan_plan& p, ScanArgs a, hipStream_t s) {
  a.waves = cc3d::scan_fwd_waves(p.d);
  a.tiles_per_group = cc3d::scan_tiles_per_group(p.d);
  int e = run_carry<T, NS, true>(a, s);
  if (!e) e = run_join(a, true, s);
  return e;
}

template <class T>
int run_scan_bwd(const cc3d_scan_plan& p, ScanArgs& a, const cc3d_scan_args_t& c, const cc3d::ScanBwdShape& v,
                 hipStream_t s) {
  int e = 0;
  if (a.chunks > 1) {
    switch (cc3d::scan_fwd_ns(p.d)) {
      case 4: e = run_carries<T, 4>(p, a, s); break;
      case 8: e = run_carries<T, 8>(p, a, s); break;
      default: e = run_carries<T, 16>(p, a, s);
    }
    if (e) return e;
  }
  switch (v.sg) {
    case 1: e = run_main<T, 1, 4, false>(a, v, s); break;
    case 2: e = run_main<T, 2, 8, false>(a, v, s); break;
    default: e = v.waves > 1 ? run_main<T, 4, 8, true>(a, v, s) : run_main<T, 4, 8, false>(a, v, s);
  }
  if (!e && (c.db.p || c.dc.p)) {
    const int64_t values = int64_t(a.n) * a.t * 2 * a.groups * a.s;
    e = launch(bc_sum<T>, std::min((values + 255) / 256, kBcGrid), 256, 0, s, a, view_of(c.db), view_of(c.dc), 4 * v.sg);
  }
  return e;
}

}  // namespace

namespace cc3d {

int launch_scan_backward(const cc3d_scan_plan& p, const cc3d_scan_args_t& c, void* stream) {
  ScanArgs a = scan_args(p, c);
  a.dy = view_of(c.dy);
  a.du = view_of(c.du);
  a.ddt = view_of(c.ddt);
  a.dz = view_of(c.dz);
  a.dh_out = c.dh_out;
  a.dh_in = c.dh_in;
  const ScanBwdShape v = scan_bwd_shape(p.d);
  a.chunk = v.chunk;
  a.chunks = p.info.backward_chunks;
  a.workers = p.bwd_workers;
  a.waves = v.waves;
  a.tiles_per_group = v.tiles_per_group;
  const int64_t state = int64_t(p.d.states) * p.d.d, items = int64_t(p.d.n) * a.chunks;
  float* w = static_cast<float*>(c.workspace);
  if (a.chunks > 1) {
    a.carry = w;
    a.gcarry = a.carry + items * state;
    a.sums = a.gcarry + items * state;
    w = a.sums + items * p.d.d;
  }
  a.part_a = w;
  a.part_d = a.part_a + a.workers * state;
  a.part_bias = a.part_d + int64_t(a.workers) * a.waves * p.d.d;
  a.part_bc = a.part_bias + int64_t(a.workers) * a.waves * p.d.d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int e = p.d.dtype == CC3D_BF16 ? run_scan_bwd<bf16_s>(p, a, c, v, s) : run_scan_bwd<float>(p, a, c, v, s);
  if (e) return e;
  const int64_t rows = int64_t(a.workers) * a.waves;
  const SumJob jobs[] = {{a.part_a, c.da, a.workers, state, state},
                         {a.part_d, c.dd, rows, p.d.d, p.d.d},
                         {a.part_bias, c.ddt_bias, rows, p.d.d, p.d.d}};
  return launch_sums(jobs, 3, stream);
}

}  // namespace cc3d
