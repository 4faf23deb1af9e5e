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

// Two neighbouring channels as they are stored.
template <class T>
struct Pair {
  using U = std::conditional_t<sizeof(T) == 4, unsigned long long, unsigned>;
  U v;
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(unsigned(v >> (32 * i)));
    else return __uint_as_float(i ? v & 0xffff0000u : v << 16);
  }
};

// Element `off` (32 bits) after a base that is the same for the whole wave.
// `whole`: rows of pairs are aligned to a pair.  Otherwise one by one, the
// second at `step` (0 when there is no second channel).
template <class T>
__device__ __forceinline__ Pair<T> load_pair(const T* base, unsigned off, bool whole, int step) {
  using U = typename Pair<T>::U;
  Pair<T> r;
  if (whole) {
    r.v = *reinterpret_cast<const U*>(base + off);
  } else if constexpr (sizeof(T) == 4) {
    r.v = __float_as_uint(base[off]) | U(__float_as_uint(base[off + step])) << 32;
  } else {
    r.v = base[off] | U(base[off + step]) << 16;
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_pair(T* base, unsigned off, float x, float y, bool whole, bool second) {
  using U = typename Pair<T>::U;
  if (whole) {
    U v;
    if constexpr (sizeof(T) == 4) v = __float_as_uint(x) | U(__float_as_uint(y)) << 32;
    else v = pack_bf16(x, y);
    *reinterpret_cast<U*>(base + off) = v;
  } else {
    base[off] = from_f32<T>(x);
    if (second) base[off + 1] = from_f32<T>(y);
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

template <class T, int SG, int SUB>
__global__ __launch_bounds__(256, 2) void scan_bwd(ScanArgs a, int wc, int whole) {
  using L = BwdLds<SG, SUB>;
  constexpr int LC = 64 / SG, CT = 2 * LC, NB = SUB / SG, kDup = LC / 8;
  constexpr int kBcEach = (L::kBc + 63) / 64;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const L at(a.chunk, a.waves, wc);
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int sw = wave % a.waves, cw = wave / a.waves;
  const int q = lane / LC, l = lane % LC;
  const int tiles = a.tiles_per_group * a.groups, tile = blockIdx.x % tiles, worker = blockIdx.x / tiles;
  const int group = tile / a.tiles_per_group;
  const int in_group = ((tile - group * a.tiles_per_group) * wc + cw) * CT + 2 * l;
  const bool on = in_group < a.wide, on2 = in_group + 1 < a.wide;
  const int chan = group * a.wide + (on ? in_group : 0), step = on2 ? 1 : 0;
  const int channels = a.groups * a.wide;
  const int s0 = sw * 4 * SG + q * 4;  // this lane's first state
  f32x4_s* kept = reinterpret_cast<f32x4_s*>(lds + wave * at.per_wave) + lane;
  float* tok = lds + wave * at.per_wave + at.kept;
  float* bc = tok + L::kTok;

  float bias[2], skip[2], a2[2][4], da[2][4] = {}, dd[2] = {}, dbias[2] = {};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    bias[c] = a.bias ? a.bias[chan + c * step] : 0.f;
    skip[c] = a.d ? a.d[chan + c * step] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a2[c][i] = s0 + i < a.s ? a.a[int64_t(chan + c * step) * a.s + s0 + i] * kLog2e : 0.f;
  }
  int turn = 0;

  for (int64_t item = worker; item < int64_t(a.n) * a.chunks; item += a.workers) {
    const int n = int(item / a.chunks), ch = int(item - int64_t(n) * a.chunks);
    const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
    const int subs = te > t0 ? (te - t0 + SUB - 1) / SUB : 0;
    // token t0 of the chunk: the same address for the whole wave, with 32-bit offsets behind it
    auto at_chunk = [&](const ScanRows& v) { return static_cast<T*>(v.p) + int64_t(n) * v.batch + int64_t(t0) * v.row; };
    const T* bp = at_chunk(a.b) + group * a.s + sw * 4 * SG;
    const T* cp = at_chunk(a.c) + group * a.s + sw * 4 * SG;
    const T *dt = at_chunk(a.dt), *u = at_chunk(a.u), *z = a.z.p ? at_chunk(a.z) : nullptr, *dy = at_chunk(a.dy);
    T* du_o = a.du.p ? at_chunk(a.du) : nullptr;
    T* ddt_o = a.ddt.p ? at_chunk(a.ddt) : nullptr;
    T* dz_o = a.dz.p ? at_chunk(a.dz) : nullptr;
    auto off = [&](const ScanRows& v, int t) { return unsigned(t - t0) * unsigned(v.row) + unsigned(chan); };
    float* pbc = a.part_bc + (int64_t(tile) * a.n + n) * a.t * a.waves * (8 * SG);

    // inputs of the tokens of one walk: this lane group's tokens, and this lane's share of B and C
    Pair<T> rdt[NB], ru[NB], rz[NB], rdy[NB];
    T rbc[kBcEach];
    auto fetch = [&](int tb, bool back) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int t = tb + b * SG + q;
        rdt[b] = ru[b] = rz[b] = rdy[b] = Pair<T>{};
        if (t < te) {
          rdt[b] = load_pair(dt, off(a.dt, t), whole, step);
          ru[b] = load_pair(u, off(a.u, t), whole, step);
          if (back) {
            if (z) rz[b] = load_pair(z, off(a.z, t), whole, step);
            rdy[b] = load_pair(dy, off(a.dy, t), whole, step);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kBcEach; ++r) {
        const int i = lane + 64 * r, half = L::kBc / 2;
        const int which = i / half, t = tb + i % half / (4 * SG), s = i % (4 * SG);
        rbc[r] = T(0);
        if (i < L::kBc && t < te && sw * 4 * SG + s < a.s && (back || !which))
          rbc[r] = which ? cp[unsigned(t - t0) * unsigned(a.c.row) + s] : bp[unsigned(t - t0) * unsigned(a.b.row) + s];
      }
    };
    // what every lane group needs of them, into LDS
    auto spread = [&](int tb, bool back) {
      wave_fence();
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = b * SG + q;
        const bool in = tb + j < te;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bool real = in && (c ? on2 : on);
          const float delta = real ? delta_of(a, rdt[b].get(c) + bias[c]) : 0.f;
          tok[j * CT + 2 * l + c] = delta;
          tok[(SUB + j) * CT + 2 * l + c] = real ? delta * ru[b].get(c) : 0.f;
          if (back) {
            float gy = rdy[b].get(c);
            if (z) {
              const float zz = rz[b].get(c);
              gy *= zz * sigmoid_f32(zz);
            }
            tok[(2 * SUB + j) * CT + 2 * l + c] = real ? gy : 0.f;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kBcEach; ++r)
        if (L::kBc % 64 == 0 || lane + 64 * r < L::kBc) bc[lane + 64 * r] = to_f32(rbc[r]);
      wave_fence();
    };
    auto pair_at = [&](int kind, int j) {
      return *reinterpret_cast<const float2*>(tok + (kind * SUB + j) * CT + 2 * l);
    };
    auto states_at = [&](int which, int j) {
      return *reinterpret_cast<const f32x4_s*>(bc + (which * SUB + j) * (4 * SG) + 4 * q);
    };

    float h[2][4] = {}, g[2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!(c ? on2 : on) || s0 + i >= a.s) continue;
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
    if (subs > 0) fetch(t0, subs == 1);
    for (int k = 0; k < subs - 1; ++k) {
      kept[(2 * k) * 64] = f32x4_s{h[0][0], h[0][1], h[0][2], h[0][3]};
      kept[(2 * k + 1) * 64] = f32x4_s{h[1][0], h[1][1], h[1][2], h[1][3]};
      spread(t0 + k * SUB, false);
      fetch(t0 + (k + 1) * SUB, k + 1 == subs - 1);
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
      spread(tb, true);
      Pair<T> mdt[NB], mu[NB], mz[NB], mdy[NB];  // this walk's, while the next one's load
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mdt[b] = rdt[b];
        mu[b] = ru[b];
        mz[b] = rz[b];
        mdy[b] = rdy[b];
      }
      if (k > 0) fetch(tb - SUB, true);
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
      float bcsum[SUB], sums[NB][6];
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
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sums[b][c] = sum_groups<SG>(y0[c]);
          sums[b][2 + c] = sum_groups<SG>(gb[c]);
          sums[b][4 + c] = sum_groups<SG>(ca[c]);
        }
      }

      // dB and dC: kDup tokens a store, one for each copy; value = which * 4 SG + q * 4 + state
      float* comb = lds + at.comb + (turn * a.waves * wc + wave) * L::kComb;
      const int copy = lane & (kDup - 1), value = l / kDup;  // value: which, state
#pragma unroll
      for (int j0 = 0; j0 < SUB; j0 += kDup) {
        float v = bcsum[j0];
#pragma unroll
        for (int i = 1; i < kDup && j0 + i < SUB; ++i) v = copy == i ? bcsum[j0 + i] : v;
        if (j0 + copy < SUB) comb[(j0 + copy) * (8 * SG) + (value >> 2) * (4 * SG) + q * 4 + (value & 3)] = v;
      }
      float* meet = lds + at.meet + turn * a.waves * wc * L::kMeet;
      if (a.waves > 1) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 6; ++i) meet[((wave * NB + b) * 6 + i) * 64 + lane] = sums[b][i];
      }
      __syncthreads();
      {
        const float* all = lds + at.comb + turn * a.waves * wc * L::kComb;
        const int threads = 64 * a.waves * wc;
        for (int i = threadIdx.x; i < a.waves * L::kComb; i += threads) {
          const int w = i / L::kComb, r = i - w * L::kComb, j = r / (8 * SG), t = tb + j;
          float s = all[w * L::kComb + r];
          for (int o = 1; o < wc; ++o) s += all[(o * a.waves + w) * L::kComb + r];
          if (t < t1) pbc[(int64_t(t) * a.waves + w) * (8 * SG) + r % (8 * SG)] = s;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (b % a.waves != sw) continue;
        if (a.waves > 1) {
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            float s = 0.f;
            for (int w = 0; w < a.waves; ++w) s += meet[(((cw * a.waves + w) * NB + b) * 6 + i) * 64 + lane];
            sums[b][i] = s;
          }
        }
        const int j = b * SG + q, t = tb + j;
        if (t >= t1 || !on) continue;
        const bool in = t < te;
        float du[2], ddt[2], dz[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float raw = mdt[b].get(c) + bias[c], uu = mu[b].get(c);
          const float delta = tok[j * CT + 2 * l + c], gy = tok[(2 * SUB + j) * CT + 2 * l + c];
          const bool real = in && (c ? on2 : on);
          ddt[c] = fmaf(sums[b][4 + c], kLn2, uu * sums[b][2 + c]);
          if (a.softplus && !(raw > 20.f)) ddt[c] *= sigmoid_f32(raw);
          ddt[c] = real ? ddt[c] : 0.f;
          du[c] = real ? fmaf(skip[c], gy, delta * sums[b][2 + c]) : 0.f;
          if (real) dd[c] = fmaf(gy, uu, dd[c]);
          dbias[c] += ddt[c];
          dz[c] = 0.f;
          if (z && real) {
            const float zz = mz[b].get(c), sg = sigmoid_f32(zz);
            dz[c] = mdy[b].get(c) * fmaf(skip[c], uu, sums[b][c]) * (sg * (1.f + zz * (1.f - sg)));
          }
        }
        if (du_o) store_pair(du_o, off(a.du, t), du[0], du[1], whole, on2);
        if (ddt_o) store_pair(ddt_o, off(a.ddt, t), ddt[0], ddt[1], whole, on2);
        if (dz_o) store_pair(dz_o, off(a.dz, t), dz[0], dz[1], whole, on2);
      }
      turn ^= 1;
    }

    // tokens after the valid ones that no walk held
    for (int t = t0 + subs * SUB + q; t < t1; t += SG) {
      if (sw != 0 || !on) continue;
      if (du_o) store_pair(du_o, off(a.du, t), 0.f, 0.f, whole, on2);
      if (ddt_o) store_pair(ddt_o, off(a.ddt, t), 0.f, 0.f, whole, on2);
      if (dz_o) store_pair(dz_o, off(a.dz, t), 0.f, 0.f, whole, on2);
    }
    const int64_t first = int64_t(t0 + subs * SUB) * a.waves * (8 * SG), last = int64_t(t1) * a.waves * (8 * SG);
    for (int64_t i = first + threadIdx.x; i < last; i += 64 * a.waves * wc) pbc[i] = 0.f;
    if (ch == 0 && a.dh_in) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((c ? on2 : on) && s0 + i < a.s) a.dh_in[(int64_t(n) * channels + chan + c) * a.s + s0 + i] = g[c][i];
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
    if (!(c ? on2 : on)) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s0 + i < a.s) a.part_a[(int64_t(worker) * channels + chan + c) * a.s + s0 + i] = da[c][i];
    if (q == 0) {
      a.part_d[(int64_t(worker) * a.waves + sw) * channels + chan + c] = sum_d;
      a.part_bias[(int64_t(worker) * a.waves + sw) * channels + chan + c] = sum_b;
    }
  }
}

// dB and dC: the sum over the group's tiles of the partial sums [tile][n][t][waves][2][each].
template <class T>
__global__ __launch_bounds__(256) void bc_sum(ScanArgs a, ScanRows db, ScanRows dc, int each) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = int64_t(2) * a.groups * a.s;  // values a token
  const int64_t tok = id / per;
  if (tok >= int64_t(a.n) * a.t) return;
  const int v = int(id - tok * per), which = v / (a.groups * a.s), gs = v - which * a.groups * a.s;
  const int group = gs / a.s, s = gs - group * a.s;
  const ScanRows& out = which ? dc : db;
  if (!out.p) return;
  const int64_t token = int64_t(a.waves) * 2 * each, tile = int64_t(a.n) * a.t * token;
  const float* p = a.part_bc + group * a.tiles_per_group * tile + tok * token + (s / each * 2 + which) * each + s % each;
  float sum = 0.f;
  for (int i = 0; i < a.tiles_per_group; ++i) sum += p[i * tile];
  const int64_t n = tok / a.t, t = tok - n * a.t;
  static_cast<T*>(out.p)[n * out.batch + t * out.row + gs] = from_f32<T>(sum);
}

// Every row of pairs starts on a multiple of a pair.
bool pairs_whole(const ScanArgs& a, int elem) {
  if (a.wide % 2) return false;
  for (const ScanRows* v : {&a.u, &a.dt, &a.z, &a.dy, &a.du, &a.ddt, &a.dz})
    if (v->p && (reinterpret_cast<uintptr_t>(v->p) % (2 * elem) || v->batch % 2 || v->row % 2)) return false;
  return true;
}

template <class T, int SG, int SUB>
int run_main(const ScanArgs& a, const cc3d::ScanBwdShape& v, hipStream_t s) {
  const int lds = 4 * BwdLds<SG, SUB>(a.chunk, v.waves, v.wc).total;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_bwd<T, SG, SUB>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();  // leave no error for the caller's next runtime call
      return int(e);
    }
  }
  const int64_t tiles = int64_t(a.groups) * a.tiles_per_group;
  scan_bwd<T, SG, SUB><<<unsigned(tiles * a.workers), 64 * v.waves * v.wc, lds, s>>>(a, v.wc, pairs_whole(a, sizeof(T)));
  return int(hipGetLastError());
}

template <class T, int NS>
int run_carries(const cc3d_scan_plan& p, ScanArgs a, hipStream_t s) {
  a.waves = cc3d::scan_fwd_waves(p.d);
  a.tiles_per_group = cc3d::scan_tiles_per_group(p.d);
  int e = run_carry<T, NS, true>(a, s);
  if (!e) e = run_join<false>(a, s);
  if (!e) e = run_join<true>(a, s);
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
    case 1: e = run_main<T, 1, 4>(a, v, s); break;
    case 2: e = run_main<T, 2, 8>(a, v, s); break;
    default: e = run_main<T, 4, 8>(a, v, s);
  }
  if (!e && (c.db.p || c.dc.p)) {
    const int64_t values = int64_t(a.n) * a.t * 2 * a.groups * a.s;
    bc_sum<T><<<unsigned((values + 255) / 256), 256, 0, s>>>(a, view_of(c.db), view_of(c.dc), 4 * v.sg);
    e = int(hipGetLastError());
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
