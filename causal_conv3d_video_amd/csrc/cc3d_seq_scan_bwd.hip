// Selective state space scan, backward.
//
//   g[t] = C gy[t] + exp(delta[t+1] A) g[t+1],  gy = dy silu(z)
//   du = D gy + delta sum g B;   ddelta = sum g (A exp(delta A) h[t-1] + u B)
//   dA = sum g delta exp(delta A) h[t-1];  dB = sum_channels g delta u;  dC = sum_channels gy h
//
// The states are not kept by the forward pass: the time axis is cut into
// chunks of 64 tokens (32 where more than 32 states need the LDS), the forward and the reverse recurrence are carried
// across them as in the forward pass, and a workgroup then takes one chunk of
// 64 channels at a time, independent of every other.  It walks the chunk
// forward, leaving the state before every eight tokens in LDS, and then back,
// eight tokens at a time: the eight decays and decayed states are made again
// into registers and the gradient walks over them.  A lane owns one channel
// with eight of its states, so sums over states stay in the lane (waves of
// other states meet in LDS), and the sums over channels for dB and dC go
// across the 64 lanes by halving: each step adds two registers' halves into
// one, 2.2 instructions a value.  Those are written as partial sums a
// tile of 64 channels and added in the tiles' order by a last small kernel.
#include "cc3d_seq_scan.h"

#include <algorithm>

namespace {

constexpr int kSub = 8;          // tokens walked back at a time

// The waves' sums over states meet in LDS in two places used in turn; past
// four waves there is room for one, with a barrier more.
__host__ __device__ inline int meet_turns(int waves) { return waves > 4 ? 1 : 2; }

// The sums over the wave of 2 * NS values, one in each of 2 * NS lanes' places:
// lane bits 5 (first or second half), 4, 3, 2 (the state's bits, highest
// first); equal in the four lanes of a quad.
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

template <int NS>
__device__ __forceinline__ float reduce_lanes(const float (&pb)[NS], const float (&pc)[NS], int lane) {
  float v[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = swap32_add(pb[i], pc[i]);
#pragma unroll
  for (int i = 0; i < NS / 2; ++i) v[i] = swap16_add(v[i], v[i + NS / 2]);
#pragma unroll
  for (int i = 0; i < NS / 4; ++i) v[i] = dpp_add<0x128>(v[i], v[i + NS / 4], lane & 8);  // row_ror:8
  float r;
  if constexpr (NS == 8) r = dpp_add<0x141>(v[0], v[1], lane & 4);  // row_half_mirror
  else r = v[0] + dpp<0x141>(v[0]);
  r += dpp<0xB1>(r);
  r += dpp<0x4E>(r);
  return r;
}

template <class T, int NS, bool MULTI>
__global__ __launch_bounds__(MULTI ? 64 * (cc3d::kScanMaxStates / NS) : 64) void scan_bwd(ScanArgs a) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const Place at(a);
  // this wave's states before every kSub tokens [chunk / kSub][NS][64], its B and C [2][kSub][NS],
  // and the waves' sums over states [turns][3][waves][kSub][64]
  const int kept_size = a.chunk / kSub * NS * 64, turns = meet_turns(a.waves);
  float* kept = lds + at.wave * kept_size + at.lane;
  float* bc = lds + a.waves * kept_size + at.wave * (2 * kSub * NS);
  float* meet = lds + a.waves * (kept_size + 2 * kSub * NS);
  const int s0 = at.wave * NS, sp = a.waves * NS;
  const int channels = a.groups * a.wide;
  const float bias = a.bias ? a.bias[at.chan] : 0.f, skip = a.d ? a.d[at.chan] : 0.f;

  float a2[NS], da[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    a2[i] = s0 + i < a.s ? a.a[int64_t(at.chan) * a.s + s0 + i] * kLog2e : 0.f;
    da[i] = 0.f;
  }
  float dd = 0.f, dbias = 0.f;
  int turn = 0;

  for (int64_t item = at.item; item < int64_t(a.n) * a.chunks; item += a.workers) {
    const int n = int(item / a.chunks), ch = int(item - int64_t(n) * a.chunks);
    const int t0 = ch * a.chunk, t1 = min(t0 + a.chunk, a.t), te = min(t1, valid_tokens(a, n));
    const int subs = te > t0 ? (te - t0 + kSub - 1) / kSub : 0;
    const T* bp = rows<T>(a.b, n) + at.group * a.s;
    const T* cp = rows<T>(a.c, n) + at.group * a.s;
    const T* dt = rows<T>(a.dt, n) + at.chan;
    const T* u = rows<T>(a.u, n) + at.chan;
    const T* z = a.z.p ? rows<T>(a.z, n) + at.chan : nullptr;
    const T* dy = rows<T>(a.dy, n) + at.chan;
    T* du_o = a.du.p ? out_rows<T>(a.du, n) + at.chan : nullptr;
    T* ddt_o = a.ddt.p ? out_rows<T>(a.ddt, n) + at.chan : nullptr;
    T* dz_o = a.dz.p ? out_rows<T>(a.dz, n) + at.chan : nullptr;
    float* pbc = a.part_bc + (int64_t(at.tile) * a.n + n) * a.t * 2 * sp;
    const int64_t state_at = (int64_t(n) * channels + at.chan) * a.s + s0;

    auto stage = [&](int tb, bool both) {
      wave_fence();
      for (int i = at.lane; i < kSub * NS; i += 64) {
        const int t = tb + i / NS, s = s0 + i % NS;
        const bool in = t < te && s < a.s;
        bc[i] = in ? to_f32(bp[int64_t(t) * a.b.row + s]) : 0.f;
        if (both) bc[kSub * NS + i] = in ? to_f32(cp[int64_t(t) * a.c.row + s]) : 0.f;
      }
      wave_fence();
    };

    float h[NS], g[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const bool in = s0 + i < a.s;
      h[i] = g[i] = 0.f;
      if (in && a.chunks > 1) {
        h[i] = a.carry[(item * a.s + s0 + i) * channels + at.chan];
        g[i] = a.gcarry[(item * a.s + s0 + i) * channels + at.chan];
      } else if (in) {
        if (a.h_in) h[i] = a.h_in[state_at + i];
        if (a.dh_out) g[i] = a.dh_out[state_at + i];
      }
    }

    // forward, to the states before every kSub tokens
    for (int q = 0; q < subs; ++q) {
#pragma unroll
      for (int i = 0; i < NS; ++i) kept[(q * NS + i) * 64] = h[i];
      if (q == subs - 1) break;
      const int tb = t0 + q * kSub;
      stage(tb, false);
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const float delta = delta_of(a, to_f32(dt[int64_t(tb + j) * a.dt.row]) + bias);
        const float x = delta * to_f32(u[int64_t(tb + j) * a.u.row]);
#pragma unroll
        for (int i = 0; i < NS; ++i)
          h[i] = fmaf(__builtin_amdgcn_exp2f(delta * a2[i]), h[i], x * bc[j * NS + i]);
      }
    }

    // and back
    for (int q = subs - 1; q >= 0; --q) {
      const int tb = t0 + q * kSub;
      stage(tb, true);
      float delta[kSub], raw[kSub], x[kSub], gy[kSub], uu[kSub];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const int t = tb + j;
        delta[j] = raw[j] = gy[j] = uu[j] = 0.f;
        if (t < te) {
          raw[j] = to_f32(dt[int64_t(t) * a.dt.row]) + bias;
          delta[j] = delta_of(a, raw[j]);
          uu[j] = to_f32(u[int64_t(t) * a.u.row]);
          gy[j] = to_f32(dy[int64_t(t) * a.dy.row]);
          if (z) {
            const float zz = to_f32(z[int64_t(t) * a.z.row]);
            gy[j] *= zz * sigmoid_f32(zz);
          }
        }
        x[j] = delta[j] * uu[j];
      }
      float decay[kSub][NS], old[kSub][NS], y0[kSub], gb[kSub], ca[kSub];
#pragma unroll
      for (int i = 0; i < NS; ++i) h[i] = kept[(q * NS + i) * 64];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        y0[j] = gb[j] = ca[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          decay[j][i] = __builtin_amdgcn_exp2f(delta[j] * a2[i]);
          old[j][i] = decay[j][i] * h[i];
          h[i] = fmaf(x[j], bc[j * NS + i], old[j][i]);
          y0[j] = fmaf(h[i], bc[(kSub + j) * NS + i], y0[j]);
        }
      }
      float sums[kSub];
#pragma unroll
      for (int j = kSub - 1; j >= 0; --j) {
        float pb[NS], pc[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const float bb = bc[j * NS + i], cc = bc[(kSub + j) * NS + i];
          const float hh = fmaf(x[j], bb, old[j][i]);
          g[i] = fmaf(cc, gy[j], g[i]);
          gb[j] = fmaf(g[i], bb, gb[j]);
          pb[i] = at.on ? g[i] * x[j] : 0.f;
          pc[i] = at.on ? hh * gy[j] : 0.f;
          const float through = g[i] * old[j][i];
          ca[j] = fmaf(through, a2[i], ca[j]);
          da[i] = fmaf(through, delta[j], da[i]);
          g[i] *= decay[j][i];
        }
        sums[j] = reduce_lanes<NS>(pb, pc, at.lane);
      }
      // dB and dC of this tile: four tokens a store
#pragma unroll
      for (int j = 0; j < kSub; j += 4) {
        const int k = at.lane & 3;
        const float v = k == 0 ? sums[j] : k == 1 ? sums[j + 1] : k == 2 ? sums[j + 2] : sums[j + 3];
        const int t = tb + j + k;
        const int s = NS == 8 ? (at.lane >> 4 & 1) * 4 + (at.lane >> 3 & 1) * 2 + (at.lane >> 2 & 1)
                              : (at.lane >> 4 & 1) * 2 + (at.lane >> 3 & 1);
        if (t < t1 && (NS == 8 || !(at.lane & 4))) pbc[(int64_t(t) * 2 + (at.lane >> 5)) * sp + s0 + s] = v;
      }
      if (MULTI) {
        if (turns == 1) __syncthreads();
        float* m = meet + turn * (3 * a.waves * kSub * 64) + at.lane;
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          m[((0 * a.waves + at.wave) * kSub + j) * 64] = y0[j];
          m[((1 * a.waves + at.wave) * kSub + j) * 64] = gb[j];
          m[((2 * a.waves + at.wave) * kSub + j) * 64] = ca[j];
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        if (MULTI && j % a.waves != at.wave) continue;
        if (MULTI) {
          const float* m = meet + turn * (3 * a.waves * kSub * 64) + at.lane;
          y0[j] = gb[j] = ca[j] = 0.f;
          for (int w = 0; w < a.waves; ++w) {
            y0[j] += m[((0 * a.waves + w) * kSub + j) * 64];
            gb[j] += m[((1 * a.waves + w) * kSub + j) * 64];
            ca[j] += m[((2 * a.waves + w) * kSub + j) * 64];
          }
        }
        const int t = tb + j;
        if (t < t1 && at.on) {
          const bool in = t < te;
          float ddt = fmaf(ca[j], kLn2, uu[j] * gb[j]);
          if (a.softplus && !(raw[j] > 20.f)) ddt *= sigmoid_f32(raw[j]);
          ddt = in ? ddt : 0.f;
          const float du = in ? fmaf(skip, gy[j], delta[j] * gb[j]) : 0.f;
          dd = fmaf(gy[j], uu[j], dd);
          dbias += ddt;
          if (du_o) du_o[int64_t(t) * a.du.row] = from_f32<T>(du);
          if (ddt_o) ddt_o[int64_t(t) * a.ddt.row] = from_f32<T>(ddt);
          if (dz_o) {
            float v = 0.f;
            if (in) {
              const float zz = to_f32(z[int64_t(t) * a.z.row]), sg = sigmoid_f32(zz);
              v = to_f32(dy[int64_t(t) * a.dy.row]) * fmaf(skip, uu[j], y0[j]) * (sg * (1.f + zz * (1.f - sg)));
            }
            dz_o[int64_t(t) * a.dz.row] = from_f32<T>(v);
          }
        }
      }
      turn = turns - 1 - turn;
    }

    // tokens after the valid ones that no group of kSub held
    for (int t = t0 + subs * kSub; t < t1; ++t) {
      if (at.wave == 0 && at.on) {
        if (du_o) du_o[int64_t(t) * a.du.row] = from_f32<T>(0.f);
        if (ddt_o) ddt_o[int64_t(t) * a.ddt.row] = from_f32<T>(0.f);
        if (dz_o) dz_o[int64_t(t) * a.dz.row] = from_f32<T>(0.f);
      }
      if (at.lane < 2 * NS) pbc[(int64_t(t) * 2 + at.lane / NS) * sp + s0 + at.lane % NS] = 0.f;
    }
    if (ch == 0 && a.dh_in && at.on) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (s0 + i < a.s) a.dh_in[state_at + i] = g[i];
    }
  }

  if (!at.on) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (s0 + i < a.s) a.part_a[(at.item * channels + at.chan) * a.s + s0 + i] = da[i];
  a.part_d[(at.item * a.waves + at.wave) * channels + at.chan] = dd;
  a.part_bias[(at.item * a.waves + at.wave) * channels + at.chan] = dbias;
}

// dB and dC: the sum over the group's tiles.
template <class T>
__global__ __launch_bounds__(256) void bc_sum(ScanArgs a, ScanRows db, ScanRows dc, int sp) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = int64_t(2) * a.groups * a.s;  // values a token
  const int64_t tok = id / per;
  if (tok >= int64_t(a.n) * a.t) return;
  const int v = int(id - tok * per), which = v / (a.groups * a.s), gs = v - which * a.groups * a.s;
  const int group = gs / a.s, s = gs - group * a.s;
  const ScanRows& out = which ? dc : db;
  if (!out.p) return;
  const float* p = a.part_bc + ((int64_t(group) * a.tiles_per_group * a.n * a.t + tok) * 2 + which) * sp + s;
  float sum = 0.f;
  for (int i = 0; i < a.tiles_per_group; ++i) sum += p[int64_t(i) * a.n * a.t * 2 * sp];
  const int64_t n = tok / a.t, t = tok - n * a.t;
  static_cast<T*>(out.p)[n * out.batch + t * out.row + gs] = from_f32<T>(sum);
}

template <class T, int NS, bool MULTI>
int run_main(const ScanArgs& a, int64_t tiles, hipStream_t s) {
  const int lds = 4 * a.waves * (a.chunk / kSub * NS * 64 + 2 * kSub * NS + (MULTI ? meet_turns(a.waves) * 3 * kSub * 64 : 0));
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_bwd<T, NS, MULTI>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();  // leave no error for the caller's next runtime call
      return int(e);
    }
  }
  scan_bwd<T, NS, MULTI><<<unsigned(tiles * a.workers), 64 * a.waves, lds, s>>>(a);
  return int(hipGetLastError());
}

template <class T, int NS>
int run_scan_bwd(const cc3d_scan_plan& p, ScanArgs& a, const cc3d_scan_args_t& c, hipStream_t s) {
  const int64_t tiles = int64_t(a.groups) * a.tiles_per_group;
  const unsigned blocks = unsigned(tiles * a.n * a.chunks);
  int e = 0;
  if (a.chunks > 1) {
    scan_carry<T, NS, false><<<blocks, 64 * a.waves, 0, s>>>(a);
    scan_carry<T, NS, true><<<blocks, 64 * a.waves, 0, s>>>(a);
    e = int(hipGetLastError());
    if (e) return e;
    scan_join<false><<<join_blocks(p.d), 256, 0, s>>>(a);
    scan_join<true><<<join_blocks(p.d), 256, 0, s>>>(a);
    e = int(hipGetLastError());
    if (e) return e;
  }
  e = a.waves > 1 ? run_main<T, NS, true>(a, tiles, s) : run_main<T, NS, false>(a, tiles, s);
  if (e) return e;
  if (c.db.p || c.dc.p) {
    const int64_t values = int64_t(a.n) * a.t * 2 * a.groups * a.s;
    bc_sum<T><<<unsigned((values + 255) / 256), 256, 0, s>>>(a, view_of(c.db), view_of(c.dc), a.waves * NS);
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
  a.chunk = p.bwd_chunk;
  a.chunks = p.info.backward_chunks;
  a.workers = p.bwd_workers;
  a.waves = scan_bwd_waves(p.d);
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
  int e;
  if (p.d.dtype == CC3D_BF16)
    e = scan_bwd_ns(p.d) == 4 ? run_scan_bwd<bf16_s, 4>(p, a, c, s) : run_scan_bwd<bf16_s, 8>(p, a, c, s);
  else
    e = scan_bwd_ns(p.d) == 4 ? run_scan_bwd<float, 4>(p, a, c, s) : run_scan_bwd<float, 8>(p, a, c, s);
  if (!e) e = launch_sum_rows(a.part_a, a.workers, state, state, c.da, stream);
  if (!e) e = launch_sum_rows(a.part_d, int64_t(a.workers) * a.waves, p.d.d, p.d.d, c.dd, stream);
  if (!e) e = launch_sum_rows(a.part_bias, int64_t(a.workers) * a.waves, p.d.d, p.d.d, c.ddt_bias, stream);
  return e;
}

}  // namespace cc3d
