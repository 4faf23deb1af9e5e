// Device helpers of the sequence operators' kernels.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "cc3d_seq_internal.h"

namespace {

// One launch; 0, or the runtime's code for this launch.  (The runtime's last
// error may be another call's: it is neither asked for nor cleared when the
// launch is taken.)
template <class T>
struct SameType {
  using type = T;
};
template <class... P>
int launch(void (*kernel)(P...), int64_t workgroups, int threads, int lds, hipStream_t s, typename SameType<P>::type... args) {
  void* at[] = {&args...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(unsigned(workgroups)),
                                       dim3(unsigned(threads)), at, size_t(lds), s);
  if (e != hipSuccess) (void)hipGetLastError();  // leave no error for the caller's next runtime call
  return int(e);
}

typedef unsigned u32x4_s __attribute__((ext_vector_type(4)));
typedef float f32x4_s __attribute__((ext_vector_type(4)));

// The hardware's exponential is of two: exp(v) rounds v * kLog2e besides, which is
// |v| units of 2^-24 of the result or so.
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Storage types: bf16 is held as its 16 bits.
using bf16_s = unsigned short;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_s v) { return __uint_as_float(unsigned(v) << 16); }

template <class T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return __builtin_bit_cast(bf16_s, static_cast<__bf16>(v));  // to nearest even
}

// Eight consecutive elements as they are stored; 16 bytes a register quad.
// They need only their element's alignment: 16-byte accesses two or four bytes
// off copy at 4.4 to 4.7 TB/s where aligned ones do at 4.8, and 2-byte accesses
// at 3.0.
template <class T>
struct Raw8 {
  u32x4_s q[sizeof(T) / 2];
};

typedef u32x4_s u32x4_by2 __attribute__((aligned(2)));
typedef u32x4_s u32x4_by4 __attribute__((aligned(4)));
template <class T>
struct Quad {
  using type = std::conditional_t<sizeof(T) == 4, u32x4_by4, u32x4_by2>;
};

template <class T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.q[i] = reinterpret_cast<const typename Quad<T>::type*>(p)[i];
  return r;
}

template <class T>
__device__ __forceinline__ Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.q[i] = u32x4_s{0, 0, 0, 0};
  return r;
}

template <class T>
__device__ __forceinline__ float get8(const Raw8<T>& r, int j) {
  if constexpr (std::is_same_v<T, float>) return __uint_as_float(r.q[j / 4][j % 4]);
  else return __uint_as_float(j & 1 ? r.q[0][j / 2] & 0xffff0000u : r.q[0][j / 2] << 16);
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  return unsigned(from_f32<bf16_s>(lo)) | (unsigned(from_f32<bf16_s>(hi)) << 16);
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  using Q = typename Quad<T>::type;
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<Q*>(p)[i] = u32x4_s{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                           __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
  } else {
    *reinterpret_cast<Q*>(p) =
        u32x4_s{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  }
}

template <class T>
__device__ __forceinline__ void set8(Raw8<T>& r, int j, T v) {
  if constexpr (sizeof(T) == 4) r.q[j / 4][j % 4] = __float_as_uint(v);
  else r.q[0][j / 2] = (r.q[0][j / 2] & (j & 1 ? 0xffffu : 0xffff0000u)) | unsigned(v) << (16 * (j & 1));
}

// The first n (1 to 7) of eight elements, the others zero: the last columns of
// a row whose length is no multiple of eight.  Every load has an address of
// its own inside the row and none waits for another.
template <class T>
__device__ __forceinline__ Raw8<T> load_some(const T* p, int n) {
  T v[7];
#pragma unroll
  for (int j = 0; j < 7; ++j) v[j] = p[min(j, n - 1)];
  Raw8<T> r{};
#pragma unroll
  for (int j = 0; j < 7; ++j) set8(r, j, j < n ? v[j] : T(0));
  return r;
}

template <class T>
__device__ __forceinline__ void store_some(T* p, int n, const float* v) {
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) p[j] = from_f32<T>(v[j]);
}

// 1 / (1 + exp(-v)): the exponential of a large -v is infinite and its
// reciprocal zero.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// log(1 + exp(v)), v itself above 20 (where exp(-v) is below half a unit in
// the last place of v).  What w = 1 + e loses of e = exp(v), e - (w - 1)
// (no rounding for e <= 1), is added back: log(1 + e) = log(w) + lost / w, the
// next order below 2^-25 of the result.  Against 64 bits over a million
// values: 4 units of 2^-24 above 0, 6.4 at -4 (55.7 without), and below that
// the rounding of the exponential's argument, |v| or so.
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(v * kLog2e), w = 1.f + e;
  const float log1p = fmaf(e - (w - 1.f), __builtin_amdgcn_rcpf(w), kLn2 * __builtin_amdgcn_logf(w));
  return v > 20.f ? v : log1p;
}

// v from lane ^ X of the wave, X = 1, 2, 4 or 8 (reached by mirroring half a
// row of 16 and then the row, once the lower bits are equal).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(unsigned(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, 0xf, 0xf, true)));
}

// Sum over aligned groups of G lanes of a wave, in every lane of the group;
// the same order whatever the lane.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G >= 2) v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  if constexpr (G >= 4) v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  if constexpr (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
  if constexpr (G >= 16) v += dpp<0x140>(v);  // row_mirror
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

}  // namespace
