// Device helpers of the operators on rows of class scores: loads and stores of
// score vectors, exponentials, wave and workgroup reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gbdt.h"
#include "gbdt_device.h"
#include "gbdt_internal.h"

namespace gbdt {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.44269504088896340736;
constexpr int kRowsMaxClasses = 32;  // rows of at most this many classes: one thread each

// A score type: its element, how many make 16 bytes, and the conversions.
template <int DT>
struct Score;
template <>
struct Score<GBDT_DTYPE_F32> {
  using Elem = float;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float to_f32(Elem e) { return e; }
  static __device__ __forceinline__ Elem from_f32(float f) { return f; }
};
template <>
struct Score<GBDT_DTYPE_BF16> {
  using Elem = __bf16;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to_f32(Elem e) {
    return __uint_as_float(uint32_t(__builtin_bit_cast(uint16_t, e)) << 16);
  }
  static __device__ __forceinline__ Elem from_f32(float f) { return static_cast<__bf16>(f); }
};
template <>
struct Score<GBDT_DTYPE_F16> {
  using Elem = _Float16;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to_f32(Elem e) { return static_cast<float>(e); }
  static __device__ __forceinline__ Elem from_f32(float f) { return static_cast<_Float16>(f); }
};

// 16 bytes of scores.  A row may start at any element, so the loads and
// stores are by the element's alignment; gfx950 does them in one access.
template <int DT>
struct Vec16 {
  typename Score<DT>::Elem e[Score<DT>::kVec];
};

template <int DT>
__device__ __forceinline__ Vec16<DT> load_vec(const typename Score<DT>::Elem* p) {
  Vec16<DT> v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Classes [c0, c0 + kVec) of a row of C, as FP32; -inf past the row's end.
template <int DT>
__device__ __forceinline__ void load_chunk(const typename Score<DT>::Elem* __restrict__ row, int32_t c0,
                                           int32_t C, float (&f)[Score<DT>::kVec]) {
  constexpr int VE = Score<DT>::kVec;
  if (c0 + VE <= C) {
    const Vec16<DT> v = load_vec<DT>(row + c0);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = Score<DT>::to_f32(v.e[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = c0 + e < C ? Score<DT>::to_f32(row[c0 + e]) : -kInf;
  }
}

// 2^y for y <= 0 in FP64: y = n + r with |r| <= 1/2, the Taylor series of
// e^(r ln 2) to degree 11 (remainder below 7e-15), scaled by 2^n.  NaN stays.
__device__ __forceinline__ double exp2_64(double y) {
  y = y < -1100.0 ? -1100.0 : y;  // (0 in FP64; keeps n in range)
  const double n = __builtin_rint(y);
  const double z = (y - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, z, 1.0 / 3628800.0);
  p = __builtin_fma(p, z, 1.0 / 362880.0);
  p = __builtin_fma(p, z, 1.0 / 40320.0);
  p = __builtin_fma(p, z, 1.0 / 5040.0);
  p = __builtin_fma(p, z, 1.0 / 720.0);
  p = __builtin_fma(p, z, 1.0 / 120.0);
  p = __builtin_fma(p, z, 1.0 / 24.0);
  p = __builtin_fma(p, z, 1.0 / 6.0);
  p = __builtin_fma(p, z, 0.5);
  p = __builtin_fma(p, z, 1.0);
  p = __builtin_fma(p, z, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// 2^y in FP32 (the hardware's exponential; results below 2^-126 become 0).
__device__ __forceinline__ float exp2_32(float y) { return __builtin_amdgcn_exp2f(y); }

__device__ __forceinline__ float wave_max(float v) {
  for (int off = 32; off > 0; off >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_min(float v) {
  for (int off = 32; off > 0; off >>= 1) v = __builtin_fminf(v, __shfl_xor(v, off, 64));
  return v;
}

// Workgroup reductions of one value per thread; every thread gets the result.
// sh: LDS [NT / 64], free again when the call returns.
template <int NT>
__device__ __forceinline__ float block_max(float v, float* sh) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = sh[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) r = __builtin_fmaxf(r, sh[w]);
  __syncthreads();
  return r;
}
template <int NT>
__device__ __forceinline__ float block_min(float v, float* sh) {
  return -block_max<NT>(-v, sh);
}
template <int NT, typename T>
__device__ __forceinline__ T block_sum(T v, T* sh) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = sh[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) r += sh[w];
  __syncthreads();
  return r;
}

// Host checks shared by the entry points.
int check_scores(const gbdt_scores* x);
int check_scores_ws(const gbdt_scores& x, const void* ws, size_t ws_bytes);

}  // namespace gbdt
