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

// 16 bytes of scores, as words (elements of two bytes would take a register
// each).  A row may start at any element, so the loads and stores are by the
// element's alignment; gfx950 does them in one access.
template <int DT>
struct Vec16 {
  uint32_t w[4];
};

template <int DT>
__device__ __forceinline__ Vec16<DT> load_vec(const typename Score<DT>::Elem* p) {
  Vec16<DT> v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

template <int DT>
__device__ __forceinline__ void unpack(const Vec16<DT>& v, float (&f)[Score<DT>::kVec]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == GBDT_DTYPE_F32) {
      f[e] = __uint_as_float(v.w[e]);
    } else if constexpr (DT == GBDT_DTYPE_BF16) {
      f[2 * e] = __uint_as_float(v.w[e] << 16);
      f[2 * e + 1] = __uint_as_float(v.w[e] & 0xffff0000u);
    } else {
      f[2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)v.w[e]);
      f[2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v.w[e] >> 16));
    }
  }
}

template <int DT>
__device__ __forceinline__ Vec16<DT> pack(const float (&f)[Score<DT>::kVec]) {
  Vec16<DT> v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == GBDT_DTYPE_F32) {
      v.w[e] = __float_as_uint(f[e]);
    } else {
      using E2 = typename Score<DT>::Elem __attribute__((ext_vector_type(2)));
      const E2 p = {Score<DT>::from_f32(f[2 * e]), Score<DT>::from_f32(f[2 * e + 1])};
      v.w[e] = __builtin_bit_cast(uint32_t, p);
    }
  }
  return v;
}

// Elements [c, c + kVec) of a row of C, c < C or not: -inf past the row's end.
// The vector that the end cuts is the row's last one, shifted down: one load
// (a load for each element would be a chain of latencies in every short row).
template <int DT>
__device__ __forceinline__ Vec16<DT> load_tail(const typename Score<DT>::Elem* __restrict__ row, int32_t c, int32_t C) {
  constexpr int VE = Score<DT>::kVec;
  if (c + VE <= C) return load_vec<DT>(row + c);
  constexpr uint32_t inf = DT == GBDT_DTYPE_F32 ? 0xff800000u : DT == GBDT_DTYPE_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  Vec16<DT> v = {{inf, inf, inf, inf}};
  if (c >= C) return v;
  if (C < VE) {
#pragma unroll 1
    for (int32_t e = C - 1; e >= c; --e) {
      if constexpr (DT == GBDT_DTYPE_F32) {
        v = {{__float_as_uint(row[e]), v.w[0], v.w[1], v.w[2]}};
      } else {
        const uint32_t x = __builtin_bit_cast(uint16_t, row[e]);
        v = {{v.w[0] << 16 | x, v.w[1] << 16 | v.w[0] >> 16, v.w[2] << 16 | v.w[1] >> 16,
              v.w[3] << 16 | v.w[2] >> 16}};
      }
    }
    return v;
  }
  v = load_vec<DT>(row + (C - VE));
  int32_t down = c + VE - C;  // elements, 1 .. VE - 1
  if constexpr (DT != GBDT_DTYPE_F32) {
    if (down & 1)
      v = {{v.w[0] >> 16 | v.w[1] << 16, v.w[1] >> 16 | v.w[2] << 16, v.w[2] >> 16 | v.w[3] << 16,
            v.w[3] >> 16 | (inf & 0xffff0000u)}};
    down >>= 1;
  }
  if (down & 1) v = {{v.w[1], v.w[2], v.w[3], inf}};
  if (down & 2) v = {{v.w[2], v.w[3], inf, inf}};
  return v;
}

template <int DT>
__device__ __forceinline__ void store_tail(typename Score<DT>::Elem* __restrict__ row, int32_t c, int32_t C,
                                           Vec16<DT> v) {
  if (c + Score<DT>::kVec <= C) {
    __builtin_memcpy(row + c, &v, 16);
    return;
  }
#pragma unroll 1
  for (; c < C; ++c) {
    if constexpr (DT == GBDT_DTYPE_F32) {
      row[c] = __uint_as_float(v.w[0]);
      v = {{v.w[1], v.w[2], v.w[3], 0u}};
    } else {
      row[c] = __builtin_bit_cast(typename Score<DT>::Elem, (uint16_t)v.w[0]);
      v = {{v.w[0] >> 16 | v.w[1] << 16, v.w[1] >> 16 | v.w[2] << 16, v.w[2] >> 16 | v.w[3] << 16, v.w[3] >> 16}};
    }
  }
}

// Classes [c0, c0 + kVec) of a row of C, as FP32; -inf past the row's end.
template <int DT>
__device__ __forceinline__ void load_chunk(const typename Score<DT>::Elem* __restrict__ row, int32_t c0,
                                           int32_t C, float (&f)[Score<DT>::kVec]) {
  unpack<DT>(load_tail<DT>(row, c0, C), f);
}

// A constant in scalar registers: fma(p, r, constant) is then one instruction.
// (From a literal the compiler makes two moves and a multiply-accumulate.)
__device__ __forceinline__ double scalar_const(double c) {
  asm("" : "+s"(c));
  return c;
}

// 2^y for -1020 <= y <= 1 in FP64: y = n + r with |r| <= 1/2 (n by adding
// 1.5 2^52, whose last bit is 1), 2^r = 1 + r Q(r) with Q the degree-9
// polynomial through (2^r - 1) / r at the Chebyshev nodes of [-1/2, 1/2]
// (relative error 5.7e-16, 1 at r = 0), n added to the exponent.
// 14 instructions, FP64 ones at the FP32 rate.
__device__ __forceinline__ double exp2_64_near(double y) {
  const double t = y + 0x1.8p52;
  const double r = y - (t - 0x1.8p52);
  double p = __builtin_fma(r, scalar_const(0x1.e5e9f550503fcp-28), scalar_const(0x1.b6571deaf97c8p-24));
  p = __builtin_fma(p, r, scalar_const(0x1.62bfe4611405ap-20));
  p = __builtin_fma(p, r, scalar_const(0x1.ffcb7678915a9p-17));
  p = __builtin_fma(p, r, scalar_const(0x1.430913037846ep-13));
  p = __builtin_fma(p, r, scalar_const(0x1.5d87fe908f8a8p-10));
  p = __builtin_fma(p, r, scalar_const(0x1.3b2ab6fba385fp-7));
  p = __builtin_fma(p, r, scalar_const(0x1.c6b08d7044119p-5));
  p = __builtin_fma(p, r, scalar_const(0x1.ebfbdff82c590p-3));
  p = __builtin_fma(p, r, scalar_const(0x1.62e42fefa39f7p-1));
  p = __builtin_fma(p, r, 1.0);
  const int32_t n = __double2loint(t);
  return __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
}
// The same, 0 for y below -1020; NaN stays.
__device__ __forceinline__ double exp2_64(double y) {
  const double e = exp2_64_near(y);
  return y < -1020.0 ? 0.0 : e;
}

// 1 / x in FP64 for normal x > 0: the hardware's estimate and two Newton steps
// (5 instructions; a division takes three times that).
__device__ __forceinline__ double rcp_64(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

// log x in FP64 (0: -inf; NaN stays): x = 2^n f, y the hardware's FP32 log2 f,
// and f 2^-y = 1 + d with |d| < 2^-18, whose logarithm is d - d^2 / 2 + d^3 / 3.
__device__ __forceinline__ double log_64(double x) {
  const double f = __builtin_amdgcn_frexp_mant(x);
  const double y = (double)__builtin_amdgcn_logf((float)f);
  const double d = __builtin_fma(f, exp2_64(-y), -1.0);
  const double t = __builtin_fma(d * d, __builtin_fma(d, 1.0 / 3.0, -0.5), d);
  const double l = __builtin_fma((double)__builtin_amdgcn_frexp_exp(x) + y, 0.69314718055994530942, t);
  return x > 0.0 && x < __builtin_inf() ? l : (x == 0.0 ? -__builtin_inf() : x);
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

// The same within groups of NT lanes (NT <= 64).
template <int NT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = (NT < 64 ? NT : 64) / 2; off > 0; off >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
template <int NT>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
  for (int off = (NT < 64 ? NT : 64) / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The waves' values sh[W] combined, in every lane (behind a barrier).
template <int W, typename T, typename F>
__device__ __forceinline__ T across_waves(const T* sh, F f) {
  T v = sh[threadIdx.x & (W - 1)];
#pragma unroll
  for (int off = 1; off < W; off <<= 1) v = f(v, __shfl_xor(v, off, 64));
  return v;
}

// Workgroup reductions of one value per thread; every thread gets the result.
// sh: LDS [NT / 64], free again when the call returns.
template <int NT>
__device__ __forceinline__ float block_max(float v, float* sh) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  const float r = across_waves<NT / 64>(sh, [](float a, float b) { return __builtin_fmaxf(a, b); });
  __syncthreads();
  return r;
}
template <int NT, typename T>
__device__ __forceinline__ T block_sum(T v, T* sh) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  const T r = across_waves<NT / 64>(sh, [](T a, T b) { return a + b; });
  __syncthreads();
  return r;
}

// A workgroup's elements of a row come in blocks of NT * kBlk: kVecs vectors
// of 16 bytes per thread, NT * kVec elements apart, so a wave's load is 1 KB
// in a row.
constexpr int kVecs = 4;
template <int DT>
constexpr int kBlk = kVecs * Score<DT>::kVec;

template <int DT>
struct RawBlock {
  Vec16<DT> v[kVecs];
};

// The thread's share of the block at `base`, -inf past C.
template <int DT, int NT>
__device__ __forceinline__ RawBlock<DT> load_block(const typename Score<DT>::Elem* __restrict__ row, int32_t base,
                                                   int32_t C) {
  constexpr int VE = Score<DT>::kVec;
  RawBlock<DT> r;
  const int32_t c0 = base + (int32_t)(threadIdx.x & (NT - 1)) * VE;
  if (base + NT * kBlk<DT> <= C) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) r.v[j] = load_vec<DT>(row + c0 + j * NT * VE);
  } else {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) r.v[j] = load_tail<DT>(row, c0 + j * NT * VE, C);
  }
  return r;
}

// All blocks of a row, the next one on its way while one is worked on.
template <int DT, int NT, typename Work>
__device__ __forceinline__ void each_block(const typename Score<DT>::Elem* __restrict__ row, int32_t C, Work work) {
  RawBlock<DT> raw = load_block<DT, NT>(row, 0, C);
  for (int32_t base = 0;;) {
    RawBlock<DT> next;
    const bool more = base + NT * kBlk<DT> < C;
    if (more) next = load_block<DT, NT>(row, base + NT * kBlk<DT>, C);
    __builtin_amdgcn_sched_barrier(0);
    work(raw, base);
    if (!more) break;
    base += NT * kBlk<DT>;
    raw = next;
  }
}

// The stores are marked as not read again soon: they leave the caches to the
// scores, which a step reads twice (4,096 rows of 131,072 bf16 classes, loss and
// gradient: 445 us with the mark, 491 us without).
template <int DT, int NT>
__device__ __forceinline__ void store_block(typename Score<DT>::Elem* __restrict__ row, int32_t base, int32_t C,
                                            const RawBlock<DT>& r) {
  constexpr int VE = Score<DT>::kVec;
  using Words = uint32_t __attribute__((ext_vector_type(4), aligned(2)));
  const int32_t c0 = base + (int32_t)(threadIdx.x & (NT - 1)) * VE;
  if (base + NT * kBlk<DT> <= C) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const Words o = {r.v[j].w[0], r.v[j].w[1], r.v[j].w[2], r.v[j].w[3]};
      __builtin_nontemporal_store(o, reinterpret_cast<Words*>(row + c0 + j * NT * VE));
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) store_tail<DT>(row, c0 + j * NT * VE, C, r.v[j]);
  }
}

template <int N>
__device__ __forceinline__ float max_of(const float (&f)[N]) {
  float m = f[0];
#pragma unroll
  for (int e = 1; e < N; ++e) m = __builtin_fmaxf(m, f[e]);
  return m;
}

// Sum by halves: at most log2 N roundings of each term.
template <int N>
__device__ __forceinline__ float sum_of(const float (&f)[N]) {
  static_assert(N == 4 || N == 8, "");
  const float a = (f[0] + f[1]) + (f[2] + f[3]);
  if (N == 4) return a;
  return a + ((f[4 % N] + f[5 % N]) + (f[6 % N] + f[7 % N]));
}

// Quotients e / C by a product with inv = ceil(2^20 / C), right as long as
// e (inv C - 2^20) < 2^20, where the bracket is at most C - 1.
template <int R, int CMAX>  // e below R C, C up to CMAX
constexpr bool kRowDivExact = (R * CMAX - 1) * (CMAX - 1) < 1 << 20;
struct RowDiv {
  uint32_t inv;
  __device__ explicit RowDiv(int32_t C) : inv(((1u << 20) + (uint32_t)C - 1u) / (uint32_t)C) {}
  // (both factors below 2^24, the quotient below 2^9: the 24-bit product is exact)
  __device__ __forceinline__ int32_t operator()(int32_t e) const { return int32_t(__umul24((uint32_t)e, inv) >> 20); }
};

constexpr int64_t kMaxRowGrid = 1 << 20;  // rows of one launch, at most
// Rows are shared by several workgroups when there are at most kSplitRows of
// them: about kSplitGrid workgroups in all.
constexpr int64_t kSplitRows = 128, kSplitGrid = 512;

// log2(e) / T as a factor of FP32 differences (finite, so 0 times it is 0).
__device__ __forceinline__ float exponent_scale(double c) { return c < 3.0e38 ? (float)c : 3.0e38f; }

// One thread per row: CMAX elements of R rows of `width` (at most CMAX), loaded
// by all threads in whole lines, and laid down in LDS rows of width | 1 words.
template <int R, int CMAX, typename T>
struct Staged {
  static_assert(kRowDivExact<R, CMAX>, "the quotients of these rows are not exact");
  T v[CMAX];
  template <typename LoadFlat, typename LoadAt>
  __device__ __forceinline__ void load(int32_t rows, int32_t width, bool flat, const RowDiv& div, LoadFlat at_flat,
                                       LoadAt at) {
    if (flat) {
#pragma unroll
      for (int u = 0; u < CMAX; ++u) {
        const int32_t e = (int32_t)threadIdx.x + u * R;
        if (u < width && e < rows * width) v[u] = at_flat(e);
      }
    } else {
#pragma unroll
      for (int u = 0; u < CMAX; ++u) {
        const int32_t e = (int32_t)threadIdx.x + u * R, row = div(e);
        if (u < width && e < rows * width) v[u] = at(row, e - __mul24(row, width));
      }
    }
  }
  __device__ __forceinline__ void put(int32_t rows, int32_t width, const RowDiv& div, T* lds) const {
#pragma unroll
    for (int u = 0; u < CMAX; ++u) {
      const int32_t e = (int32_t)threadIdx.x + u * R;
      if (u < width && e < rows * width) lds[width & 1 ? e : e + div(e)] = v[u];
    }
  }
};
// The way back.
template <int R, int CMAX, typename T, typename PutFlat, typename PutAt>
__device__ __forceinline__ void unstage(int32_t rows, int32_t width, bool flat, const RowDiv& div, const T* lds,
                                        PutFlat put_flat, PutAt put) {
  if (flat) {
#pragma unroll
    for (int u = 0; u < CMAX; ++u) {
      const int32_t e = (int32_t)threadIdx.x + u * R;
      if (u < width && e < rows * width) put_flat(e, lds[width & 1 ? e : e + div(e)]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < CMAX; ++u) {
      const int32_t e = (int32_t)threadIdx.x + u * R, row = div(e);
      if (u < width && e < rows * width)
        put(row, e - __mul24(row, width), lds[width & 1 ? e : e + row]);
    }
  }
}

// Workspace of the row calls: the control block, then partial results of rows
// that several workgroups share.
constexpr size_t kScoresPartBytes = size_t(1) << 20;

// Host checks shared by the entry points.
int check_scores(const gbdt_scores* x);
int check_scores_ws(const gbdt_scores& x, const void* ws, size_t ws_bytes);

}  // namespace gbdt
