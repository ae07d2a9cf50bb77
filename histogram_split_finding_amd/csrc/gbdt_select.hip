// Selections from rows of class scores: a teacher's record (the first k of the
// order, and the mass of the others) and a class drawn with temperature, top-k,
// top-p and min-p from a given random number.
//
// Both come down to places in a row's order (score descending, class
// ascending).  The kept classes of a draw are a prefix of the order whichever
// filters are on, and the draw itself is the place where a running sum passes
// a target.  Two ways to a place:
//  - collect_top (k small): the k-th largest of the threads' own maxima is a
//    lower bound of the k-th largest score; the few scores that reach it are
//    listed in LDS and ranked by counting.
//  - locate (any place, by count or by mass): the scores between two bounds
//    are summed into value bins in LDS (64-bit integers, so the order of the
//    atomics changes nothing), the bin with the target is found, its members
//    are listed and ranked, or, when they are too many, take the place of the
//    bounds; equal scores are counted off in class order.
//
// Masses are integers: rint(e_c 2^s), s = min(50, 62 - ceil(log2 C)), so C of
// them fit 62 bits and a sum is exact.

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "gbdt.h"
#include "gbdt_device.h"
#include "gbdt_internal.h"
#include "gbdt_scores.h"

#pragma clang fp contract(off)

namespace gbdt {

namespace {

constexpr int kBins = 2048;   // value bins of a locate level
constexpr int kList = 1024;   // members that are ranked in LDS
constexpr uint32_t kKeyNegInf = 0x007fffffu;

// Order-preserving key of a score: larger for a larger score, the same for -0
// and +0, that of -inf for NaN.
__device__ __forceinline__ float canon(float x) { return x == x ? x + 0.0f : -kInf; }
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (uint32_t(int32_t(~k) >> 31) | 0x80000000u));
}
// (score, class) as one integer: larger earlier in the order.
__device__ __forceinline__ uint64_t place_of(float x, int32_t c) {
  return uint64_t(key_of(x)) << 32 | uint32_t(~c);
}
__device__ __forceinline__ float score_of(uint64_t p) { return of_key(uint32_t(p >> 32)); }
__device__ __forceinline__ int32_t class_of(uint64_t p) { return int32_t(~uint32_t(p)); }

// A row's e_c = 2^((x - m) c) as FP64 and as an integer of s fraction bits.
struct Mass {
  double m, c, magic;
  bool inf;  // m = +inf: e is 1 for +inf, 0 otherwise
  __device__ __forceinline__ double e(float x) const {
    if (inf) return x == kInf ? 1.0 : 0.0;
    return exp2_64(((double)x - m) * c);
  }
  // rint(e 2^s): added to 2^(52 - s), e's last bit is the sum's last bit
  __device__ __forceinline__ uint64_t q(float x) const {
    return uint64_t(__double_as_longlong(e(x) + magic)) - uint64_t(__double_as_longlong(magic));
  }
};
__device__ __forceinline__ int mass_bits(int32_t C) {
  const int lg = C <= 1 ? 0 : 32 - __builtin_clz(uint32_t(C - 1));
  return 62 - lg < 50 ? 62 - lg : 50;
}
__device__ __forceinline__ Mass make_mass(float m, double c, int bits) {
  Mass r;
  r.inf = m == kInf;
  r.m = (double)m;
  r.c = c;
  r.magic = __builtin_ldexp(1.0, 52 - bits);
  return r;
}

struct SelLds {
  uint64_t hist[kBins];
  uint64_t list[kList];
  uint64_t sorted[kList];
  double shd[16];
  uint64_t shu[16];
  uint64_t found[4];
  float shf[16];
  uint32_t cnt[2][16];
  int32_t sh32[32];
  uint32_t n_list, kmin, kmax;
  int32_t ibest;
};

// Exclusive scan of one uint64 per thread; *total = the sum.
template <int NT>
__device__ inline uint64_t block_scan_u64(uint64_t v, uint64_t* total, uint64_t* sh) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  uint64_t x = v;
  for (int off = 1; off < 64; off <<= 1) {
    const uint64_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) sh[wid] = x;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    if (w < wid) before += sh[w];
    all += sh[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// The k-th largest of the threads' keys (0 when fewer than k are above 0).
template <int NT>
__device__ inline uint32_t kth_key(uint32_t key, int32_t k, uint32_t (*cnt)[16]) {
  uint32_t thr = 0u;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = thr | (1u << bit);
    const uint64_t b = __ballot(key >= trial);
    uint32_t* sh = cnt[bit & 1];  // (two buffers: one barrier a step)
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = uint32_t(__popcll(b));
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) n += sh[w];
    if (n >= (uint32_t)k) thr = trial;
  }
  __syncthreads();
  return thr;
}

// list[0..n) into sorted[], first of the order first (all entries differ).
template <int NT>
__device__ inline void rank_list(SelLds& L, int32_t n) {
  for (int32_t i = threadIdx.x; i < n; i += NT) {
    const uint64_t p = L.list[i];
    int32_t r = 0;
    for (int32_t j = 0; j < n; ++j) r += L.list[j] > p ? 1 : 0;
    L.sorted[r] = p;
  }
  __syncthreads();
}

// What a place search finds: the place, the sum up to and with it, the sum of
// all kept ones.
struct Found {
  uint64_t place, upto, total;
};

// Kept: every place >= keep (places order as integers).  Target: an integer
// running sum; kTargetFrac: ceil(frac total), at least 1; kTargetOver:
// floor(frac total) + 1 (the first running sum above frac total); kTargetCount:
// `count` classes.
enum { kTargetCount, kTargetFrac, kTargetOver };

template <int DT, int NT, int TARGET>
__device__ Found locate(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, uint64_t keep,
                        uint64_t count, double frac, float m, float lowest, int bits, const Mass& mass,
                        SelLds& L) {
  constexpr int VE = Score<DT>::kVec;
  constexpr bool kCount = TARGET == kTargetCount;
  const int tid = threadIdx.x;
  float vhi = m, vlo = __builtin_fmaxf(lowest, score_of(keep));
  if (!kCount) {
    if (mass.inf) {
      vlo = kInf;
    } else {
      // scores whose integer mass is 0 (e < 2^-(s+1)) need no bins
      const float floor_v = (float)((double)m - (double)(bits + 2) / mass.c);
      vlo = __builtin_fmaxf(vlo, __builtin_fminf(floor_v, m));
    }
  }
  uint64_t above = 0, total = 0, target = count;
  bool first = true;
  Found out;
  for (;;) {
    const bool flat = vlo == vhi;
    const bool open = vhi == kInf && !flat;  // +inf in a bin of its own
    const double scale = (double)kBins / ((double)vhi - (double)vlo);
    const double hi = (double)vhi;
    auto bin_of = [&](float v) -> int32_t {
      if (flat) return 0;
      if (open) return v == kInf ? 0 : 1;
      const int32_t b = (int32_t)((hi - (double)v) * scale);
      return b < kBins - 1 ? b : kBins - 1;
    };
    for (int b = tid; b < kBins; b += NT) L.hist[b] = 0ull;
    if (tid == 0) {
      L.n_list = 0u;
      L.kmin = 0xffffffffu;
      L.kmax = 0u;
    }
    __syncthreads();
    if (flat) {
      uint64_t n = 0;
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const float v = canon(f[q]);
          n += v == vhi && place_of(v, c0 + q) >= keep ? 1 : 0;
        }
      }
      const uint64_t w = kCount ? 1ull : mass.q(vhi);
      const uint64_t n_eq = block_sum<NT>(n, L.shu);
      if (first) {
        total = n_eq * w;
        if (TARGET == kTargetFrac) target = (uint64_t)__builtin_ceil(frac * (double)total);
        if (TARGET == kTargetOver) target = (uint64_t)(frac * (double)total) + 1ull;
      }
      if (target < 1) target = 1;
      if (target > total) target = total;
      // the r-th of the equal scores, in class order
      uint64_t r = target > above ? (target - above + w - 1) / (w > 0 ? w : 1) : 1;
      if (r > n_eq) r = n_eq;
      int32_t seen = 0;
      for (int32_t base = 0; base < C; base += NT * VE) {
        const int32_t c0 = base + tid * VE;
        uint32_t eq = 0u;
        if (c0 < C) {
          float f[VE];
          load_chunk<DT>(xr, c0, C, f);
#pragma unroll
          for (int q = 0; q < VE; ++q) {
            const float v = canon(f[q]);
            if (c0 + q < C && v == vhi && place_of(v, c0 + q) >= keep) eq |= 1u << q;
          }
        }
        int32_t sum;
        const int32_t before = seen + block_exclusive_scan(__popc(eq), &sum, L.sh32);
        if ((int64_t)r > before && (int64_t)r <= before + __popc(eq)) {
          int32_t skip = (int32_t)r - before - 1;
          for (; skip > 0; --skip) eq &= eq - 1u;
          L.found[0] = place_of(vhi, c0 + __builtin_ctz(eq));
        }
        seen += sum;
        if ((int64_t)seen >= (int64_t)r) break;
      }
      __syncthreads();
      out.place = L.found[0];
      out.upto = above + r * w;
      out.total = total;
      __syncthreads();
      return out;
    }
    for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
      float f[VE];
      load_chunk<DT>(xr, c0, C, f);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const float v = canon(f[q]);
        if (c0 + q < C && v >= vlo && v <= vhi && v > -kInf && place_of(v, c0 + q) >= keep)
          atomicAdd(reinterpret_cast<unsigned long long*>(&L.hist[bin_of(v)]),
                    kCount ? 1ull : (unsigned long long)mass.q(v));
      }
    }
    __syncthreads();
    // the bin in which the running sum reaches the target
    constexpr int PB = kBins / NT;
    uint64_t mine = 0;
#pragma unroll
    for (int b = 0; b < PB; ++b) mine += L.hist[tid * PB + b];
    uint64_t sum;
    uint64_t run = block_scan_u64<NT>(mine, &sum, L.shu);
    if (first) {
      total = sum;
      if (TARGET == kTargetFrac) target = (uint64_t)__builtin_ceil(frac * (double)total);
      if (TARGET == kTargetOver) target = (uint64_t)(frac * (double)total) + 1ull;
      if (target < 1) target = 1;
      if (target > total) target = total;
      first = false;
    }
    run += above;
#pragma unroll
    for (int b = 0; b < PB; ++b) {
      const uint64_t h = L.hist[tid * PB + b];
      if (run < target && run + h >= target) {
        L.found[0] = uint64_t(tid * PB + b);
        L.found[1] = run;
      }
      run += h;
    }
    __syncthreads();
    const int32_t bin = (int32_t)L.found[0];
    above = L.found[1];
    for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
      float f[VE];
      load_chunk<DT>(xr, c0, C, f);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const float v = canon(f[q]);
        if (c0 + q < C && v >= vlo && v <= vhi && v > -kInf && place_of(v, c0 + q) >= keep &&
            bin_of(v) == bin) {
          const uint32_t at = atomicAdd(&L.n_list, 1u);
          if (at < (uint32_t)kList) L.list[at] = place_of(v, c0 + q);
          atomicMin(&L.kmin, key_of(v));
          atomicMax(&L.kmax, key_of(v));
        }
      }
    }
    __syncthreads();
    const int32_t n = (int32_t)L.n_list;
    if (n <= kList) {
      rank_list<NT>(L, n);
      // running sums in the order, by one wave
      if (tid < 64) {
        uint64_t carry = above;
        for (int32_t b = 0; b < n; b += 64) {
          const int32_t at = b + tid;
          const uint64_t w = at < n ? (kCount ? 1ull : mass.q(score_of(L.sorted[at]))) : 0ull;
          uint64_t x = w;
          for (int off = 1; off < 64; off <<= 1) {
            const uint64_t y = __shfl_up(x, off, 64);
            if (tid >= off) x += y;
          }
          x += carry;
          if (at < n && x >= target && x - w < target) {
            L.found[0] = L.sorted[at];
            L.found[1] = x;
          }
          carry = __shfl(x, 63, 64);
        }
      }
      __syncthreads();
      out.place = L.found[0];
      out.upto = L.found[1];
      out.total = total;
      __syncthreads();
      return out;
    }
    const uint32_t kmin = L.kmin, kmax = L.kmax;
    __syncthreads();
    vlo = of_key(kmin);
    vhi = of_key(kmax);
  }
}

// The first min(k, scores above -inf) places of the order into L.sorted, in
// order; returns how many.  tmax: this thread's largest score.
template <int DT, int NT>
__device__ int32_t collect_top(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, int32_t k,
                               float tmax, float m, float lowest, const Mass& mass, SelLds& L) {
  constexpr int VE = Score<DT>::kVec;
  uint32_t thr = kth_key<NT>(key_of(tmax), k, L.cnt);
  uint64_t keep = uint64_t(thr > kKeyNegInf ? thr : kKeyNegInf + 1u) << 32;
  for (;;) {
    if (threadIdx.x == 0) L.n_list = 0u;
    __syncthreads();
    for (int32_t c0 = threadIdx.x * VE; c0 < C; c0 += NT * VE) {
      float f[VE];
      load_chunk<DT>(xr, c0, C, f);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const uint64_t p = place_of(canon(f[q]), c0 + q);
        if (c0 + q < C && p >= keep) {
          const uint32_t at = atomicAdd(&L.n_list, 1u);
          if (at < (uint32_t)kList) L.list[at] = p;
        }
      }
    }
    __syncthreads();
    const int32_t n = (int32_t)L.n_list;
    if (n <= kList) {
      rank_list<NT>(L, n);
      return n < k ? n : k;
    }
    // too many reach the bound: the exact k-th place (then exactly k are listed)
    __syncthreads();
    keep = locate<DT, NT, kTargetCount>(xr, C, uint64_t(kKeyNegInf + 1u) << 32, (uint64_t)k, 0.0, m, lowest, 0,
                                        mass, L)
               .place;
  }
}

// Largest score of the row, this thread's own, and the lowest above -inf.
template <int DT, int NT>
__device__ void row_range(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, float* m, float* tmax,
                          float* lowest, SelLds& L) {
  constexpr int VE = Score<DT>::kVec;
  float hi = -kInf, lo = kInf;
  for (int32_t c0 = threadIdx.x * VE; c0 < C; c0 += NT * VE) {
    float f[VE];
    load_chunk<DT>(xr, c0, C, f);
#pragma unroll
    for (int q = 0; q < VE; ++q) {
      const float v = canon(f[q]);
      hi = __builtin_fmaxf(hi, v);
      lo = v > -kInf ? __builtin_fminf(lo, v) : lo;
    }
  }
  *tmax = hi;
  *m = block_max<NT>(hi, L.shf);
  *lowest = block_min<NT>(lo, L.shf);
}

// -------------------------------------------------------------- top scores --

struct TopArgs {
  const void* x;
  int64_t n, ld;
  int32_t C, k;
  double c;  // log2(e) / T
  float* values;
  int32_t* classes;
  float* rest;
};

template <int DT, int NT>
__global__ void __launch_bounds__(NT) k_top_block(const TopArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec;
  __shared__ SelLds L;
  const int tid = threadIdx.x;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
    float m, tmax, lowest;
    row_range<DT, NT>(xr, a.C, &m, &tmax, &lowest, L);
    int32_t got = 0;
    if (m > -kInf) {
      const Mass mass = make_mass(m, a.c, mass_bits(a.C));
      got = collect_top<DT, NT>(xr, a.C, a.k, tmax, m, lowest, mass, L);
      if (a.rest != nullptr) {
        const uint64_t last = L.sorted[got - 1];
        const float cf = (float)a.c;
        double in = 0.0, out = 0.0;
        for (int32_t j = tid; j < got; j += NT) in += mass.e(score_of(L.sorted[j]));
        for (int32_t c0 = tid * VE; c0 < a.C; c0 += NT * VE) {
          float f[VE];
          load_chunk<DT>(xr, c0, a.C, f);
#pragma unroll
          for (int q = 0; q < VE; ++q) {
            const float v = canon(f[q]);
            const float w = mass.inf ? (v == kInf ? 1.0f : 0.0f) : exp2_32((v - m) * cf);
            out += c0 + q < a.C && place_of(v, c0 + q) < last ? (double)w : 0.0;
          }
        }
        in = block_sum<NT>(in, L.shd);
        out = block_sum<NT>(out, L.shd);
        if (tid == 0) a.rest[i] = (float)(out / (in + out));
      }
    } else if (a.rest != nullptr && tid == 0) {
      a.rest[i] = 0.0f;
    }
    for (int32_t j = tid; j < a.k; j += NT) {
      a.values[i * a.k + j] = j < got ? score_of(L.sorted[j]) : -kInf;
      a.classes[i * a.k + j] = j < got ? class_of(L.sorted[j]) : -1;
    }
    __syncthreads();
  }
}

// A row of at most CMAX classes in one thread: its places sorted in registers
// (bitonic network, largest first; 0 past the row's end).
template <int DT, int CMAX>
__device__ __forceinline__ void sort_row(const typename Score<DT>::Elem* __restrict__ xr, int32_t C,
                                         uint64_t (&p)[CMAX]) {
#pragma unroll
  for (int c = 0; c < CMAX; ++c) p[c] = c < C ? place_of(canon(Score<DT>::to_f32(xr[c])), c) : 0ull;
#pragma unroll
  for (int len = 2; len <= CMAX; len <<= 1) {
#pragma unroll
    for (int d = len >> 1; d > 0; d >>= 1) {
#pragma unroll
      for (int a = 0; a < CMAX; ++a) {
        const int b = a ^ d;
        if (b > a) {
          const bool down = (a & len) == 0;
          const bool swap = down ? p[a] < p[b] : p[a] > p[b];
          const uint64_t u = swap ? p[b] : p[a], v = swap ? p[a] : p[b];
          p[a] = u;
          p[b] = v;
        }
      }
    }
  }
}

template <int DT, int CMAX>
__global__ void __launch_bounds__(256) k_top_rows(const TopArgs a) {
  using Elem = typename Score<DT>::Elem;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.n) return;
  uint64_t p[CMAX];
  sort_row<DT, CMAX>(static_cast<const Elem*>(a.x) + i * a.ld, a.C, p);
  const float m = score_of(p[0]);
  double in = 0.0, out = 0.0;
  if (a.rest != nullptr && m > -kInf) {
    const Mass mass = make_mass(m, a.c, 50);
#pragma unroll
    for (int c = 0; c < CMAX; ++c) {
      const float v = score_of(p[c]);
      const double e = c < a.C && v > -kInf ? mass.e(v) : 0.0;
      if (c < a.k) in += e; else out += e;
    }
  }
  if (a.rest != nullptr) a.rest[i] = in > 0.0 ? (float)(out / (in + out)) : 0.0f;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    const float v = score_of(p[c]);
    if (c < a.k) {
      a.values[i * a.k + c] = v > -kInf ? v : -kInf;
      a.classes[i * a.k + c] = v > -kInf ? class_of(p[c]) : -1;
    }
  }
}

// ---------------------------------------------------------------- sampling --

struct SampleArgs {
  const void* x;
  int64_t n, ld;
  int32_t C;
  const float* u;
  gbdt_sampling p;
  int32_t* out;
  float* logp;
  int32_t* err;
};

struct RowParams {
  double T, u, top_p, min_p;
  int32_t top_k;
  bool ok;
};

__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t i) {
  RowParams r;
  const float T = a.p.temperature != nullptr ? a.p.temperature[i] : 1.0f;
  const float tp = a.p.top_p != nullptr ? a.p.top_p[i] : 1.0f;
  const float mp = a.p.min_p != nullptr ? a.p.min_p[i] : 0.0f;
  const float u = a.u[i];
  const int32_t k = a.p.top_k != nullptr ? a.p.top_k[i] : 0;
  r.ok = T >= 0.0f && T < kInf && tp >= 0.0f && tp <= 1.0f && mp >= 0.0f && mp <= 1.0f && u >= 0.0f && u < 1.0f;
  r.T = (double)T;
  r.u = (double)u;
  r.top_p = (double)tp;
  r.min_p = (double)mp;
  r.top_k = k <= 0 || k > a.C ? a.C : k;
  if (T == 0.0f) r.top_k = 1;
  return r;
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT) k_sample_block(const SampleArgs a) {
  using Elem = typename Score<DT>::Elem;
  __shared__ SelLds L;
  const int tid = threadIdx.x;
  const int bits = mass_bits(a.C);
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
    const RowParams r = row_params(a, i);
    float m = -kInf, tmax = -kInf, lowest = -kInf;
    if (r.ok) row_range<DT, NT>(xr, a.C, &m, &tmax, &lowest, L);
    if (!(m > -kInf)) {
      if (tid == 0) {
        if (!r.ok) dev_error(a.err, GBDT_E_RANGE);
        a.out[i] = -1;
        if (a.logp != nullptr) a.logp[i] = -kInf;
      }
      continue;
    }
    const Mass mass = make_mass(m, r.T > 0.0 ? kLog2e / r.T : 0.0, bits);
    uint64_t place = 0, total = 0;
    if (r.top_k <= GBDT_MAX_LISTED) {
      const int32_t got = collect_top<DT, NT>(xr, a.C, r.top_k, tmax, m, lowest, mass, L);
      // running sums over the list, then its two cuts and the draw, by one wave
      if (tid < 64) {
        constexpr int PL = GBDT_MAX_LISTED / 64;
        uint64_t w[PL], run[PL], carry = 0;
#pragma unroll
        for (int b = 0; b < PL; ++b) {
          const int32_t at = b * 64 + tid;
          w[b] = at < got ? mass.q(score_of(L.sorted[at])) : 0ull;
          uint64_t x = w[b];
          for (int off = 1; off < 64; off <<= 1) {
            const uint64_t y = __shfl_up(x, off, 64);
            if (tid >= off) x += y;
          }
          run[b] = x + carry;
          carry = __shfl(run[b], 63, 64);
        }
        const uint64_t target =
            r.top_p < 1.0 ? (uint64_t)__builtin_ceil(r.top_p * (double)carry) : ~uint64_t(0);
        uint64_t W = 0;
#pragma unroll
        for (int b = 0; b < PL; ++b) {
          const int32_t at = b * 64 + tid;
          const bool kept = at < got && w[b] > 0 && (at == 0 || run[b] - w[b] < target) &&
                            (at == 0 || mass.e(score_of(L.sorted[at])) >= r.min_p);
          if (kept) W = run[b];  // (a prefix is kept: the last one's running sum is the largest)
        }
        for (int off = 32; off > 0; off >>= 1) {
          const uint64_t y = __shfl_xor(W, off, 64);
          W = y > W ? y : W;
        }
        uint64_t over = (uint64_t)(r.u * (double)W) + 1ull;
        if (over > W) over = W;
#pragma unroll
        for (int b = 0; b < PL; ++b) {
          if (b * 64 + tid < got && run[b] >= over && run[b] - w[b] < over) L.found[0] = L.sorted[b * 64 + tid];
        }
        if (tid == 0) L.found[1] = W;
      }
      __syncthreads();
      place = L.found[0];
      total = L.found[1];
    } else {
      uint64_t keep = uint64_t(kKeyNegInf + 1u) << 32;
      if (r.top_k < a.C)
        keep = locate<DT, NT, kTargetCount>(xr, a.C, keep, (uint64_t)r.top_k, 0.0, m, lowest, bits, mass, L).place;
      if (r.top_p < 1.0)
        keep = locate<DT, NT, kTargetFrac>(xr, a.C, keep, 0, r.top_p, m, lowest, bits, mass, L).place;
      if (r.min_p > 0.0 && !mass.inf) {
        // e >= min_p exactly where x >= m + log2(min_p) / c
        const double v = mass.m + log2(r.min_p) / mass.c;
        const float f = (float)v + 0.0f;
        uint64_t cut = uint64_t(key_of(f) + ((double)f < v ? 1u : 0u)) << 32;
        const uint64_t top = uint64_t(key_of(m)) << 32;
        cut = cut < top ? cut : top;
        keep = cut > keep ? cut : keep;
      }
      const Found f = locate<DT, NT, kTargetOver>(xr, a.C, keep, 0, r.u, m, lowest, bits, mass, L);
      place = f.place;
      total = f.total;
    }
    if (tid == 0) {
      a.out[i] = class_of(place);
      if (a.logp != nullptr) {
        const double x = (double)score_of(place);
        const double d = mass.inf || r.T == 0.0 ? 0.0 : (x - mass.m) / r.T;
        a.logp[i] = (float)(d - log(__builtin_ldexp((double)total, -bits)));
      }
    }
    __syncthreads();
  }
}

template <int DT, int CMAX>
__global__ void __launch_bounds__(256) k_sample_rows(const SampleArgs a) {
  using Elem = typename Score<DT>::Elem;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.n) return;
  const RowParams r = row_params(a, i);
  uint64_t p[CMAX];
  sort_row<DT, CMAX>(static_cast<const Elem*>(a.x) + i * a.ld, a.C, p);
  const float m = score_of(p[0]);
  if (!r.ok || !(m > -kInf)) {
    if (!r.ok) dev_error(a.err, GBDT_E_RANGE);
    a.out[i] = -1;
    if (a.logp != nullptr) a.logp[i] = -kInf;
    return;
  }
  const Mass mass = make_mass(m, r.T > 0.0 ? kLog2e / r.T : 0.0, 50);
  double e[CMAX], all = 0.0;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    const float v = score_of(p[c]);
    e[c] = c < r.top_k && c < a.C && v > -kInf ? mass.e(v) : 0.0;
    all += e[c];
  }
  const double most = r.top_p < 1.0 ? r.top_p * all : kInf;
  double run = 0.0, W = 0.0;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    const bool kept = c == 0 || (run < most && e[c] >= r.min_p && e[c] > 0.0);
    run += e[c];
    e[c] = kept ? e[c] : 0.0;
    W += e[c];
  }
  const double over = r.u * W;
  uint64_t place = p[0];
  double ew = e[0];
  run = 0.0;
  bool done = false;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    run += e[c];
    // (the last kept one where rounding leaves none)
    if (!done && e[c] > 0.0) {
      place = p[c];
      ew = e[c];
      done = run > over;
    }
  }
  a.out[i] = class_of(place);
  if (a.logp != nullptr) a.logp[i] = (float)log(ew / W);
}

template <int DT>
int launch_top(const TopArgs& a, hipStream_t s) {
  diag_begin(kDiagTopScores, s);
  const dim3 lanes((unsigned)((a.n + 255) / 256));
  const dim3 rows((unsigned)(a.n < kMaxRowGrid ? a.n : kMaxRowGrid));
  if (a.C <= 8)
    hipLaunchKernelGGL((k_top_rows<DT, 8>), lanes, dim3(256), 0, s, a);
  else if (a.C <= 16)
    hipLaunchKernelGGL((k_top_rows<DT, 16>), lanes, dim3(256), 0, s, a);
  else if (a.C <= kRowsMaxClasses)
    hipLaunchKernelGGL((k_top_rows<DT, 32>), lanes, dim3(256), 0, s, a);
  else if (a.C <= 8192)
    hipLaunchKernelGGL((k_top_block<DT, 256>), rows, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_top_block<DT, 1024>), rows, dim3(1024), 0, s, a);
  diag_end(s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_top");
}

template <int DT>
int launch_sample(const SampleArgs& a, hipStream_t s) {
  diag_begin(kDiagSample, s);
  const dim3 lanes((unsigned)((a.n + 255) / 256));
  const dim3 rows((unsigned)(a.n < kMaxRowGrid ? a.n : kMaxRowGrid));
  if (a.C <= 8)
    hipLaunchKernelGGL((k_sample_rows<DT, 8>), lanes, dim3(256), 0, s, a);
  else if (a.C <= 16)
    hipLaunchKernelGGL((k_sample_rows<DT, 16>), lanes, dim3(256), 0, s, a);
  else if (a.C <= kRowsMaxClasses)
    hipLaunchKernelGGL((k_sample_rows<DT, 32>), lanes, dim3(256), 0, s, a);
  else if (a.C <= 8192)
    hipLaunchKernelGGL((k_sample_block<DT, 256>), rows, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_sample_block<DT, 1024>), rows, dim3(1024), 0, s, a);
  diag_end(s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_sample");
}

}  // namespace

}  // namespace gbdt

using namespace gbdt;

extern "C" {

int gbdt_top_scores(const gbdt_scores* x, int32_t k, float temperature, float* values, int32_t* classes,
                    float* rest, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_scores(x);
  if (rc) return rc;
  if (k < 1 || k > GBDT_MAX_LISTED) return fail(GBDT_E_ARG, "k out of [1, GBDT_MAX_LISTED]");
  if (k > x->n_classes) return fail(GBDT_E_SHAPE, "k larger than n_classes");
  if (!std::isfinite(temperature) || !(temperature > 0.0f))
    return fail(GBDT_E_ARG, "temperature must be finite and > 0");
  if (x->n_rows == 0) return GBDT_OK;
  if (!values || !classes) return fail(GBDT_E_ARG, "values or classes is null");
  rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  TopArgs a;
  a.x = x->data;
  a.n = x->n_rows;
  a.ld = x->row_stride;
  a.C = x->n_classes;
  a.k = k;
  a.c = kLog2e / (double)temperature;
  a.values = values;
  a.classes = classes;
  a.rest = rest;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (x->dtype) {
    case GBDT_DTYPE_F32: return launch_top<GBDT_DTYPE_F32>(a, s);
    case GBDT_DTYPE_BF16: return launch_top<GBDT_DTYPE_BF16>(a, s);
    default: return launch_top<GBDT_DTYPE_F16>(a, s);
  }
}

int gbdt_sample_classes(const gbdt_scores* x, const float* u, const gbdt_sampling* p, int32_t* out,
                        float* logp, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_scores(x);
  if (rc) return rc;
  if (!p) return fail(GBDT_E_ARG, "sampling parameters are null");
  if (x->n_rows == 0) return GBDT_OK;
  if (!u || !out) return fail(GBDT_E_ARG, "u or out is null");
  rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  SampleArgs a;
  a.x = x->data;
  a.n = x->n_rows;
  a.ld = x->row_stride;
  a.C = x->n_classes;
  a.u = u;
  a.p = *p;
  a.out = out;
  a.logp = logp;
  a.err = &static_cast<WsCtrl*>(ws)->err;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (x->dtype) {
    case GBDT_DTYPE_F32: return launch_sample<GBDT_DTYPE_F32>(a, s);
    case GBDT_DTYPE_BF16: return launch_sample<GBDT_DTYPE_BF16>(a, s);
    default: return launch_sample<GBDT_DTYPE_F16>(a, s);
  }
}

}  // extern "C"
