// Selections from rows of class scores: a teacher's record (the first k of the
// order, and the mass of the others) and a class drawn with temperature, top-k,
// top-p and min-p from a given random number.
//
// Both come down to places in a row's order (score descending, class
// ascending).  The kept classes of a draw are a prefix of the order whichever
// filters are on, and the draw itself is the place where a running sum passes
// a target.
//  - One pass over the row lists in LDS the few classes that reach a threshold
//    and adds up what lies below it (a record's rest, a draw's other masses).
//    The threshold comes from the row's first block: the r-th largest of its
//    threads' (or of four times as many groups') maxima, r so that the whole
//    row should list about twice what is needed.  The list is ranked by
//    counting.  Records, draws with top-k, and draws whose cut and target fall
//    on listed classes are complete then, from one read of the row.
//  - A row that lists too few or too many, and other draws: counts or masses
//    are summed into value bins in LDS (64-bit integers, so the order of the
//    atomics changes nothing), the bin with the target is found, and its members
//    are listed and ranked; members that are too many take the place of the row,
//    and equal scores are counted off in class order.
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
// (score, class) as one integer: larger earlier in the order.  The bits are
// those of an FP64 number in [2, 4), whose comparison is one full-rate
// instruction (an integer one of 64 bits takes four times that).
constexpr int kClassBits = 20;
static_assert(GBDT_MAX_CLASSES <= 1 << kClassBits, "a place holds any class");
__device__ __forceinline__ uint64_t first_place(uint32_t key) {  // below all places of the key
  return uint64_t(1) << 62 | uint64_t(key) << kClassBits;
}
__device__ __forceinline__ uint64_t place_of(float x, int32_t c) {
  return first_place(key_of(x)) | uint32_t((1 << kClassBits) - 1 - c);
}
__device__ __forceinline__ float score_of(uint64_t p) { return of_key(uint32_t(p >> kClassBits)); }
__device__ __forceinline__ int32_t class_of(uint64_t p) {
  return (1 << kClassBits) - 1 - int32_t(p & ((1u << kClassBits) - 1u));
}

// A row's e_c = 2^((x - m) c) as FP64 and as an integer of s fraction bits.
struct Mass {
  double m, c, magic, low;  // low: 2^low rounds to mass 0
  bool inf;                 // m = +inf: e is 1 for +inf, 0 otherwise
  __device__ __forceinline__ double e(float x) const {
    if (inf) return x == kInf ? 1.0 : 0.0;
    return exp2_64(((double)x - m) * c);
  }
  // rint(e 2^s): added to 2^(52 - s), e's last bit is the sum's last bit
  __device__ __forceinline__ uint64_t raw(double e) const { return uint64_t(__double_as_longlong(e + magic)); }
  __device__ __forceinline__ uint64_t raw_zero() const { return uint64_t(__double_as_longlong(magic)); }
  __device__ __forceinline__ uint64_t q(float x) const { return raw(e(x)) - raw_zero(); }
  // the same plus raw_zero() for any score (NaN: 0) of a row whose m is finite;
  // d = x - m
  __device__ __forceinline__ uint64_t raw_at(double d) const {
    return raw(exp2_64_near(__builtin_fmax(d * c, low)));
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
  r.low = -(double)(bits + 2);
  return r;
}

// Waves per SIMD of the record kernel.
template <int NT>
constexpr int kHotWaves = NT == 64 ? 4 : 6;

template <int NT>
struct ListLds {
  static constexpr int kList = NT == 64 ? 512 : 1024;  // members that are ranked in LDS
  alignas(16) uint64_t list[kList];
  uint64_t sorted[kList];
  uint64_t shu[16];
  double shd[16];
  uint64_t cnt[2][16];
  uint64_t found[4];
  float shf[2][16];
  int32_t sh32[32];
  uint32_t n_list, kmin, kmax, n_vec;
  // vectors with a class that reaches the threshold, and where they begin
  static constexpr int kVectors = NT > 256 ? kList : 1;
  alignas(16) uint32_t vec[4 * kVectors];
  int32_t vec_at[kVectors];
};
template <int NT>
struct SelLds : ListLds<NT> {
  static constexpr int kBins = NT == 64 ? 256 : 2048;  // value bins of a locate level
  uint64_t hist[kBins];
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

// A key that at least k of the groups' maxima gm (all scores above -inf, if
// those are fewer) reach, and not many more than k; m, lowest: the largest and
// the smallest of the maxima.
template <int NT>
__device__ uint32_t group_threshold(const float (&gm)[kVecs], float m, float lowest, int32_t k, ListLds<NT>& L) {
  // (with 1,024 threads their own maxima are enough groups)
  constexpr int G = NT >= 1024 ? 1 : kVecs;
  uint32_t key[G];
#pragma unroll
  for (int j = 0; j < G; ++j) key[j] = key_of(gm[j]);
  if (G == 1) key[0] = key_of(max_of(gm));
  if (k > G * NT) return kKeyNegInf + 1u;
  uint32_t lo = key_of(lowest), hi = key_of(m) + 1u;  // reached by >= k, by none
  lo = lo > kKeyNegInf ? lo : kKeyNegInf + 1u;
  for (int step = 0; hi - lo > 1u; ++step) {
    // three points of the interval at a time: half the barriers
    // (quarters of the values first, of the keys if that is not enough)
    const uint32_t q = (hi - lo) / 4u;
    uint32_t p1 = lo + q, p2 = lo + (hi - lo) / 2u, p3 = p2 + q;
    if (step < 6 && hi <= 0xff800000u) {
      const float a = of_key(lo), d = of_key(hi) * 0.25f - a * 0.25f;
      const uint32_t v1 = key_of(a + d), v2 = key_of(a + 2.0f * d), v3 = key_of(a + 3.0f * d);
      if (lo < v1 && v1 < v2 && v2 < v3 && v3 < hi) {
        p1 = v1;
        p2 = v2;
        p3 = v3;
      }
    }
    p1 = p1 > lo ? p1 : p2;
    uint64_t n = 0;  // three counts of 21 bits
    if (NT == 64) {
      // (one wave has no barriers to save: the middle alone)
      int32_t n2 = 0;
#pragma unroll
      for (int j = 0; j < G; ++j) n2 += __popcll(__ballot(key[j] >= p2));
      if (n2 >= k) {
        lo = p2;
        if (n2 <= k + k / 4 + 8) break;
      } else {
        hi = p2;
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      n += uint64_t(__popcll(__ballot(key[j] >= p1)));
      n += uint64_t(__popcll(__ballot(key[j] >= p2))) << 21;
      n += uint64_t(__popcll(__ballot(key[j] >= p3))) << 42;
    }
    if (NT > 64) {
      uint64_t* sh = L.cnt[step & 1];  // (two buffers: one barrier a step)
      if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = n;
      __syncthreads();
      n = across_waves<NT / 64>(sh, [](uint64_t a, uint64_t b) { return a + b; });
    }
    const int32_t n1 = int32_t(n & 0x1fffffu), n2 = int32_t(n >> 21 & 0x1fffffu), n3 = int32_t(n >> 42);
    int32_t at_lo;
    if (n3 >= k) {
      lo = p3;
      at_lo = n3;
    } else if (n2 >= k) {
      lo = p2;
      hi = p3;
      at_lo = n2;
    } else if (n1 >= k) {
      lo = p1;
      hi = p2;
      at_lo = n1;
    } else {
      hi = p1;
      continue;
    }
    if (at_lo <= k + k / 4 + 8) break;
  }
  if (NT > 64) __syncthreads();
  return lo;
}

// list[0..n) into sorted[], first of the order first (all entries differ): each
// entry's place is the number of entries before it.  Eight entries are read at
// a time, for all of the thread's own ones.
template <int NT>
__device__ inline void rank_list(ListLds<NT>& L, int32_t n) {
  constexpr int PT = NT == 64 ? 4 : NT == 256 ? 2 : 1;
  const int tid = threadIdx.x;
  const int32_t n8 = (n + 7) & ~7;
  double* list = reinterpret_cast<double*>(L.list);
  double* sorted = reinterpret_cast<double*>(L.sorted);
  if (tid < n8 - n) list[n + tid] = 0.0;
  __syncthreads();
  for (int32_t i0 = 0; i0 < n; i0 += PT * NT) {
    double p[PT];
    int32_t r[PT];
#pragma unroll
    for (int u = 0; u < PT; ++u) {
      const int32_t i = i0 + tid + u * NT;
      p[u] = i < n ? list[i] : 4.0;
      r[u] = 0;
    }
    if (i0 + (tid & ~63) < n) {  // (whole waves)
      for (int32_t j = 0; j < n8; j += 8) {
        double e[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) e[v] = list[j + v];
#pragma unroll
        for (int u = 0; u < PT; ++u) {
          if (u == 0 || u * NT < n - i0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) r[u] += e[v] > p[u] ? 1 : 0;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < PT; ++u)
      if (i0 + tid + u * NT < n) sorted[r[u]] = p[u];
  }
  __syncthreads();
}

// The value of the first lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}
__device__ __forceinline__ double uniform(double x) {
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(x)),
                          __builtin_amdgcn_readfirstlane(__double2loint(x)));
}

// Bins of the exponents y = (x - ref) c in [low, 0].
template <int NB>
__device__ __forceinline__ int32_t bin_of_exponent(double y, double scale) {
  const int32_t b = (int32_t)(y * scale);
  return b < NB - 1 ? b : NB - 1;
}

// What the pass over a row gives: the maximum, how many classes reached the
// threshold (the first kList of them are in L.list), and the sum of the others'
// exp2((x - ref) c), in FP64; with kSum32 the exponentials are the hardware's;
// with kBinned they are integers of `bits` fraction bits, also in L.hist by
// their exponents.  scan_begin() finds the threshold; with depth > 0 classes
// with an exponent down to -depth are to be listed too: if that should take
// too many places, `deep` says so.
enum { kNoSum, kSum32, kSum64, kBinned };
struct Scan {
  float m, ref, thr;
  int32_t n;
  double sum;
  double bins_low;  // exponent of the lowest bin's end
  bool deep;
};

template <int DT, int NT, bool BINS>
__device__ __forceinline__ Scan scan_begin(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, int32_t k,
                                           double c, double depth, RawBlock<DT>& raw, ListLds<NT>& L) {
  constexpr int VE = Score<DT>::kVec, NL = ListLds<NT>::kList, STEP = NT * kBlk<DT>;
  const int tid = threadIdx.x;
  raw = load_block<DT, NT>(xr, 0, C);
  float gm[kVecs], hi = -kInf, lo = kInf, least = kInf;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[VE];
    unpack<DT>(raw.v[j], f);
    gm[j] = __builtin_fmaxf(max_of(f), -kInf) + 0.0f;
    if (BINS) {
#pragma unroll
      for (int q = 0; q < VE; ++q) least = __builtin_fminf(least, f[q] == -kInf ? kInf : f[q]);
    }
    hi = __builtin_fmaxf(hi, gm[j]);
    lo = __builtin_fminf(lo, gm[j]);
  }
  hi = wave_max(hi);
  lo = wave_min(lo);
  if ((tid & 63) == 0) {
    L.shf[0][tid >> 6] = hi;
    L.shf[1][tid >> 6] = lo;
  }
  if (tid == 0) {
    L.n_list = 0u;
    L.n_vec = 0u;
  }
  if (BINS) {
    least = wave_min(least);
    if ((tid & 63) == 0) L.shd[tid >> 6] = (double)least;
  }
  __syncthreads();
  hi = across_waves<NT / 64>(L.shf[0], [](float a, float b) { return __builtin_fmaxf(a, b); });
  lo = across_waves<NT / 64>(L.shf[1], [](float a, float b) { return __builtin_fminf(a, b); });
  // of a row of one block at least k; of a longer one its share of 2 k + 64
  // (k = 64 of 8 blocks: 24 of the first, so 192 +- 39 of the row)
  const int32_t r = C <= STEP ? k : (int32_t)((int64_t)(2 * k + 64) * STEP / C) + 1;
  Scan s;
  s.deep = false;
  float thr = uniform(of_key(group_threshold<NT>(gm, hi, lo, r, L)));
  if (depth > 0.0) {
    // (a little lower: roundings take no class off that belongs)
    const float cut = (float)((double)hi - depth / c * (1.0 + 1e-6)) - 1e-6f * __builtin_fabsf(hi);
    int32_t n = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[VE];
      unpack<DT>(raw.v[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) n += f[q] >= cut ? 1 : 0;
    }
    n = block_sum<NT>(n, L.sh32);
    const int64_t all = C <= STEP ? n : (int64_t)n * C / STEP;
    s.deep = all > NL / 3 * 2;
    if (!s.deep) thr = uniform(__builtin_fminf(thr, cut));
  }
  s.thr = thr;
  s.ref = hi > -kInf ? uniform(hi) : 0.0f;  // (a masked block: the rest is listed or binned)
  // the bins end a little below the block's lowest class (what is lower shares
  // the last one), or where masses end
  s.bins_low = -1100.0;
  if (BINS) {
    const double l = across_waves<NT / 64>(L.shd, [](double a, double b) { return a < b ? a : b; });
    s.bins_low = uniform((l - (double)hi) * c * 1.125 - 0.01);
    __syncthreads();
  }
  return s;
}

// The pass itself; raw: the first block.
template <int DT, int NT, int SUM, typename Lds>
__device__ __forceinline__ void scan_blocks(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, double c,
                                            int bits, RawBlock<DT> raw, Lds& L, Scan& s) {
  constexpr int VE = Score<DT>::kVec, NL = ListLds<NT>::kList, STEP = NT * kBlk<DT>;
  const int tid = threadIdx.x;
  if constexpr (SUM == kBinned) {
    for (int b = tid; b < Lds::kBins; b += NT) L.hist[b] = 0ull;
    __syncthreads();
  }
  const float thr = s.thr;
  const float cf = uniform(exponent_scale(c));
  const double ref = (double)s.ref, cd = uniform(c);
  float m = -kInf;
  double sum = 0.0;
  uint64_t sum_q = 0;
  const double magic = __builtin_ldexp(1.0, 52 - bits), low = -(double)(bits + 2);
  const uint64_t zero = uint64_t(__double_as_longlong(magic));
  // the elements that reach the threshold into the list, leaving -inf
  auto list_vector = [&](float (&f)[VE], int32_t c0) {
#pragma unroll
    for (int q = 0; q < VE; ++q) {
      if (f[q] >= thr) {
        const uint32_t at = atomicAdd(&L.n_list, 1u);
        if (at < (uint32_t)NL) L.list[at] = place_of(f[q] + 0.0f, c0 + q);
        f[q] = -kInf;
      }
    }
  };
  auto add = [&](float (&f)[VE]) {
    if (SUM == kSum32) {
#pragma unroll
      // (NaN, as -inf, has no mass)
      for (int q = 0; q < VE; ++q) f[q] = exp2_32(__builtin_fmaxf((f[q] - s.ref) * cf, -200.0f));
      sum += (double)sum_of(f);
    }
    if (SUM == kSum64) {
      // four at a time: enough to cover an addition's latency, in few registers
#pragma unroll
      for (int h = 0; h < VE; h += 4) {
#pragma unroll
        for (int q = h; q < h + 4; ++q)
          sum += exp2_64_near(__builtin_fmax(((double)f[q] - ref) * cd, -1000.0));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (SUM == kBinned) {
      const double scale = (double)Lds::kBins / (s.bins_low > low ? s.bins_low : low);
#pragma unroll
      for (int h = 0; h < VE; h += 4) {
#pragma unroll
        for (int q = h; q < h + 4; ++q) {
          const double y = __builtin_fmax(((double)f[q] - ref) * cd, low);
          const uint64_t w = uint64_t(__double_as_longlong(exp2_64_near(y) + magic)) - zero;
          sum_q += w;
          if (w != 0)
            atomicAdd(reinterpret_cast<unsigned long long*>(&L.hist[bin_of_exponent<Lds::kBins>(y, scale)]),
                      (unsigned long long)w);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  for (int32_t base = 0;;) {
    // the next block is on its way while this one is worked on
    RawBlock<DT> next;
    const bool more = base + STEP < C;
    if (more) next = load_block<DT, NT>(xr, base + STEP, C);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[VE];
      unpack<DT>(raw.v[j], f);
      const float vm = max_of(f);
      m = __builtin_fmaxf(m, vm);
      if (vm >= thr) {
        // a wave meets such a vector every other time: what it does here has to
        // be little, so its likely elements wait (with up to 256 threads a row
        // the LDS for that would cost workgroups).  The others are added here and
        // not by the thread that lists them, which the atomic chooses: the order
        // of the additions is always the same.
        const int32_t c0 = base + (j * NT + tid) * VE;
        if constexpr (NT > 256) {
          const uint32_t at = atomicAdd(&L.n_vec, 1u);
          if (at < (uint32_t)Lds::kVectors) {
            __builtin_memcpy(&L.vec[4 * at], &raw.v[j], 16);
            L.vec_at[at] = c0;
          }
#pragma unroll
          for (int q = 0; q < VE; ++q) f[q] = f[q] >= thr ? -kInf : f[q];
        } else {
          list_vector(f, c0);
        }
      }
      add(f);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!more) break;
    base += STEP;
    raw = next;
  }
  if constexpr (NT > 256) {
    __syncthreads();
    const int32_t n_vec = (int32_t)L.n_vec;
    if (n_vec > Lds::kVectors) {
      if (tid == 0) L.n_list = NL + 1;
    } else {
      for (int32_t v = tid; v < n_vec; v += NT) {
        Vec16<DT> e;
        __builtin_memcpy(&e, &L.vec[4 * v], 16);
        float f[VE];
        unpack<DT>(e, f);
        list_vector(f, L.vec_at[v]);
      }
    }
  }
  m = wave_max(m);
  if ((tid & 63) == 0) L.shf[0][tid >> 6] = m;
  if (SUM == kBinned) {
    sum_q = wave_sum(sum_q);
    if ((tid & 63) == 0) L.shu[tid >> 6] = sum_q;
  } else if (SUM != kNoSum) {
    sum = wave_sum(sum);
    if ((tid & 63) == 0) L.shd[tid >> 6] = sum;
  }
  __syncthreads();
  s.m = uniform(across_waves<NT / 64>(L.shf[0], [](float a, float b) { return __builtin_fmaxf(a, b); }) + 0.0f);
  if (SUM == kBinned)
    s.sum = (double)across_waves<NT / 64>(L.shu, [](uint64_t a, uint64_t b) { return a + b; });
  else
    s.sum = SUM == kNoSum ? 0.0 : across_waves<NT / 64>(L.shd, [](double a, double b) { return a + b; });
  s.n = (int32_t)L.n_list;
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

// Value bins between vlo and vhi, bin 0 first in the order.
struct Bins {
  double hi, scale;
  float vlo, vhi;
  bool flat, open;  // one value; +inf in a bin of its own
  template <int NB>
  __device__ __forceinline__ void set(float lo, float h) {
    vlo = lo;
    vhi = h;
    flat = lo == h;
    open = h == kInf && !flat;
    hi = (double)h;
    scale = (double)NB / ((double)h - (double)lo);
  }
  template <int NB>
  __device__ __forceinline__ int32_t at(double below) const {  // below: hi - v
    const int32_t b = (int32_t)(below * scale);
    return b < NB - 1 ? b : NB - 1;
  }
  template <int NB>
  __device__ __forceinline__ int32_t of(float v) const {
    if (flat) return 0;
    if (open) return v == kInf ? 0 : 1;
    return at<NB>(hi - (double)v);
  }
};

// The bins of a row's masses: scores below them have mass 0.
template <int NB>
__device__ __forceinline__ void mass_bins(const Mass& mass, float m, Bins* b) {
  const float floor_v = (float)(mass.m + mass.low / mass.c);
  b->set<NB>(mass.inf ? kInf : __builtin_fminf(floor_v > -kInf ? floor_v : -3.4e38f, m), m);
}

// have: L.hist holds the masses in the bins of mass_bins() (cleared when it no
// longer does), and `total` is the kept ones' sum; otherwise the first level
// finds both.
template <int DT, int NT, int TARGET>
__device__ Found locate(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, uint64_t keep,
                        uint64_t count, double frac, float m, const Mass& mass, SelLds<NT>& L, bool& have,
                        uint64_t total) {
  constexpr int VE = Score<DT>::kVec, NB = SelLds<NT>::kBins, NL = ListLds<NT>::kList;
  constexpr bool kCount = TARGET == kTargetCount;
  const int tid = threadIdx.x;
  Bins bins;
  if (kCount)
    bins.set<NB>(score_of(keep), m);
  else
    mass_bins<NB>(mass, m, &bins);
  uint64_t above = 0, target = count;
  bool first = true;
  Found out;
  for (;;) {
    if (!have)
      for (int b = tid; b < NB; b += NT) L.hist[b] = 0ull;
    if (tid == 0) {
      L.n_list = 0u;
      L.kmin = 0xffffffffu;
      L.kmax = 0u;
    }
    __syncthreads();
    if (bins.flat) {
      const float vhi = bins.vhi;
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
        if (target < 1) target = 1;
        if (target > total) target = total;
      }
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
    if (!have) {
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const float v = canon(f[q]);
          if (c0 + q < C && v >= bins.vlo && v <= bins.vhi && v > -kInf && place_of(v, c0 + q) >= keep)
            atomicAdd(reinterpret_cast<unsigned long long*>(&L.hist[bins.of<NB>(v)]),
                      kCount ? 1ull : (unsigned long long)mass.q(v));
        }
      }
      __syncthreads();
    }
    // the bin in which the running sum reaches the target
    constexpr int PB = NB / NT;
    uint64_t mine = 0;
#pragma unroll
    for (int b = 0; b < PB; ++b) mine += L.hist[tid * PB + b];
    uint64_t sum;
    uint64_t run = block_scan_u64<NT>(mine, &sum, L.shu);
    if (first) {
      if (!have) total = sum;
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
    // an interval that holds the bin's scores (half a bin more on both sides),
    // so that the exact test is made for few
    float from = bins.vlo, to = bins.vhi;
    if (!bins.open) {
      to = __builtin_fminf(to, (float)(bins.hi - ((double)bin - 0.5) / bins.scale));
      if (bin < NB - 1) from = __builtin_fmaxf(from, (float)(bins.hi - ((double)bin + 1.5) / bins.scale));
    }
    from = uniform(__builtin_fmaxf(from, score_of(keep)));
    to = uniform(to);
    each_block<DT, NT>(xr, C, [&](const RawBlock<DT>& raw, int32_t base) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float f[VE];
        unpack<DT>(raw.v[j], f);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          // (NaN fails; past the row's end is -inf, as a masked class)
          if (f[q] >= from && f[q] <= to) {
            const float v = f[q] + 0.0f;
            const uint64_t p = place_of(v, base + (j * NT + tid) * VE + q);
            if (bins.of<NB>(v) == bin && p >= keep) {
              const uint32_t at = atomicAdd(&L.n_list, 1u);
              if (at < (uint32_t)NL) L.list[at] = p;
              atomicMin(&L.kmin, key_of(v));
              atomicMax(&L.kmax, key_of(v));
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    __syncthreads();
    const int32_t n = (int32_t)L.n_list;
    if (n <= NL) {
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
    bins.set<NB>(of_key(kmin), of_key(kmax));
    have = false;
  }
}

// The list of all places >= keep into L.sorted, in order; returns how many
// there are (ranked only when they fit).
template <int DT, int NT>
__device__ int32_t list_from(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, uint64_t keep,
                             ListLds<NT>& L) {
  constexpr int VE = Score<DT>::kVec, NL = ListLds<NT>::kList;
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
        if (at < (uint32_t)NL) L.list[at] = p;
      }
    }
  }
  __syncthreads();
  const int32_t n = (int32_t)L.n_list;
  if (n <= NL) rank_list<NT>(L, n);
  return n;
}

// Rows that the one-read kernel could not finish carry kUnfinished where their
// first class belongs; a second kernel finds and finishes them.  (Its code in
// the first one would cost that registers, and every row is done faster by a
// kernel that has them.)  Each workgroup looks after the rows blockIdx.x +
// j gridDim.x, a thread a row at a time, and lists the unfinished in LDS.
//
// Such rows are slow, and there are calls that have no others: a top-k above
// GBDT_MAX_LISTED, and in rows of 513 to 2,048 classes a k that their at most 256
// vectors cannot separate (above C / 8 in 16 bits; in f32 above C / 4 up to 1,024
// classes, C / 8 - 32 in longer rows), so that all classes are listed: records of
// 50,000 x 1,000 bf16 with k = 200 take 17.5 ms.
constexpr int32_t kUnfinished = -2;
constexpr int64_t kRestGrid = 256;

template <int NT, typename Work>
__device__ __forceinline__ void each_unfinished(const int32_t* first, int64_t stride, int64_t n, Work work) {
  __shared__ int32_t todo[NT];
  __shared__ uint32_t n_todo;
  for (int64_t j0 = 0; blockIdx.x + j0 * gridDim.x < n; j0 += NT) {
    if (threadIdx.x == 0) n_todo = 0u;
    __syncthreads();
    const int64_t i = blockIdx.x + (j0 + threadIdx.x) * gridDim.x;
    if (i < n && first[i * stride] == kUnfinished) todo[atomicAdd(&n_todo, 1u)] = (int32_t)threadIdx.x;
    __syncthreads();
    const int32_t left = (int32_t)n_todo;
    for (int32_t t = 0; t < left; ++t) {
      work(blockIdx.x + (j0 + todo[t]) * gridDim.x);
      __syncthreads();
    }
    __syncthreads();
  }
}

// The largest score of the row.
template <int DT, int NT>
__device__ float row_max(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, ListLds<NT>& L) {
  float m = -kInf;
  each_block<DT, NT>(xr, C, [&](const RawBlock<DT>& raw, int32_t) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[Score<DT>::kVec];
      unpack<DT>(raw.v[j], f);
      m = __builtin_fmaxf(m, max_of(f));
    }
  });
  return block_max<NT>(m, L.shf[0]) + 0.0f;
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
  int64_t row0;  // of this launch
};

// One workgroup per row.  A long row's time is its read (2,048 x 131,072 bf16:
// 118 us, 4.6 TB/s; with each likely class listed on the spot 131); the threshold,
// the ranking and the workgroup's reductions are 5 to 8 us a row, which the
// CU's other two workgroups cover in part.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, kHotWaves<NT>) k_top_block(const TopArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int NL = ListLds<NT>::kList;
  __shared__ ListLds<NT> L;
  const int tid = threadIdx.x;
  const int32_t C = a.C, k = a.k;
  const int64_t i = a.row0 + blockIdx.x;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  RawBlock<DT> raw;
  Scan sc = scan_begin<DT, NT, false>(xr, C, k, a.c, 0.0, raw, L);
  scan_blocks<DT, NT, kSum32>(xr, C, a.c, 0, raw, L, sc);
  const float m = sc.m;
  const int32_t n = sc.n, got = n < k ? n : k;
  if (m > -kInf && !(n <= NL && (n >= k || C <= NT * kBlk<DT>))) {
    if (tid == 0) a.classes[i * k] = kUnfinished;
    return;
  }
  if (n > 0) rank_list<NT>(L, n);
  if (a.rest != nullptr) {
    const bool inf = m == kInf;
    const float cf = exponent_scale(a.c);
    double in = 0.0, out = 0.0;
    for (int32_t j = tid; j < n; j += NT) {
      const float v = score_of(L.sorted[j]);
      const double w = (double)(inf ? (v == kInf ? 1.0f : 0.0f) : exp2_32((v - m) * cf));
      if (j < got) in += w; else out += w;
    }
    if (tid == 0 && !inf && sc.sum > 0.0) out += sc.sum * exp2_64(((double)sc.ref - (double)m) * a.c);
    in = block_sum<NT>(in, L.shd);
    out = block_sum<NT>(out, L.shd);
    if (tid == 0) a.rest[i] = n > 0 ? (float)(out / (in + out)) : 0.0f;
  }
  for (int32_t j = tid; j < k; j += NT) {
    a.values[i * k + j] = j < got ? score_of(L.sorted[j]) : -kInf;
    a.classes[i * k + j] = j < got ? class_of(L.sorted[j]) : -1;
  }
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT, 2) k_top_rest(const TopArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec;
  __shared__ SelLds<NT> L;
  const int tid = threadIdx.x;
  const int32_t C = a.C, k = a.k;
  each_unfinished<NT>(a.classes, k, a.n, [&](int64_t i) {
    const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
    const float m = row_max<DT, NT>(xr, C, L);
    // from the exact k-th place on, exactly k (or all above -inf) are listed
    uint64_t last = first_place(kKeyNegInf + 1u);
    bool have = false;
    last = locate<DT, NT, kTargetCount>(xr, C, last, (uint64_t)k, 0.0, m, Mass(), L, have, 0).place;
    const int32_t got = list_from<DT, NT>(xr, C, last, L);
    if (a.rest != nullptr) {
      const bool inf = m == kInf;
      const float cf = exponent_scale(a.c);
      double in = 0.0, out = 0.0;
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const float v = canon(f[q]);
          const double w = (double)(inf ? (v == kInf ? 1.0f : 0.0f) : exp2_32((v - m) * cf));
          if (c0 + q < C) {
            if (place_of(v, c0 + q) >= last) in += w; else out += w;
          }
        }
      }
      in = block_sum<NT>(in, L.shd);
      out = block_sum<NT>(out, L.shd);
      if (tid == 0) a.rest[i] = (float)(out / (in + out));
    }
    for (int32_t j = tid; j < k; j += NT) {
      a.values[i * k + j] = j < got ? score_of(L.sorted[j]) : -kInf;
      a.classes[i * k + j] = j < got ? class_of(L.sorted[j]) : -1;
    }
  });
}

// Rows of at most this many classes: one thread each (300,000 rows of 100
// classes: records 455 us, 720 with a wave a row; draws 640 and 1,134).
constexpr int kSortedClasses = 128;

// A row of at most CMAX classes in one thread: its places sorted in registers
// (Batcher's odd-even merge network, largest first).  A place is a positive
// FP64 number here, key and class in its last 56 bits: its order is the
// place's, and a comparator is two instructions, max and min.
template <int CMAX>
__device__ __forceinline__ double short_place(float x, int32_t c) {
  return __longlong_as_double(int64_t(uint64_t(1) << 62 | uint64_t(key_of(x)) << 24 | uint64_t(CMAX - 1 - c)));
}
__device__ __forceinline__ float short_score(double p) {
  return of_key(uint32_t(uint64_t(__double_as_longlong(p)) >> 24));
}
template <int CMAX>
__device__ __forceinline__ int32_t short_class(double p) {
  return CMAX - 1 - (__double2loint(p) & (CMAX - 1));
}
template <int CMAX>
__device__ __forceinline__ void sort_row(const float* __restrict__ x, int32_t C, double (&p)[CMAX]) {
#pragma unroll
  for (int c = 0; c < CMAX; ++c) p[c] = short_place<CMAX>(c < C ? canon(x[c]) : -kInf, c);
#pragma unroll
  for (int s = 1; s < CMAX; s <<= 1) {
#pragma unroll
    for (int d = s; d >= 1; d >>= 1) {
#pragma unroll
      for (int i = 0; i + d < CMAX; ++i) {
        // (i from d mod s on, in runs of d, both ends in one half of 2 s)
        if (i >= d % s && (i - d % s) / d % 2 == 0 && i / (2 * s) == (i + d) / (2 * s)) {
          const double u = __builtin_fmax(p[i], p[i + d]), v = __builtin_fmin(p[i], p[i + d]);
          p[i] = u;
          p[i + d] = v;
        }
      }
    }
  }
}

// The rows of a workgroup into LDS, in rows of C | 1 words.
template <int DT, int R, int CMAX>
__device__ __forceinline__ void stage_scores(const void* x, int64_t i0, int32_t rows, int32_t C, int64_t ld,
                                             const RowDiv& by_c, float* lds) {
  const auto* __restrict__ xg = static_cast<const typename Score<DT>::Elem*>(x) + i0 * ld;
  Staged<R, CMAX, float> xs;
  xs.load(
      rows, C, ld == C, by_c, [&](int32_t e) { return Score<DT>::to_f32(xg[(uint32_t)e]); },
      [&](int32_t row, int32_t c) { return Score<DT>::to_f32(xg[row * ld + c]); });
  xs.put(rows, C, by_c, lds);
}

// One thread per row, R rows a workgroup (581,012 rows of 7 f32, k = 3: 11 us,
// 2.9 TB/s; without the staging through LDS 27 us).
template <int DT, int R, int CMAX>
__global__ void __launch_bounds__(R) k_top_rows(const TopArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x;
  const int64_t i0 = int64_t(blockIdx.x) * R, i = i0 + tid;
  const int32_t rows = (int32_t)(a.n - i0 < R ? a.n - i0 : R);
  const int32_t C = a.C, k = a.k, P = C | 1, PK = k | 1;
  const RowDiv by_c(C), by_k(k);
  float* __restrict__ values = lds + R * P;
  int32_t* __restrict__ classes = reinterpret_cast<int32_t*>(values + R * PK);
  stage_scores<DT, R, CMAX>(a.x, i0, rows, C, a.ld, by_c, lds);
  __syncthreads();
  if (tid < rows) {
    double p[CMAX];
    sort_row<CMAX>(lds + tid * P, C, p);
    const float m = short_score(p[0]);
    if (a.rest != nullptr) {
      const bool inf = m == kInf;
      const float cf = exponent_scale(a.c);
      double in = 0.0, out = 0.0;
#pragma unroll
      for (int c = 0; c < CMAX; ++c) {
        if (c < C) {
          const float v = short_score(p[c]);
          const double e = (double)(inf ? (v == kInf ? 1.0f : 0.0f) : exp2_32((v - m) * cf));
          if (c < k) in += e; else out += e;
        }
      }
      a.rest[i] = m > -kInf ? (float)(out * rcp_64(in + out)) : 0.0f;
    }
#pragma unroll
    for (int c = 0; c < CMAX; ++c) {
      if (c < k) {
        const float v = short_score(p[c]);
        values[tid * PK + c] = v;
        classes[tid * PK + c] = v > -kInf ? short_class<CMAX>(p[c]) : -1;
      }
    }
  }
  __syncthreads();
  float* __restrict__ vg = a.values + i0 * k;
  int32_t* __restrict__ cg = a.classes + i0 * k;
  unstage<R, CMAX>(
      rows, k, true, by_k, values, [&](int32_t e, float v) { vg[(uint32_t)e] = v; }, [](int32_t, int32_t, float) {});
  unstage<R, CMAX>(
      rows, k, true, by_k, classes, [&](int32_t e, int32_t c) { cg[(uint32_t)e] = c; },
      [](int32_t, int32_t, int32_t) {});
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
  int64_t row0;  // of this launch
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

// The mass of all places >= keep (m finite).
template <int DT, int NT>
__device__ uint64_t kept_sum(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, uint64_t keep,
                             const Mass& mass, ListLds<NT>& L) {
  constexpr int VE = Score<DT>::kVec;
  uint64_t sum = 0;
  for (int32_t c0 = threadIdx.x * VE; c0 < C; c0 += NT * VE) {
    float f[VE];
    load_chunk<DT>(xr, c0, C, f);
#pragma unroll
    for (int q = 0; q < VE; ++q) {
      const float v = canon(f[q]);
      if (c0 + q < C && place_of(v, c0 + q) >= keep) sum += mass.q(v);
    }
  }
  return block_sum<NT>(sum, L.shu);
}

// All masses of a row into the bins; returns their sum.
template <int DT, int NT>
__device__ uint64_t bin_masses(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, const Mass& mass,
                               const Bins& bins, SelLds<NT>& L) {
  constexpr int VE = Score<DT>::kVec, NB = SelLds<NT>::kBins;
  const int tid = threadIdx.x;
  uint64_t sum = 0;
  for (int b = tid; b < NB; b += NT) L.hist[b] = 0ull;
  __syncthreads();
  const uint64_t zero = mass.raw_zero();
  each_block<DT, NT>(xr, C, [&](const RawBlock<DT>& raw, int32_t) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[VE];
      unpack<DT>(raw.v[j], f);
#pragma unroll
      for (int h = 0; h < VE; h += 4) {
#pragma unroll
        for (int q = h; q < h + 4; ++q) {
          const double d = (double)f[q] - mass.m;
          const uint64_t w = mass.raw_at(d) - zero;
          sum += w;
          if (w != 0)
            atomicAdd(reinterpret_cast<unsigned long long*>(&L.hist[bins.at<NB>(-d)]), (unsigned long long)w);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  });
  return block_sum<NT>(sum, L.shu);
}

__device__ __forceinline__ void write_draw(const SampleArgs& a, int64_t i, const RowParams& r, float m, uint64_t place,
                                           uint64_t total, int bits) {
  a.out[i] = class_of(place);
  if (a.logp != nullptr) {
    const double d = m == kInf || r.T == 0.0 ? 0.0 : ((double)score_of(place) - (double)m) / r.T;
    a.logp[i] = (float)(d - log_64(__builtin_ldexp((double)total, -bits)));
  }
}

// The bin in which the running sum reaches the target (1 <= target <= their
// sum), or the given bin, and the sum before it: into L.found[0..1]; the target
// (at most the sum) into L.found[2].
template <int NT>
__device__ __forceinline__ void find_bin(uint64_t target, int32_t given, SelLds<NT>& L) {
  constexpr int PB = SelLds<NT>::kBins / NT;
  uint64_t mine = 0, all;
#pragma unroll
  for (int b = 0; b < PB; ++b) mine += L.hist[threadIdx.x * PB + b];
  uint64_t run = block_scan_u64<NT>(mine, &all, L.shu);
  target = target < all ? target : all;
#pragma unroll
  for (int b = 0; b < PB; ++b) {
    const int32_t at = (int32_t)threadIdx.x * PB + b;
    const uint64_t h = L.hist[at];
    if (given >= 0 ? at == given : run < target && run + h >= target) {
      L.found[0] = uint64_t(at);
      L.found[1] = run;
      L.found[2] = target;
    }
    run += h;
  }
  __syncthreads();
}

// Of the classes below the list, in the order: the place where their running
// sum reaches the target (into L.found[0]) and the sum up to it (L.found[1]); or
// with by_value the sum of those with a score >= least.  False if the bin has
// more members than the list holds.
template <int DT, int NT>
__device__ __forceinline__ bool search_bins(const typename Score<DT>::Elem* __restrict__ xr, int32_t C,
                                            uint64_t target, bool by_value, float least, const Scan& sc, double c,
                                            int bits, SelLds<NT>& L) {
  constexpr int VE = Score<DT>::kVec, NL = ListLds<NT>::kList, NB = SelLds<NT>::kBins;
  const int tid = threadIdx.x;
  const double low = -(double)(bits + 2), ref = (double)sc.ref;
  const double scale = (double)NB / (sc.bins_low > low ? sc.bins_low : low);
  const double magic = __builtin_ldexp(1.0, 52 - bits);
  const uint64_t zero = uint64_t(__double_as_longlong(magic));
  int32_t given = -1;
  if (by_value) given = bin_of_exponent<NB>(__builtin_fmax(((double)least - ref) * c, low), scale);
  find_bin<NT>(target, given, L);
  const int32_t bin = (int32_t)L.found[0];
  const uint64_t above = L.found[1];
  target = L.found[2];
  if (tid == 0) L.n_list = 0u;
  __syncthreads();
  // The bin's scores lie within a bin's width of its middle (the last one's
  // anywhere below); where a vector has one, the exact test.
  const float mid = uniform((float)(ref + ((double)bin + 0.5) / scale / c));
  const float wide = bin == NB - 1 ? kInf : uniform((float)(-1.0 / scale / c) + 1e-6f * __builtin_fabsf(mid));
  each_block<DT, NT>(xr, C, [&](const RawBlock<DT>& raw, int32_t base) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[VE], d[VE];
      unpack<DT>(raw.v[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) d[q] = -__builtin_fabsf(f[q] - mid);
      if (max_of(d) >= -wide) {
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const double y = ((double)f[q] - ref) * c;
          if (f[q] < sc.thr && y >= low && bin_of_exponent<NB>(y, scale) == bin) {
            const uint32_t at = atomicAdd(&L.n_list, 1u);
            if (at < (uint32_t)NL) L.list[at] = place_of(f[q] + 0.0f, base + (j * NT + tid) * VE + q);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  });
  __syncthreads();
  const int32_t n = (int32_t)L.n_list;
  if (n > NL) return false;
  rank_list<NT>(L, n);
  // running sums in the order, by one wave
  if (tid < 64) {
    uint64_t carry = above;
    if (tid == 0 && by_value) L.found[1] = above;
    for (int32_t b = 0; b < n; b += 64) {
      const int32_t at = b + tid;
      const float v = at < n ? score_of(L.sorted[at]) : -kInf;
      const double y = at < n ? ((double)v - ref) * c : low;
      const uint64_t w = uint64_t(__double_as_longlong(exp2_64_near(y) + magic)) - zero;
      uint64_t x = w;
      for (int off = 1; off < 64; off <<= 1) {
        const uint64_t up = __shfl_up(x, off, 64);
        if (tid >= off) x += up;
      }
      x += carry;
      if (by_value) {
        const uint64_t in = __ballot(v >= least);
        if (in != 0 && tid == 63 - __builtin_clzll(in)) L.found[1] = x;
      } else if (at < n && x >= target && x - w < target) {
        L.found[0] = L.sorted[at];
        L.found[1] = x;
      }
      carry = __shfl(x, 63, 64);
    }
  }
  __syncthreads();
  return true;
}

// The first place of the scores with e >= min_p (x >= m + log2(min_p) / c).
__device__ __forceinline__ uint64_t min_p_place(double min_p, const Mass& mass) {
  const double v = mass.m + log2(min_p) / mass.c;
  const float f = (float)v + 0.0f;
  const uint64_t cut = first_place(key_of(f) + ((double)f < v ? 1u : 0u));
  const uint64_t top = first_place(key_of((float)mass.m));
  return cut < top ? cut : top;
}

// A row is drawn from its first top-k classes (FEW); or from its likely classes
// and the others' sum, where a min-p cuts not far below the maximum; or with
// the others' masses in bins, whose atomics make the pass half as long again.
template <int DT, int NT, bool FEW>
__device__ __forceinline__ bool sample_row(const SampleArgs& a, int64_t i, const RowParams& r, SelLds<NT>& L) {
  using Elem = typename Score<DT>::Elem;
  constexpr int NL = ListLds<NT>::kList, PL = NL / NT;
  const int tid = threadIdx.x;
  const int32_t C = a.C;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  const double c = r.T > 0.0 ? kLog2e / r.T : 0.0;
  const int bits = mass_bits(C);
  RawBlock<DT> raw;
  const double depth = !FEW && r.min_p > 0.0 ? -log_64(r.min_p) * kLog2e : 0.0;
  Scan sc = scan_begin<DT, NT, !FEW>(xr, C, FEW ? r.top_k : 32, c, depth, raw, L);
  const bool binned = !FEW && (r.min_p == 0.0 || sc.deep);
  if (FEW)
    scan_blocks<DT, NT, kNoSum>(xr, C, c, bits, raw, L, sc);
  else if (binned)
    scan_blocks<DT, NT, kBinned>(xr, C, c, bits, raw, L, sc);
  else
    scan_blocks<DT, NT, kSum64>(xr, C, c, bits, raw, L, sc);
  const float m = sc.m;
  const int32_t n = sc.n, got = FEW && n > r.top_k ? r.top_k : n;
  if (!(m > -kInf)) {
    if (tid == 0) {
      a.out[i] = -1;
      if (a.logp != nullptr) a.logp[i] = -kInf;
    }
    return true;
  }
  if (n > NL || n == 0 || (FEW ? n < r.top_k && C > NT * kBlk<DT> : m == kInf)) return false;
  rank_list<NT>(L, n);
  const Mass mass = make_mass(m, c, bits);
  // running sums over the list (thread by thread PL entries), its two cuts, and
  // the draw
  uint64_t p[PL], w[PL], mine = 0;
#pragma unroll
  for (int b = 0; b < PL; ++b) {
    const int32_t at = tid * PL + b;
    p[b] = at < got ? L.sorted[at] : 0;
    w[b] = at < got ? mass.q(score_of(p[b])) : 0;
    mine += w[b];
  }
  uint64_t in_list;
  const uint64_t before = block_scan_u64<NT>(mine, &in_list, L.shu);
  // the others' sum is against another reference
  const double below = FEW ? 0.0 : binned ? sc.sum : __builtin_ldexp(sc.sum, bits);
  const double to_m = below > 0.0 ? exp2_64(((double)sc.ref - (double)m) * c) : 0.0;
  const uint64_t sum = in_list + (uint64_t)__builtin_rint(below * to_m);
  const uint64_t most = r.top_p < 1.0 ? (uint64_t)__builtin_ceil(r.top_p * (double)sum) : ~uint64_t(0);
  uint64_t run = before, upto = 0;
  int32_t kept = 0;
#pragma unroll
  for (int b = 0; b < PL; ++b) {
    const int32_t at = tid * PL + b;
    const bool keep =
        at < got && w[b] > 0 && (at == 0 || (run < most && (r.min_p == 0.0 || mass.e(score_of(p[b])) >= r.min_p)));
    run += w[b];
    // (a prefix is kept: the last one's running sum is the largest)
    if (keep) {
      upto = run;
      ++kept;
    }
  }
  kept = block_sum<NT>(kept, L.sh32);
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t y = __shfl_xor(upto, off, 64);
    upto = y > upto ? y : upto;
  }
  if ((tid & 63) == 0) L.shu[tid >> 6] = upto;
  __syncthreads();
  uint64_t W = across_waves<NT / 64>(L.shu, [](uint64_t u, uint64_t v) { return u > v ? u : v; });
  // is what is kept known: cut inside the list, or all of the row?
  // (a min-p cut that is not deep is above the threshold)
  bool known = FEW || kept < got || in_list >= most || sum == in_list || (r.min_p > 0.0 && !sc.deep);
  if (!known && r.top_p >= 1.0 && r.min_p == 0.0) {
    W = sum;
    known = true;
  }
  uint64_t last = 0;  // (below the list: the last place that is kept)
  if (binned && !known) {
    W = sum;
    if (most < sum) {
      const uint64_t target = (uint64_t)__builtin_ceil((double)(most - in_list) / to_m);
      if (!search_bins<DT, NT>(xr, C, target, false, 0.0f, sc, c, bits, L)) return false;
      last = L.found[0];
      W = in_list + (uint64_t)__builtin_rint((double)L.found[1] * to_m);
      __syncthreads();
    }
    if (r.min_p > 0.0) {
      const uint64_t cut = min_p_place(r.min_p, mass);
      if (cut > last) {
        if (!search_bins<DT, NT>(xr, C, 0, true, score_of(cut), sc, c, bits, L)) return false;
        last = cut;
        W = in_list + (uint64_t)__builtin_rint((double)L.found[1] * to_m);
        __syncthreads();
      }
    }
    known = true;
  }
  if (!known) return false;
  uint64_t over = (uint64_t)(r.u * (double)W) + 1ull;
  if (over > W) over = W;
  if (over <= in_list) {
    run = before;
#pragma unroll
    for (int b = 0; b < PL; ++b) {
      if (run < over && run + w[b] >= over) write_draw(a, i, r, m, p[b], W, bits);
      run += w[b];
    }
    return true;
  }
  if (!binned) return false;
  const uint64_t target = (uint64_t)__builtin_ceil((double)(over - in_list) / to_m);
  if (!search_bins<DT, NT>(xr, C, target, false, 0.0f, sc, c, bits, L)) return false;
  if (tid == 0) write_draw(a, i, r, m, L.found[0], W, bits);
  return true;
}

// FP64 bounds draws without top-k: 20 instructions a class, 57 us of 191 for
// 1,024 x 100,003 bf16 with top-p and min-p; the rest is the row's latencies
// (threshold, ranking, cuts: 20 us) with two workgroups a CU.  Four waves a
// SIMD: with six the pass spills (314 us).
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 4) k_sample_block(const SampleArgs a) {
  __shared__ SelLds<NT> L;
  const int64_t i = a.row0 + blockIdx.x;
  const RowParams r = row_params(a, i);
  if (!r.ok) {
    if (threadIdx.x == 0) {
      dev_error(a.err, GBDT_E_RANGE);
      a.out[i] = -1;
      if (a.logp != nullptr) a.logp[i] = -kInf;
    }
  } else if (r.top_k <= GBDT_MAX_LISTED) {
    if (sample_row<DT, NT, true>(a, i, r, L)) return;
    if (threadIdx.x == 0) a.out[i] = kUnfinished;
  } else if (r.top_k >= a.C) {
    if (sample_row<DT, NT, false>(a, i, r, L)) return;
    if (threadIdx.x == 0) a.out[i] = kUnfinished;
  } else if (threadIdx.x == 0) {
    a.out[i] = kUnfinished;
  }
}

// The rows that are left, by places: the top-k and top-p cuts, the min-p cut,
// the draw.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 2) k_sample_rest(const SampleArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int NB = SelLds<NT>::kBins;
  __shared__ SelLds<NT> L;
  const int32_t C = a.C;
  const int bits = mass_bits(C);
  each_unfinished<NT>(a.out, 1, a.n, [&](int64_t i) {
    const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
    const RowParams r = row_params(a, i);
    const float m = row_max<DT, NT>(xr, C, L);
    if (!(m > -kInf)) {
      if (threadIdx.x == 0) {
        a.out[i] = -1;
        if (a.logp != nullptr) a.logp[i] = -kInf;
      }
      return;
    }
    const Mass mass = make_mass(m, r.T > 0.0 ? kLog2e / r.T : 0.0, bits);
    uint64_t keep = first_place(kKeyNegInf + 1u), total = 0;
    bool have = false;
    if (r.top_k < C) {
      keep = locate<DT, NT, kTargetCount>(xr, C, keep, (uint64_t)r.top_k, 0.0, m, mass, L, have, 0).place;
    } else if (!mass.inf) {
      Bins bins;
      mass_bins<NB>(mass, m, &bins);
      if (!bins.flat) {
        total = bin_masses<DT, NT>(xr, C, mass, bins, L);
        have = true;
      }
    }
    if (r.T > 0.0 && r.top_p < 1.0) {
      const Found f = locate<DT, NT, kTargetFrac>(xr, C, keep, 0, r.top_p, m, mass, L, have, total);
      keep = f.place;
      total = f.upto;
    }
    bool known = true;  // total: the kept ones' sum
    if (r.T > 0.0 && r.min_p > 0.0 && !mass.inf) {
      const uint64_t cut = min_p_place(r.min_p, mass);
      if (cut > keep) {
        keep = cut;
        known = false;
      }
    }
    if (have && !known) total = kept_sum<DT, NT>(xr, C, keep, mass, L);
    uint64_t place = keep;
    if (r.T > 0.0) {
      const Found f = locate<DT, NT, kTargetOver>(xr, C, keep, 0, r.u, m, mass, L, have, total);
      place = f.place;
      total = f.total;
    } else {
      total = uint64_t(1) << bits;  // (top_k is 1: the first place has all the mass)
    }
    if (threadIdx.x == 0) write_draw(a, i, r, m, place, total, bits);
  });
}

// One thread per row of at most CMAX classes, R rows a workgroup (581,012 rows
// of 7 f32, all filters: 16 us; vector instructions, half of them FP64).
template <int DT, int R, int CMAX>
__global__ void __launch_bounds__(R, CMAX == 8 ? 6 : CMAX <= 32 ? 3 : 1) k_sample_rows(const SampleArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x;
  const int64_t i0 = int64_t(blockIdx.x) * R, i = i0 + tid;
  const int32_t rows = (int32_t)(a.n - i0 < R ? a.n - i0 : R);
  const int32_t C = a.C;
  const RowDiv by_c(C);
  stage_scores<DT, R, CMAX>(a.x, i0, rows, C, a.ld, by_c, lds);
  RowParams r;
  if (tid < rows) r = row_params(a, i);
  __syncthreads();
  if (tid >= rows) return;
  double p[CMAX];
  sort_row<CMAX>(lds + tid * (C | 1), C, p);
  const float m = short_score(p[0]);
  if (!r.ok || !(m > -kInf)) {
    if (!r.ok) dev_error(a.err, GBDT_E_RANGE);
    a.out[i] = -1;
    if (a.logp != nullptr) a.logp[i] = -kInf;
    return;
  }
  const bool inf = m == kInf;
  const double ms = (double)m, c_T = r.T > 0.0 ? kLog2e / r.T : 0.0;
  // (the first one's e is 1; longer rows have no registers for the others')
  constexpr int kHeld = CMAX <= 64 ? CMAX : 1;
  double held[kHeld], all = 1.0;
  auto weight = [&](int c) {
    const float v = short_score(p[c]);
    const double x = inf ? (v == kInf ? 1.0 : 0.0) : exp2_64(((double)v - ms) * c_T);
    return c < r.top_k && v > -kInf ? x : 0.0;
  };
#pragma unroll
  for (int c = 1; c < CMAX; ++c) {
    if (c < C) {
      const double e = weight(c);
      if (kHeld > 1) held[c % kHeld] = e;
      all += e;
    }
  }
  const double most = r.top_p < 1.0 ? r.top_p * all : kInf;
  double run = 1.0, W = 1.0;
  int32_t n_kept = 1;
#pragma unroll
  for (int c = 1; c < CMAX; ++c) {
    if (c < C) {
      const double e = kHeld > 1 ? held[c % kHeld] : weight(c);
      if (run < most && e >= r.min_p && e > 0.0) {
        W += e;
        n_kept = c + 1;
      }
      run += e;
    }
  }
  const double over = r.u * W;
  double place = p[0], ew = 1.0;
  run = 1.0;
  bool found = run > over;
#pragma unroll
  for (int c = 1; c < CMAX; ++c) {
    if (c < C) {
      const double e = kHeld > 1 ? held[c % kHeld] : weight(c);
      // (the last kept one where rounding leaves none)
      run += e;
      const bool take = !found && c < n_kept;
      place = take ? p[c] : place;
      ew = take ? e : ew;
      found = found || (take && run > over);
    }
  }
  a.out[i] = short_class<CMAX>(place);
  if (a.logp != nullptr) a.logp[i] = (float)log_64(ew * rcp_64(W));
}

template <int DT, int NT>
void launch_top_block(TopArgs a, hipStream_t s) {
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid) {
    const int64_t n = a.n - a.row0 < kMaxRowGrid ? a.n - a.row0 : kMaxRowGrid;
    diag_begin(kDiagTopScores, s);
    hipLaunchKernelGGL((k_top_block<DT, NT>), dim3((unsigned)n), dim3(NT), 0, s, a);
    diag_end(s);
  }
  // (a row of one block that fits the list is always finished)
  if (a.C <= ListLds<NT>::kList && a.C <= NT * kBlk<DT>) return;
  const dim3 rest((unsigned)(a.n < kRestGrid ? a.n : kRestGrid));
  constexpr int RT = NT < 256 ? NT : 256;
  diag_begin(kDiagTopScores, s);
  hipLaunchKernelGGL((k_top_rest<DT, RT>), rest, dim3(RT), 0, s, a);
  diag_end(s);
}
template <int DT, int R, int CMAX>
void launch_top_rows(const TopArgs& a, hipStream_t s) {
  const size_t lds = size_t(R) * 4 * ((a.C | 1) + 2 * (a.k | 1));
  diag_begin(kDiagTopScores, s);
  hipLaunchKernelGGL((k_top_rows<DT, R, CMAX>), dim3((unsigned)((a.n + R - 1) / R)), dim3(R), lds, s, a);
  diag_end(s);
}

// Threads for a row: a wave up to 2,048 classes, 256 up to 40,000 (draws of
// 2,000 x 20,000 f32: 95 us with 256, 104 with 512), then 512 (records of
// 2,048 x 131,072 bf16: 126 us with 512, 147 with 256, 209 with 1,024); at most
// a row a CU: 1,024 (records of 32 such rows: 29 us, 31 with 512; 64 draws of
// 65,536 f32: 51 and 58).
constexpr int64_t kFewRows = 256;

template <int DT>
int launch_top(const TopArgs& a, hipStream_t s) {
  if (a.C <= 8)
    launch_top_rows<DT, 256, 8>(a, s);
  else if (a.C <= 16)
    launch_top_rows<DT, 128, 16>(a, s);
  else if (a.C <= 32)
    launch_top_rows<DT, 64, 32>(a, s);
  else if (a.C <= 64)
    launch_top_rows<DT, 64, 64>(a, s);
  else if (a.C <= kSortedClasses)
    launch_top_rows<DT, 64, 128>(a, s);
  else if (a.C <= 2048)
    launch_top_block<DT, 64>(a, s);
  else if (a.C <= 40000)
    launch_top_block<DT, 256>(a, s);
  else if (a.n > kFewRows)
    launch_top_block<DT, 512>(a, s);
  else
    launch_top_block<DT, 1024>(a, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_top");
}

template <int DT, int NT>
void launch_sample_block(SampleArgs a, hipStream_t s) {
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid) {
    const int64_t n = a.n - a.row0 < kMaxRowGrid ? a.n - a.row0 : kMaxRowGrid;
    diag_begin(kDiagSample, s);
    hipLaunchKernelGGL((k_sample_block<DT, NT>), dim3((unsigned)n), dim3(NT), 0, s, a);
    diag_end(s);
  }
  const dim3 rest((unsigned)(a.n < kRestGrid ? a.n : kRestGrid));
  constexpr int RT = NT < 256 ? NT : 256;
  diag_begin(kDiagSample, s);
  hipLaunchKernelGGL((k_sample_rest<DT, RT>), rest, dim3(RT), 0, s, a);
  diag_end(s);
}
template <int DT, int R, int CMAX>
void launch_sample_rows(const SampleArgs& a, hipStream_t s) {
  const size_t lds = size_t(R) * 4 * (a.C | 1);
  diag_begin(kDiagSample, s);
  hipLaunchKernelGGL((k_sample_rows<DT, R, CMAX>), dim3((unsigned)((a.n + R - 1) / R)), dim3(R), lds, s, a);
  diag_end(s);
}

template <int DT>
int launch_sample(const SampleArgs& a, hipStream_t s) {
  if (a.C <= 8)
    launch_sample_rows<DT, 256, 8>(a, s);
  else if (a.C <= 16)
    launch_sample_rows<DT, 128, 16>(a, s);
  else if (a.C <= 32)
    launch_sample_rows<DT, 64, 32>(a, s);
  else if (a.C <= 64)
    launch_sample_rows<DT, 64, 64>(a, s);
  else if (a.C <= kSortedClasses)
    launch_sample_rows<DT, 64, 128>(a, s);
  else if (a.C <= 2048)
    launch_sample_block<DT, 64>(a, s);
  else if (a.C <= 40000)
    launch_sample_block<DT, 256>(a, s);
  else if (a.n > kFewRows)
    launch_sample_block<DT, 512>(a, s);
  else
    launch_sample_block<DT, 1024>(a, s);
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
