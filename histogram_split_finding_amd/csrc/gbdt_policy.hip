// Learning from drawn classes: the log-probability of a class of each row with
// its gradient, the clipped policy loss with a KL term, and the preference loss
// of pairs of row sequences.
//
// Of a row x with class a, at temperature T, with the other classes' largest
// score m = max_{c != a} x_c and their sum against it, o = sum_{c != a} v_c,
// v_c = exp((x_c - m) / T), which is at least 1:
//   the logarithm of the odds against a:  L = (m - x_a) / T + log o,
//   log p_a = -log(1 + e^L),   1 - p_a = 1 / (1 + e^-L),   p_c = (1 - p_a) v_c / o.
// Nothing cancels or underflows on the way: a policy that is all but certain of
// a keeps its log p_a, and its gradient, which is 1 - p_a times values of order 1,
// to the last digit.  With d the loss's slope in log p_a, and k = (1 - p_a) d / T,
//   gradient: k at a, -k v_c / o at the others.

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

// Where a launch takes the sums of its rows from: the scores, the statistics of
// an earlier call, or the parts that a first launch left (kParts writes them).
constexpr int kSums = 0, kStats = 1, kParts = 2, kJoin = 3;

struct PartSum {
  double o;
  float m;
  uint32_t pad;
};

struct LogpArgs {
  const void* x;
  int64_t n, ld;
  const int32_t* cls;
  int32_t C, n_parts, part_len, last;  // last: of range
  int32_t reverse;                     // from the last row to the first
  const int64_t* range;                // rows [range[0], range[last]) only, or NULL: all
  double c, inv_T;                     // log2(e) / T, 1 / T
  // c as c_hi + c_lo, both positive: rounding c alone would move all terms of a sum the
  // same way, by D 2^-25 (and c_lo > 0 leaves -inf what it is); and c rounded
  float c_hi, c_lo, c_near;
  const float *old_logp, *ref_logp, *adv, *weight;
  double low, high, kl;  // borders of the ratio
  double log_low, log_high;
  float *loss, *logp, *dlogp;
  float* stats;
  void* grad;
  int64_t ldg;
  int32_t* err;
  PartSum* parts;     // [n][n_parts]
  uint32_t* arrived;  // a byte a row: its parts that are done, zero between calls
  int64_t row0;       // of this launch
};

// exp(d / T) as a term of a sum, and as a factor of a gradient.  In FP32 by choice (each
// off by some 3 D 2^-24, the sums of them are FP64): FP64 ones bounded all rows of 33 to
// 2,000 classes (sums of 262,144 x 256 bf16: 62 us, now 33, floor 24).  What they could
// decide wrongly is taken again in FP64, see next_to_border.
__device__ __forceinline__ float sum_term(const LogpArgs& a, float d) {
  return exp2_32(__builtin_fmaf(d, a.c_hi, d * a.c_lo));
}
__device__ __forceinline__ float grad_term(const LogpArgs& a, float d) { return exp2_32(d * a.c_near); }

// The rows of the call, and one of them.
struct Span {
  int64_t lo, hi;
};
__device__ __forceinline__ Span span_of(const int64_t* __restrict__ offsets, int32_t last, int64_t n) {
  int64_t lo = offsets[0], hi = offsets[last];
  lo = lo < 0 ? 0 : lo > n ? n : lo;
  hi = hi < lo ? lo : hi > n ? n : hi;
  return {lo, hi};
}
__device__ __forceinline__ Span row_span(const LogpArgs& a) {
  if (a.range == nullptr) return {0, a.n};
  return span_of(a.range, a.last, a.n);
}

__device__ __forceinline__ int32_t row_class(const LogpArgs& a, int64_t i, bool report) {
  const int32_t k = a.cls[i];
  if (k < a.C) return k < 0 ? -1 : k;
  if (report) dev_error(a.err, GBDT_E_RANGE);
  return -1;
}

// e^y for any y (overflow: inf; NaN stays).
__device__ __forceinline__ double exp_64(double y) {
  const double z = y * kLog2e;
  return z > 1023.0 ? __builtin_inf() : exp2_64(z);
}

// log(1 + e) for 0 <= e <= 1.
__device__ __forceinline__ double log1p_64(double e) { return e < 0x1p-20 ? e - 0.5 * e * e : log_64(1.0 + e); }

// A row's end: what its sums say about its class.  t = e^L, the odds against it, is
// o e^d with d = (m - x_a) / T: one exponential and one logarithm.  d is cut where t
// would overflow; there log(1 + t) is log o + d to the last digit.
struct RowEnd {
  bool live;             // the row counts
  double logp, against;  // log p_a, 1 - p_a
};
__device__ __forceinline__ RowEnd row_end(double inv_T, bool named, double m, double o, double xa) {
  constexpr double kMostD = 690.0;
  RowEnd r;
  r.live = named && !(o == 0.0 && xa == -__builtin_inf());
  const double d = (m - xa) * inv_T;
  const double over = d > kMostD ? d - kMostD : 0.0;
  double t = o * exp2_64((d > kMostD ? kMostD : d) * kLog2e);
  if (!(xa < __builtin_inf())) t = __builtin_nan("");
  r.against = t * rcp_64(1.0 + t);
  r.logp = -((t < 0x1p-20 ? t - 0.5 * t * t : log_64(1.0 + t)) + over);
  return r;
}

// The clipped policy loss of a row and its slope in logp.  ratio and A: NaN stays,
// A = 0 leaves nothing whatever the ratio.  q = e^y - y - 1, by its series where
// the terms cancel.
struct PolicyRow {
  double loss, slope;
};
__device__ __forceinline__ PolicyRow policy_row(const LogpArgs& a, double logp, float old_logp, float ref_logp,
                                                float advantage) {
  const double A = advantage, ratio = exp_64(logp - (double)old_logp);
  const double by = A == 0.0 ? 0.0 : ratio * A;
  const double kept = ratio < a.low ? a.low : (ratio > a.high ? a.high : ratio);
  const double cut = A == 0.0 ? 0.0 : kept * A;
  PolicyRow r;
  r.loss = -(by < cut || by != by ? by : cut);
  const bool clipped = (A > 0.0 && ratio > a.high) || (A < 0.0 && ratio < a.low);
  r.slope = clipped ? 0.0 : -by;
  if (a.ref_logp != nullptr) {
    const double y = (double)ref_logp - logp;
    double q, em1;
    if (__builtin_fabs(y) < 0x1p-5) {
      double p = __builtin_fma(y, 1.0 / 40320.0, 1.0 / 5040.0);
      p = __builtin_fma(y, p, 1.0 / 720.0);
      p = __builtin_fma(y, p, 1.0 / 120.0);
      p = __builtin_fma(y, p, 1.0 / 24.0);
      p = __builtin_fma(y, p, 1.0 / 6.0);
      q = y * y * __builtin_fma(y, p, 0.5);
      em1 = y + q;
    } else {
      em1 = exp_64(y) - 1.0;
      q = y == __builtin_inf() ? y : em1 - y;
    }
    r.loss += a.kl * q;
    r.slope -= a.kl * em1;
  }
  return r;
}

struct RowIn {
  float old_logp, ref_logp, adv, weight, dlogp;
};
template <int FROM>
__device__ __forceinline__ RowIn row_in(const LogpArgs& a, int64_t i) {
  RowIn r = {0.0f, 0.0f, 0.0f, 1.0f, 0.0f};
  if (FROM == kStats) {
    r.dlogp = a.dlogp[i];
  } else if (a.adv != nullptr) {
    r.old_logp = a.old_logp[i];
    r.adv = a.adv[i];
    if (a.ref_logp != nullptr) r.ref_logp = a.ref_logp[i];
    if (a.weight != nullptr) r.weight = a.weight[i];
  }
  return r;
}

// Whether a row's ratio is so near to a border of the clip that FP32 exponentials
// (off by at most (3 D + 6) 2^-24 in logp, D = |x - m| / T at most 40 where it matters:
// 7.5e-6) could take it to the other side: such a row's sum is taken again in FP64.
__device__ __forceinline__ bool next_to_border(const LogpArgs& a, const RowEnd& e, const RowIn& in) {
  const double y = e.logp - (double)in.old_logp;
  return a.adv != nullptr && e.live && in.adv != 0.0f &&
         (__builtin_fabs(y - a.log_low) < 0x1p-16 || __builtin_fabs(y - a.log_high) < 0x1p-16);
}

// Writes what a row has to say (`write`: by this thread) and returns what its
// gradient is made of: mine at the class, scale v at the others; both 0 for a row
// that leaves the scores alone, whatever they are.
struct RowGrad {
  float mine, scale;
  __device__ __forceinline__ bool any() const { return !(mine == 0.0f && scale == 0.0f); }
};
template <int FROM>
__device__ __forceinline__ RowGrad row_out(const LogpArgs& a, int64_t i, bool write, const RowEnd& e, const RowIn& in,
                                           float m, double o, float xa) {
  double slope = in.dlogp;
  if (FROM != kStats) {
    PolicyRow p = {0.0, 0.0};
    if (a.adv != nullptr) p = policy_row(a, e.logp, in.old_logp, in.ref_logp, in.adv);
    slope = in.weight == 0.0f ? 0.0 : p.slope * (double)in.weight;
    if (!e.live || xa == -kInf) slope = 0.0;
    if (write) {
      if (a.logp != nullptr) a.logp[i] = e.live ? (float)e.logp : 0.0f;
      if (a.stats != nullptr) {
        a.stats[2 * i] = e.live ? m : 0.0f;
        a.stats[2 * i + 1] = e.live ? (float)o : 0.0f;
      }
      if (a.adv != nullptr) {
        if (a.loss != nullptr) a.loss[i] = e.live ? (float)p.loss : 0.0f;
        if (a.dlogp != nullptr) a.dlogp[i] = (float)slope;
      }
    }
  }
  RowGrad g = {0.0f, 0.0f};
  if (e.live && xa != -kInf && slope != 0.0) {
    const double k = slope * a.inv_T * e.against;
    g.mine = (float)k;
    g.scale = o == 0.0 ? 0.0f : (float)(-k * rcp_64(o));
  }
  return g;
}

// The class's element of a vector of classes c0, c0 + 1, ...
template <int VE>
__device__ __forceinline__ void set_class(float (&f)[VE], int32_t cls, int32_t c0, float v) {
  const uint32_t at = (uint32_t)cls - (uint32_t)c0;  // (cls may be any number)
  if (at < (uint32_t)VE) {
#pragma unroll
    for (int q = 0; q < VE; ++q) f[q] = at == (uint32_t)q ? v : f[q];
  }
}

// One thread per row of at most CMAX classes, R rows a workgroup; rows and
// gradients pass through LDS, so that memory sees whole lines: packed rows of an odd
// length as they lie there, 16 bytes at a time, others (up to 8 classes; longer ones
// do not come here) in rows of C | 1 words.  Four classes at a time, -inf behind the
// row's end.  Step of 581,012 x 7 f32: 12.6 us, floor 8.3 (19.1 when rows were staged word
// by word and the exponentials were FP64).  Vector instructions, 432 a wave and some 250
// of them the row's FP64, are 6.6 us of it by the counters: what is left is that a
// workgroup's loads, work and stores follow each other, and that nearly all workgroups
// run at once, in phase.
constexpr int kShortStep = 4;
template <int DT, int R, int CMAX, int FROM>
__global__ void __launch_bounds__(R) k_logp_short(const LogpArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, V = (CMAX + VE - 1) / VE;
  extern __shared__ __align__(16) float lds[];
  const Span span = row_span(a);
  const int tid = threadIdx.x;
  const int64_t i0 = span.lo + int64_t(blockIdx.x) * R, i = i0 + tid;
  if (i0 >= span.hi) return;
  const int32_t rows = (int32_t)(span.hi - i0 < R ? span.hi - i0 : R);
  const int32_t C = a.C, P = C | 1, all = rows * C;
  const RowDiv by_c(C);
  const Elem* __restrict__ xg = static_cast<const Elem*>(a.x) + i0 * a.ld;
  const bool mine = tid < rows;
  int32_t cls = -1;
  RowIn in = {};
  float m = -kInf;
  double o = 0.0;
  if (mine) {
    cls = row_class(a, i, true);
    in = row_in<FROM>(a, i);
    if (FROM == kStats) {
      m = a.stats[2 * i];
      o = a.stats[2 * i + 1];
    }
  }
  if (CMAX > 8 || ((C & 1) && a.ld == C)) {
    Vec16<DT> raw[V];
    load_vecs<DT, V>(xg, tid * VE, R * VE, all, raw);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int32_t e = (tid + j * R) * VE;
      float f[VE];
      unpack<DT>(raw[j], f);
      if (e < all) __builtin_memcpy(__builtin_assume_aligned(lds + e, 16), f, sizeof(f));
    }
  } else {
    Staged<R, CMAX, float> xs;
    xs.load(
        rows, C, a.ld == C, by_c, [&](int32_t e) { return Score<DT>::to_f32(xg[(uint32_t)e]); },
        [&](int32_t row, int32_t c) { return Score<DT>::to_f32(xg[row * a.ld + c]); });
    xs.put(rows, C, by_c, lds);
  }
  __syncthreads();
  float* __restrict__ x = lds + tid * P;
  if (mine) {
    const bool named = cls >= 0;
    const float xa = named ? x[cls] : 0.0f;
    float v[CMAX];
#pragma unroll
    for (int c0 = 0; c0 < CMAX; c0 += kShortStep) {
      if (c0 < C) {
#pragma unroll
        for (int q = 0; q < kShortStep; ++q) {
          const int c = c0 + q;
          v[c] = c < C ? x[c] : -kInf;  // (the read stays inside the LDS of the launch)
          if (FROM != kStats) m = c == cls ? m : __builtin_fmaxf(m, v[c]);
        }
      }
    }
    const float mf = m == -kInf ? 0.0f : m;
#pragma unroll
    for (int c0 = 0; c0 < CMAX; c0 += kShortStep) {
      if (c0 < C) {
        float w[kShortStep];
#pragma unroll
        for (int q = 0; q < kShortStep; ++q) {
          v[c0 + q] = FROM == kStats ? grad_term(a, v[c0 + q] - mf) : sum_term(a, v[c0 + q] - mf);
          w[q] = c0 + q == cls ? 0.0f : v[c0 + q];
        }
        if (FROM != kStats) o += (double)sum_of(w);
      }
    }
    RowEnd e = row_end(a.inv_T, named, m, o, xa);
    if (FROM != kStats && next_to_border(a, e, in)) {
      o = 0.0;
      for (int c = 0; c < C; ++c)
        if (c != cls) o += exp2_64(((double)x[c] - (double)mf) * a.c);
      e = row_end(a.inv_T, named, m, o, xa);
    }
    const RowGrad g = row_out<FROM>(a, i, true, e, in, m, o, xa);
    if (a.grad != nullptr) {
#pragma unroll
      for (int c = 0; c < CMAX; ++c)
        if (c < C) x[c] = !g.any() ? 0.0f : (c == cls ? g.mine : v[c] * g.scale);
    }
  }
  if (a.grad != nullptr) {
    __syncthreads();
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i0 * a.ldg;
    if (CMAX > 8 || ((C & 1) && a.ldg == C)) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int32_t e = (tid + j * R) * VE;
        if (e < all) {
          float f[VE];
          __builtin_memcpy(f, __builtin_assume_aligned(lds + e, 16), sizeof(f));
          store_tail<DT>(gr, e, all, pack<DT>(f));
        }
      }
    } else {
      unstage<R, CMAX>(
          rows, C, a.ldg == C, by_c, lds, [&](int32_t e, float f) { gr[(uint32_t)e] = Score<DT>::from_f32(f); },
          [&](int32_t row, int32_t c, float f) { gr[row * a.ldg + c] = Score<DT>::from_f32(f); });
    }
  }
}

// NT lanes for a row that their V vectors of 16 bytes each hold whole, B rows one
// after the other in registers.  What is FP64 about a row (some 250 instructions where
// there is a policy) is done for B rows at once: lane b of the NT has row b.  From some
// 200 classes on it is near memory's rate (steps of 67,108 x 1,000 bf16: 51 us, 5.3 TB/s;
// of 33,537 x 2,001 f32: 101 us, 5.3 TB/s), with 16-bit scores near that of the vector
// instructions too.  Below that these bound it, the row's ends and odd tails most (600,000
// x 33 bf16: sums 34 us, floor 9, steps 48 to 55, floor 17; two thirds of the time by the
// counters).
template <int DT, int NT, int V, int B, int FROM>
__global__ void __launch_bounds__(256) k_logp_wave(const LogpArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, R = 64 / NT;
  const Span span = row_span(a);
  const int lane = threadIdx.x & (NT - 1), sub = (threadIdx.x & 63) / NT;
  const int64_t first = span.lo + a.row0 + (int64_t(blockIdx.x) * 4 + threadIdx.x / 64) * (R * B) + sub;
  if (first - sub >= span.hi) return;
  const int32_t C = a.C, c0 = lane * VE;
  const Elem* __restrict__ x = static_cast<const Elem*>(a.x);
  auto row = [&](int b) { return first + b * R < span.hi ? first + b * R : span.hi - 1; };
  Vec16<DT> raw[B][V];
  int32_t cls_of[B];
#pragma unroll
  for (int b = 0; b < B; ++b) cls_of[b] = a.cls[row(b)];
#pragma unroll
  for (int b = 0; b < B; ++b) load_vecs<DT, V>(x + row(b) * a.ld, c0, NT * VE, C, raw[b]);
  const int mine = lane < B ? lane : B - 1;
  const int64_t i = row(mine);
  const bool own = lane < B && first + mine * R < span.hi;
  const int32_t cls = row_class(a, i, own);
  const bool named = cls >= 0;
  const float xa = named ? Score<DT>::to_f32(x[i * a.ld + cls]) : 0.0f;
  const RowIn in = row_in<FROM>(a, i);
  float m_of[B], m = -kInf;
  double o = 0.0;
#pragma unroll
  for (int b = 0; b < B; ++b) {
    if (FROM == kStats) {
      m_of[b] = a.stats[2 * row(b)];
      continue;
    }
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[VE];
      forget<DT>(raw[b][j]);
      unpack<DT>(raw[b][j], f);
      set_class<VE>(f, cls_of[b], c0 + j * NT * VE, -kInf);
      top = __builtin_fmaxf(top, max_of(f));
      settle(top);  // (vector by vector: fewer registers)
    }
    top = lanes_reduce<NT>(top, [](float p, float q) { return __builtin_fmaxf(p, q); });
    const float base = top == -kInf ? 0.0f : top;
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j > 0 && j * NT * VE >= C) break;
      float f[VE];
      forget<DT>(raw[b][j]);
      unpack<DT>(raw[b][j], f);
      set_class<VE>(f, cls_of[b], c0 + j * NT * VE, -kInf);
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = sum_term(a, f[q] - base);
      sum += (double)sum_of(f);
      settle(sum);
    }
    sum = lanes_reduce<NT>(sum, [](double p, double q) { return p + q; });
    m_of[b] = top;
    if (mine == b) {
      m = top;
      o = sum;
    }
  }
  if (FROM == kStats) {
    m = a.stats[2 * i];
    o = a.stats[2 * i + 1];
  }
  RowEnd e = row_end(a.inv_T, named, m, o, xa);
  if (FROM != kStats) {
    const bool near = own && next_to_border(a, e, in);
    if (__any(near)) {
#pragma unroll 1
      for (int b = 0; b < B; ++b) {
        const Elem* __restrict__ xr = x + row(b) * a.ld;
        const int32_t skip = a.cls[row(b)];
        const float top = __shfl(m, (threadIdx.x & 63 & ~(NT - 1)) + b, 64);
        const double base = top == -kInf ? 0.0 : (double)top;
        double sum = 0.0;
#pragma unroll 1
        for (int32_t k = lane; k < C; k += 4 * NT) {
          float f[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = k + q * NT < C ? Score<DT>::to_f32(xr[k + q * NT]) : -kInf;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sum += k + q * NT == skip ? 0.0 : exp2_64(((double)f[q] - base) * a.c);
        }
        sum = lanes_reduce<NT>(sum, [](double p, double q) { return p + q; });
        if (near && mine == b) o = sum;
      }
      e = row_end(a.inv_T, named, m, o, xa);
    }
  }
  const RowGrad all = row_out<FROM>(a, i, own, e, in, m, o, xa);
  if (a.grad == nullptr) return;
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int from = (threadIdx.x & 63 & ~(NT - 1)) + b;
    const RowGrad g = {__shfl(all.mine, from, 64), __shfl(all.scale, from, 64)};
    if (first + b * R >= span.hi) continue;
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + (first + b * R) * a.ldg;
    const float base = m_of[b] == -kInf ? 0.0f : m_of[b];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j > 0 && j * NT * VE >= C) break;
      float f[VE];
      forget<DT>(raw[b][j]);
      unpack<DT>(raw[b][j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = g.any() ? grad_term(a, f[q] - base) * g.scale : 0.0f;
      set_class<VE>(f, cls_of[b], c0 + j * NT * VE, g.mine);
      store_tail<DT>(gr, c0 + j * NT * VE, C, pack<DT>(f));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The sums of N neighbouring lanes, each o against its own m, as one against the
// largest m.
template <int N>
__device__ __forceinline__ void join_lanes(double c, float& m, double& o) {
  const float top = lanes_reduce<N>(m, [](float p, float q) { return __builtin_fmaxf(p, q); });
  // (o of 0 or NaN stays what it is; a maximum of -inf has o = 0 or NaN)
  if (m != top && m != -kInf) o *= exp2_64(((double)m - (double)top) * c);
  m = top;
  o = lanes_reduce<N>(o, [](double p, double q) { return p + q; });
}
// The same of a workgroup's W waves; sh_m, sh_o: [W].
template <int W>
__device__ __forceinline__ void join_waves(double c, float& m, double& o, float* sh_m, double* sh_o) {
  const int tid = threadIdx.x;
  join_lanes<64>(c, m, o);
  if ((tid & 63) == 0) {
    sh_m[tid >> 6] = m;
    sh_o[tid >> 6] = o;
  }
  __syncthreads();
  m = sh_m[tid & (W - 1)];
  o = sh_o[tid & (W - 1)];
  join_lanes<W>(c, m, o);
}

// The sum over a row's other classes in FP64, by a workgroup (which all of it calls).
template <int DT, int NT>
__device__ __forceinline__ double exact_sum(const typename Score<DT>::Elem* __restrict__ xr, int32_t C, int32_t cls,
                                            float m, double c, double* sh) {
  constexpr int VE = Score<DT>::kVec;
  const double base = m == -kInf ? 0.0 : (double)m;
  double o = 0.0;
#pragma unroll 1
  for (int32_t c0 = threadIdx.x * VE; c0 < C; c0 += NT * VE) {
    float f[VE];
    load_chunk<DT>(xr, c0, C, f);
    set_class<VE>(f, cls, c0, -kInf);
#pragma unroll
    for (int q = 0; q < VE; ++q) o += exp2_64(((double)f[q] - base) * c);
  }
  return block_sum<NT>(o, sh);
}

// The end of a workgroup's row, in all its threads: the first wave does what is FP64
// about it.  A row next to a border has its sum taken again; what the caller has of it
// in registers need not be kept for that, it has it read again.
struct RowShared {
  float mine, scale;
  int again;
};
template <int DT, int NT, int FROM, bool GRAD, typename Reload>
__device__ __forceinline__ RowGrad finish_row(const LogpArgs& a, int64_t i, bool write,
                                              const typename Score<DT>::Elem* __restrict__ xr, int32_t cls, float m,
                                              double o, double* sh, RowShared& out, Reload reload) {
  const bool first = threadIdx.x < 64, writes = write && threadIdx.x == 0;
  if (first) {
    const RowIn in = row_in<FROM>(a, i);
    const float xa = cls >= 0 ? Score<DT>::to_f32(xr[cls]) : 0.0f;
    const RowEnd e = row_end(a.inv_T, cls >= 0, m, o, xa);
    const RowGrad g = row_out<FROM>(a, i, writes, e, in, m, o, xa);
    if (threadIdx.x == 0) out = RowShared{g.mine, g.scale, FROM != kStats && next_to_border(a, e, in)};
  }
  if (!GRAD && a.adv == nullptr) return RowGrad{0.0f, 0.0f};  // (nothing follows)
  __syncthreads();
  if (FROM != kStats && out.again) {
    o = exact_sum<DT, NT>(xr, a.C, cls, m, a.c, sh);
    if (first) {
      const RowIn in = row_in<FROM>(a, i);
      const float xa = Score<DT>::to_f32(xr[cls]);
      const RowGrad g = row_out<FROM>(a, i, writes, row_end(a.inv_T, true, m, o, xa), in, m, o, xa);
      if (threadIdx.x == 0) out = RowShared{g.mine, g.scale, 0};
    }
    __syncthreads();
    reload();
  }
  return RowGrad{out.mine, out.scale};
}

// A workgroup of NT threads for a row that their V vectors each hold whole: one read
// where the gradient follows.  The first wave does what is FP64 about the row.  Memory
// bounds it: steps of 22,369 x 3,000 bf16 50 us (5.4 TB/s; 122 when each row was read
// twice by 256 threads), of 8,388 x 8,000 bf16 45 us.  A row that fills its registers
// badly waits for its own end (13,421 x 5,000 bf16, 625 vectors of 1,024: 58 to 65 us).
template <int DT, int NT, int V>
__global__ void __launch_bounds__(NT, 8) k_logp_wide(const LogpArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, W = NT / 64;
  __shared__ float sh_m[W];
  __shared__ double sh_o[W];
  __shared__ RowShared sh_end;
  const Span span = row_span(a);
  const int tid = threadIdx.x;
  const int64_t i = span.lo + a.row0 + blockIdx.x;
  if (i >= span.hi) return;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  const int32_t C = a.C, c0 = tid * VE;
  const int32_t cls = row_class(a, i, tid == 0);
  const bool named = cls >= 0;
  Vec16<DT> raw[V];
  float m = -kInf;
  double o = 0.0;
  if (named) {
    load_vecs<DT, V>(xr, c0, NT * VE, C, raw);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[VE];
      forget<DT>(raw[j]);
      unpack<DT>(raw[j], f);
      set_class<VE>(f, cls, c0 + j * NT * VE, -kInf);
      m = __builtin_fmaxf(m, max_of(f));
      settle(m);  // (vector by vector: fewer registers)
    }
    const float base = m == -kInf ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j > 0 && j * NT * VE >= C) break;
      float f[VE];
      forget<DT>(raw[j]);
      unpack<DT>(raw[j], f);
      set_class<VE>(f, cls, c0 + j * NT * VE, -kInf);
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = sum_term(a, f[q] - base);
      o += (double)sum_of(f);
      settle(o);
    }
    join_waves<W>(a.c, m, o, sh_m, sh_o);
  }
  const RowGrad g = finish_row<DT, NT, kSums, true>(a, i, true, xr, cls, m, o, sh_o, sh_end,
                                                  [&] { load_vecs<DT, V>(xr, c0, NT * VE, C, raw); });
  const float base = m == -kInf ? 0.0f : m;
  Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (j > 0 && j * NT * VE >= C) break;
    float f[VE] = {};
    if (g.any()) {
      forget<DT>(raw[j]);
      unpack<DT>(raw[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = grad_term(a, f[q] - base) * g.scale;
      set_class<VE>(f, cls, c0 + j * NT * VE, g.mine);
    }
    store_stream<DT>(gr, c0 + j * NT * VE, C, pack<DT>(f));
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One workgroup per row, or per part of one: part_len classes (a multiple of
// NT * kBlk) of a row that n_parts workgroups share.  The sum is taken against a
// reference that is the first maximum the thread meets and moves only when a
// score is above it by 2^20 in the exponential; a second read writes the gradient.
// Parts leave their sums behind; where no gradient follows, the last workgroup of
// a row to arrive adds them up, else a second launch does.
//
// Memory bounds it where rows are many: step of 4,096 x 131,072 bf16 419 us (4.9 TB/s of
// what has to move, the rate of a copy; the second read comes from the last-level
// cache), gradient of 2,048 x 50,001 f32 148 us (5.5 TB/s), sums of 4,096 x 65,537 bf16
// 112 to 119 us (4.5 to 4.8 TB/s; 94 in a preference step, which ends on the rows that
// the next one begins with).  Loading the next block before this one is worked on made it
// slower (policy loss of 1,000 x 32,003 f16: 19.4 us, 17.6 without): four to eight
// workgroups a CU cover for each other.  What is left there is the chain of a row of
// its own, class, scores, joined sums, FP64 (4 us of 17, floor 10), and 3 us not accounted
// for.
template <int DT, int NT, int FROM, bool GRAD>
__global__ void __launch_bounds__(NT, 8) k_logp_block(const LogpArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, BLK = kBlk<DT>, W = NT / 64;
  __shared__ float sh_m[W];
  __shared__ double sh_o[W];
  __shared__ RowShared sh_end;
  __shared__ int sh_last;
  const Span span = row_span(a);
  const int tid = threadIdx.x;
  const uint32_t in_launch = a.n_parts > 1 ? blockIdx.x / (uint32_t)a.n_parts : blockIdx.x;
  const int32_t part = (int32_t)(blockIdx.x - in_launch * (uint32_t)a.n_parts);
  const int64_t row = a.row0 + in_launch, i = a.reverse ? span.hi - 1 - row : span.lo + row;
  if (row >= span.hi - span.lo) return;
  const int32_t lo = part * a.part_len;
  const int32_t hi = a.C - lo < a.part_len ? a.C : lo + a.part_len;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  constexpr bool kFromScores = FROM == kSums || FROM == kParts;
  const int32_t cls = row_class(a, i, tid == 0 && part == 0);
  const bool named = cls >= 0;
  float m = -kInf;
  double o = 0.0;
  if (kFromScores && named) {
    float ref = -kInf;
    const int32_t c0 = tid * VE;
    RawBlock<DT> raw = load_block<DT, NT>(xr, lo, hi);
    for (int32_t base = lo;;) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        if (j > 0 && base + j * NT * VE >= hi) break;
        float f[VE];
        unpack<DT>(raw.v[j], f);
        set_class<VE>(f, cls, base + c0 + j * NT * VE, -kInf);
        const float vm = max_of(f);
        m = __builtin_fmaxf(m, vm);
        if ((vm - ref) * a.c_hi > 20.0f) {  // (the first finite score among them)
          o *= exp2_64(((double)ref - (double)vm) * a.c);
          ref = vm;
        }
        const float rf = ref == -kInf ? 0.0f : ref;
#pragma unroll
        for (int q = 0; q < VE; ++q) f[q] = sum_term(a, f[q] - rf);
        o += (double)sum_of(f);
        __builtin_amdgcn_sched_barrier(0);  // (vector by vector: fewer registers)
      }
      base += NT * BLK;
      if (base >= hi) break;
      raw = load_block<DT, NT>(xr, base, hi);
    }
    if (ref != m && m != -kInf) o *= exp2_64(((double)ref - (double)m) * a.c);
    join_waves<W>(a.c, m, o, sh_m, sh_o);
  }
  PartSum* __restrict__ parts = a.parts + row * a.n_parts;
  if constexpr (FROM == kParts) {
    if (tid == 0) {
      __hip_atomic_store(&parts[part].o, o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&parts[part].m, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if constexpr (GRAD) return;
    // (at most 64 parts: no byte carries into its neighbour)
    uint32_t* word = a.arrived + row / 4;
    const int shift = (int)(row % 4) * 8;
    if (tid == 0) {
      const uint32_t before = __hip_atomic_fetch_add(word, 1u << shift, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      sh_last = (before >> shift & 0xffu) == (uint32_t)a.n_parts - 1u;
    }
    __syncthreads();
    if (!sh_last) return;
    if (tid == 0)
      __hip_atomic_fetch_sub(word, (uint32_t)a.n_parts << shift, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if constexpr (FROM == kJoin || FROM == kParts) {
    m = -kInf;
    o = 0.0;
    const int lane = tid & 63;
    if (lane < a.n_parts) {  // (at most 64 parts, as many as a row has steps of the split)
      o = __hip_atomic_load(&parts[lane].o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      m = __hip_atomic_load(&parts[lane].m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    join_lanes<64>(a.c, m, o);
  } else if constexpr (FROM == kStats) {
    m = a.stats[2 * i];
    o = a.stats[2 * i + 1];
  }
  const RowGrad g =
      finish_row<DT, NT, FROM, GRAD>(a, i, FROM == kParts || part == 0, xr, cls, m, o, sh_o, sh_end, [] {});
  if constexpr (GRAD && FROM != kParts) {
    const float mf = m == -kInf ? 0.0f : m;
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
    for (int32_t base = lo; base < hi; base += NT * BLK) {
      RawBlock<DT> out = {};
      if (g.any()) {
        const RawBlock<DT> raw = load_block<DT, NT>(xr, base, hi);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          if (j > 0 && base + j * NT * VE >= hi) break;
          float f[VE];
          unpack<DT>(raw.v[j], f);
#pragma unroll
          for (int q = 0; q < VE; ++q) f[q] = grad_term(a, f[q] - mf) * g.scale;
          set_class<VE>(f, cls, base + tid * VE + j * NT * VE, g.mine);
          out.v[j] = pack<DT>(f);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      store_block<DT, NT>(gr, base, hi, out);
    }
  }
}

// ------------------------------------------------------------------- pairs --

struct PairArgs {
  const void* x;
  int64_t n, ld;
  const int32_t* cls;
  double inv_T;
  const int64_t* offsets;
  const float *ref_logp, *weight;
  double beta, smoothing;
  int32_t C, n_pairs, average;
  const float* stats;
  float *loss, *rewards, *dlogp;
  int32_t* err;
};

// One workgroup per pair: the two sequences' sums of logp - ref over the rows that
// count (statistics other than (0, 0)), in FP64 in a fixed order, then the slope of
// each row.  logp is taken from the statistics again: its FP32 value is off by up to
// 2^-24 |logp|, some 10 times what o is, and the sums are small differences of many.
// Latencies bound it: offsets, statistics, score, FP64 (4 pairs of 25 rows: 4.6 us).  A
// pair has one workgroup however long it is: the loss of one pair of 100,000 rows of 7
// classes takes 143 us, of two of 50,000 73.
template <int DT, int NT>
__global__ void __launch_bounds__(NT) k_pairs(const PairArgs a) {
  __shared__ double sh[4][NT / 64];
  const int tid = threadIdx.x, wid = tid >> 6;
  const int64_t p = blockIdx.x;
  // (no rows but those that the launch before had: of others there are no statistics)
  const Span span = span_of(a.offsets, 2 * a.n_pairs, a.n);
  int64_t cut[3];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const int64_t v = a.offsets[2 * p + u];
    const int64_t from = u == 0 ? span.lo : cut[u - 1];
    cut[u] = v < from ? from : v > span.hi ? span.hi : v;
    bad = bad || cut[u] != v;
  }
  if (bad && tid == 0) dev_error(a.err, GBDT_E_RANGE);
  // a row's class and score, if it counts; sum: logp - ref and rows of both sequences
  uint32_t moves = 0u;  // the thread's first 32 rows: whether they have a gradient
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  auto score = [&](int64_t i, bool& counts) {
    const float m = a.stats[2 * i], o = a.stats[2 * i + 1];
    const int32_t cls = a.cls[i];
    counts = !(m == 0.0f && o == 0.0f) && (uint32_t)cls < (uint32_t)a.C;
    return counts ? Score<DT>::to_f32(static_cast<const typename Score<DT>::Elem*>(a.x)[i * a.ld + cls]) : -kInf;
  };
  int32_t turn = 0;
  for (int64_t i = cut[0] + tid; i < cut[2]; i += NT, ++turn) {
    const double ref = a.ref_logp == nullptr ? 0.0 : (double)a.ref_logp[i];
    bool counts;
    const float xa = score(i, counts);
    if (!counts) continue;
    const double lead = row_end(a.inv_T, true, a.stats[2 * i], a.stats[2 * i + 1], xa).logp - ref;
    const bool second = i >= cut[1];
    sum[0] += second ? 0.0 : lead;
    sum[1] += second ? lead : 0.0;
    sum[2] += second ? 0.0 : 1.0;
    sum[3] += second ? 1.0 : 0.0;
    if (turn < 32) moves |= xa == -kInf ? 0u : 1u << turn;
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    sum[s] = wave_sum(sum[s]);
    if ((tid & 63) == 0) sh[s][wid] = sum[s];
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 4; ++s) sum[s] = across_waves<NT / 64>(sh[s], [](double u, double v) { return u + v; });
  double per[2], reward[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    per[s] = a.average && sum[2 + s] > 1.0 ? 1.0 / sum[2 + s] : 1.0;
    reward[s] = a.beta * sum[s] * per[s];
  }
  // (1 - e) log(1 + e^-z) + e log(1 + e^z), and its slope
  const double z = reward[0] - reward[1], e = a.smoothing;
  const double near = exp_64(-__builtin_fabs(z)), inv = 1.0 / (1.0 + near), tail = log1p_64(near);
  const double up = z < 0.0 ? near * inv : inv, down = z < 0.0 ? inv : near * inv;  // 1 / (1 + e^-z), 1 / (1 + e^z)
  const double lose = (z < 0.0 ? -z : 0.0) + tail, win = (z > 0.0 ? z : 0.0) + tail;
  double loss = (1.0 - e) * lose + (e == 0.0 ? 0.0 : e * win);
  double slope = e * up - (1.0 - e) * down;
  if (z != z) loss = slope = z;
  if (tid == 0) {
    if (a.loss != nullptr) a.loss[p] = (float)loss;
    if (a.rewards != nullptr) {
      a.rewards[2 * p] = (float)reward[0];
      a.rewards[2 * p + 1] = (float)reward[1];
    }
  }
  const float wt = a.weight == nullptr ? 1.0f : a.weight[p];
  slope = wt == 0.0f ? 0.0 : slope * (double)wt * a.beta;
  const float d[2] = {(float)(slope * per[0]), (float)(-slope * per[1])};
  turn = 0;
  for (int64_t i = cut[0] + tid; i < cut[2]; i += NT, ++turn) {
    bool counts, moving = moves >> (turn & 31) & 1u;
    if (turn >= 32) moving = score(i, counts) != -kInf;
    a.dlogp[i] = moving ? d[i >= cut[1]] : 0.0f;
  }
}

// -------------------------------------------------------------------- host --

template <int DT, int R, int CMAX, int FROM>
void launch_short(const LogpArgs& a, hipStream_t s) {
  // (a row's last step of classes, and the last vector, may end behind the rows)
  const size_t lds = size_t(R) * 4 * (a.C | 1) + 32;
  diag_begin(kDiagClassLogp, s);
  hipLaunchKernelGGL((k_logp_short<DT, R, CMAX, FROM>), dim3((unsigned)((a.n + R - 1) / R)), dim3(R), lds, s, a);
  diag_end(s);
}

template <int DT, int NT, int V, int B, int FROM>
void launch_wave(LogpArgs a, hipStream_t s) {
  constexpr int64_t kRows = 256 / NT * B;
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid * kRows) {
    const int64_t left = (a.n - a.row0 + kRows - 1) / kRows;
    diag_begin(kDiagClassLogp, s);
    hipLaunchKernelGGL((k_logp_wave<DT, NT, V, B, FROM>), dim3((unsigned)(left < kMaxRowGrid ? left : kMaxRowGrid)),
                       dim3(256), 0, s, a);
    diag_end(s);
  }
}

template <int DT, int NT, int V>
void launch_wide(LogpArgs a, hipStream_t s) {
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid) {
    const int64_t left = a.n - a.row0;
    diag_begin(kDiagClassLogp, s);
    hipLaunchKernelGGL((k_logp_wide<DT, NT, V>), dim3((unsigned)(left < kMaxRowGrid ? left : kMaxRowGrid)), dim3(NT), 0,
                       s, a);
    diag_end(s);
  }
}

template <int DT, int NT, int FROM, bool GRAD>
void launch_block(LogpArgs a, hipStream_t s) {
  constexpr int32_t kStep = NT * kBlk<DT>;
  if (a.n_parts == 1) a.part_len = (a.C + kStep - 1) / kStep * kStep;
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid) {
    const int64_t n = a.n - a.row0 < kMaxRowGrid ? a.n - a.row0 : kMaxRowGrid;
    diag_begin(kDiagClassLogp, s);
    hipLaunchKernelGGL((k_logp_block<DT, NT, FROM, GRAD>), dim3((unsigned)(n * a.n_parts)), dim3(NT), 0, s, a);
    diag_end(s);
  }
}

// Threads for a row.  Up to 8 classes one, and up to 32 where rows are packed and of
// odd length, whose LDS rows need no padding (600,000 steps of 31 f32: 30 us, 36 with
// lanes; of 16, with padding: 28, and 22 with lanes).  Then as many lanes as hold the
// row in at most 8 vectors each, up to a wave (33,554 steps of 2,000 bf16: 50 us, 80
// when the row was read twice).  A step of a longer row keeps it in a workgroup's
// registers while they take it: 512 threads rather than 1,024 up to 4,096 vectors, so
// that four rows a CU are at different stages (3,355 x 20,000 bf16: 49 us, 65 with
// 1,024).  Longer rows are read twice, 1,024 threads each, so that the second read
// finds more of them in the last-level cache.  Where no gradient follows, 256
// threads: more rows side by side (4,096 x 65,537 bf16 in a preference step: 94 us, 130
// with 1,024).  A gradient from statistics reads a row once: 256 threads up to 2,500
// vectors, 1,024 from there on (f32, 256 / 1,024: 13,421 x 5,000 94 / 120 us, 26,843 x 10,000 426 / 375,
// 13,421 x 20,000 424 / 390; bf16: 6,710 x 10,000 44 / 57, 13,421 x 20,000 212 / 198,
// 6,710 x 40,000 213 / 191).  Few long rows are split.
template <int DT, int FROM>
int launch_logp(LogpArgs a, hipStream_t s) {
  constexpr int VE = Score<DT>::kVec;
  constexpr int32_t kPartStep = 256 * kBlk<DT>;
  a.n_parts = 1;
  a.part_len = 0;
  const int32_t vecs = (a.C + VE - 1) / VE, steps = (a.C + kPartStep - 1) / kPartStep;
  const bool step = FROM == kSums && a.grad != nullptr;
  const bool packed = (a.C & 1) && a.ld == a.C && (a.grad == nullptr || a.ldg == a.C);
  if (a.C <= 8) {
    launch_short<DT, 64, 8, FROM>(a, s);
  } else if (packed && a.C <= 16) {
    launch_short<DT, 128, 16, FROM>(a, s);
  } else if (packed && a.C <= kRowsMaxClasses) {
    launch_short<DT, 64, 32, FROM>(a, s);
  } else if (vecs <= 4) {
    launch_wave<DT, 4, 1, 4, FROM>(a, s);
  } else if (vecs <= 8) {
    launch_wave<DT, 8, 1, 8, FROM>(a, s);
  } else if (vecs <= 16) {
    launch_wave<DT, 8, 2, 4, FROM>(a, s);
  } else if (vecs <= 32) {
    launch_wave<DT, 8, 4, 2, FROM>(a, s);
  } else if (vecs <= 64) {
    launch_wave<DT, 16, 4, 2, FROM>(a, s);
  } else if (vecs <= 128) {
    launch_wave<DT, 32, 4, 1, FROM>(a, s);
  } else if (vecs <= 256) {
    launch_wave<DT, 64, 4, 1, FROM>(a, s);
  } else if (vecs <= 512) {
    launch_wave<DT, 64, 8, 1, FROM>(a, s);
  } else if (a.n <= kSplitRows && steps >= 4) {
    const int32_t want = (int32_t)(kSplitGrid / a.n);
    const int32_t per = (steps + want - 1) / want;
    a.part_len = per * kPartStep;
    a.n_parts = (steps + per - 1) / per;
    if constexpr (FROM == kStats) {
      launch_block<DT, 256, kStats, true>(a, s);
    } else if (step) {
      launch_block<DT, 256, kParts, true>(a, s);
      launch_block<DT, 256, kJoin, true>(a, s);
    } else {
      launch_block<DT, 256, kParts, false>(a, s);
    }
  } else if (step && vecs <= 1024) {
    launch_wide<DT, 256, 4>(a, s);
  } else if (step && vecs <= 2048) {
    launch_wide<DT, 256, 8>(a, s);
  } else if (step && vecs <= 4096) {
    launch_wide<DT, 512, 8>(a, s);
  } else if (step && vecs <= 8192) {
    launch_wide<DT, 1024, 8>(a, s);
  } else if (FROM == kSums && !step) {
    launch_block<DT, 256, kSums, false>(a, s);
  } else if (FROM == kStats && vecs <= 2500) {
    launch_block<DT, 256, kStats, true>(a, s);
  } else {
    launch_block<DT, 1024, FROM, true>(a, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_logp");
}

template <int FROM>
int launch_logp(int32_t dtype, const LogpArgs& a, hipStream_t s) {
  switch (dtype) {
    case GBDT_DTYPE_F32: return launch_logp<GBDT_DTYPE_F32, FROM>(a, s);
    case GBDT_DTYPE_BF16: return launch_logp<GBDT_DTYPE_BF16, FROM>(a, s);
    default: return launch_logp<GBDT_DTYPE_F16, FROM>(a, s);
  }
}

int check_logp(const gbdt_scores* x, double temperature) {
  const int rc = check_scores(x);
  if (rc) return rc;
  if (!(temperature >= 1e-30) || !(temperature <= 1e30)) return fail(GBDT_E_ARG, "temperature out of [1e-30, 1e30]");
  return GBDT_OK;
}

LogpArgs logp_args(const gbdt_scores& x, const int32_t* classes, double temperature, void* ws) {
  LogpArgs a = {};
  a.x = x.data;
  a.n = x.n_rows;
  a.ld = x.row_stride;
  a.C = x.n_classes;
  a.cls = classes;
  a.c = kLog2e / temperature;
  a.inv_T = 1.0 / temperature;
  a.c_near = a.c_hi = (float)a.c;
  if ((double)a.c_hi >= a.c) a.c_hi = std::nextafterf(a.c_hi, 0.0f);
  a.c_lo = std::fmax((float)(a.c - (double)a.c_hi), 0x1p-126f);
  a.err = &static_cast<WsCtrl*>(ws)->err;
  a.parts = reinterpret_cast<PartSum*>(static_cast<char*>(ws) + sizeof(WsCtrl));
  a.arrived = static_cast<WsCtrl*>(ws)->arrived;
  return a;
}

int check_policy(const gbdt_policy* p) {
  if (!p) return fail(GBDT_E_ARG, "policy is null");
  if (!(p->clip_low >= 0.0) || !(p->clip_low <= 1.0)) return fail(GBDT_E_ARG, "clip_low out of [0, 1]");
  if (!(p->clip_high >= 0.0)) return fail(GBDT_E_ARG, "clip_high must be >= 0");
  if (!(p->kl >= 0.0) || !std::isfinite(p->kl)) return fail(GBDT_E_ARG, "kl must be finite and >= 0");
  return GBDT_OK;
}

int policy(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_policy* p, float* loss,
           float* logp, float* dlogp, float* stats, void* grad, int64_t grad_stride, bool step, void* ws,
           size_t ws_bytes, hipStream_t s) {
  int rc = check_logp(x, temperature);
  if (!rc) rc = check_policy(p);
  if (rc) return rc;
  if (x->n_rows == 0) return GBDT_OK;
  if (!classes || !p->old_logp || !p->advantage) return fail(GBDT_E_ARG, "classes, old_logp or advantage is null");
  if (!loss) return fail(GBDT_E_ARG, "loss is null");
  if (!step && (!dlogp || !stats)) return fail(GBDT_E_ARG, "dlogp or stats is null");
  if (step) rc = check_grad(*x, grad, grad_stride);
  if (!rc) rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  LogpArgs a = logp_args(*x, classes, temperature, ws);
  a.old_logp = p->old_logp;
  a.ref_logp = p->kl == 0.0 ? nullptr : p->ref_logp;
  a.adv = p->advantage;
  a.weight = p->weight;
  a.low = 1.0 - p->clip_low;
  a.high = 1.0 + p->clip_high;
  a.log_low = std::log(a.low);
  a.log_high = std::log(a.high);
  a.kl = p->kl;
  a.loss = loss;
  a.logp = logp;
  a.dlogp = dlogp;
  a.stats = stats;
  a.grad = grad;
  a.ldg = grad_stride;
  return launch_logp<kSums>(x->dtype, a, s);
}

// The preference step's workspace: that of the rows, then each row's statistics and
// slope.
constexpr size_t preference_rows_at() {
  return sizeof(WsCtrl) + kScoresPartBytes;
}

int check_pairs(const gbdt_pairs* p) {
  if (!p) return fail(GBDT_E_ARG, "pairs is null");
  if (p->n_pairs < 0 || p->n_pairs > 1 << 21) return fail(GBDT_E_ARG, "n_pairs out of [0, 2^21]");
  if (!std::isfinite(p->beta)) return fail(GBDT_E_ARG, "beta must be finite");
  if (!(p->smoothing >= 0.0) || !(p->smoothing < 0.5)) return fail(GBDT_E_ARG, "smoothing out of [0, 1/2)");
  return GBDT_OK;
}

// Threads for a pair by its rows in the mean: each of a thread's rows costs latencies
// (32 pairs of 128: 6 us with 256 threads, 10 with 64), each wave of a pair the pair's own
// arithmetic, which counts where pairs are many (a step of 9,375 pairs of 64 rows of 3
// classes: 28 us with 64 threads, 50 with 256).  1,024 threads pay for long pairs that do
// not fill the CUs (losses over 7 classes, 1,024 / 256 threads: 16 pairs of 1,500 rows
// 12 / 12 us, of 4,000 14 / 20; 128 of 4,000 19 / 28; 512 of 600 18 / 13, of 3,000
// 37 / 34; 1,024 of 4,000 79 / 65).
template <int DT>
void launch_pairs_of(const PairArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.n_pairs);
  if (a.n / a.n_pairs > 1500 && a.n_pairs < 512) {
    hipLaunchKernelGGL((k_pairs<DT, 1024>), grid, dim3(1024), 0, s, a);
  } else if (a.n / a.n_pairs <= 128 && a.n_pairs >= 2048) {
    hipLaunchKernelGGL((k_pairs<DT, 64>), grid, dim3(64), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_pairs<DT, 256>), grid, dim3(256), 0, s, a);
  }
}

int launch_pairs(const gbdt_pairs& p, const gbdt_scores& x, const int32_t* classes, double temperature,
                 const float* stats, float* loss, float* rewards, float* dlogp, void* ws, hipStream_t s) {
  PairArgs a = {};
  a.x = x.data;
  a.n = x.n_rows;
  a.ld = x.row_stride;
  a.C = x.n_classes;
  a.cls = classes;
  a.inv_T = 1.0 / temperature;
  a.offsets = p.offsets;
  a.ref_logp = p.ref_logp;
  a.weight = p.weight;
  a.beta = p.beta;
  a.smoothing = p.smoothing;
  a.n_pairs = p.n_pairs;
  a.average = p.average;
  a.stats = stats;
  a.loss = loss;
  a.rewards = rewards;
  a.dlogp = dlogp;
  a.err = &static_cast<WsCtrl*>(ws)->err;
  diag_begin(kDiagPairs, s);
  switch (x.dtype) {
    case GBDT_DTYPE_F32: launch_pairs_of<GBDT_DTYPE_F32>(a, s); break;
    case GBDT_DTYPE_BF16: launch_pairs_of<GBDT_DTYPE_BF16>(a, s); break;
    default: launch_pairs_of<GBDT_DTYPE_F16>(a, s);
  }
  diag_end(s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_pairs");
}

// Both passes: the rows' statistics (and logp, if asked for), the pairs, and the
// gradient where there is one.
int preference(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_pairs* p, float* loss,
               float* rewards, float* logp, float* dlogp, float* stats, void* grad, int64_t grad_stride, bool step,
               void* ws, size_t ws_bytes, hipStream_t s) {
  int rc = check_logp(x, temperature);
  if (!rc) rc = check_pairs(p);
  if (rc) return rc;
  if (p->n_pairs == 0) return GBDT_OK;
  if (!p->offsets || !loss) return fail(GBDT_E_ARG, "offsets or loss is null");
  if (x->n_rows > 0) {
    if (!classes) return fail(GBDT_E_ARG, "classes is null");
    if (!step && (!logp || !dlogp || !stats)) return fail(GBDT_E_ARG, "logp, dlogp or stats is null");
    if (step) rc = check_grad(*x, grad, grad_stride);
    if (rc) return rc;
  }
  rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  if (step) {
    if (ws_bytes < gbdt_preference_workspace_bytes(x->n_rows, x->n_classes))
      return fail(GBDT_E_ARG, "workspace smaller than gbdt_preference_workspace_bytes()");
    stats = reinterpret_cast<float*>(static_cast<char*>(ws) + preference_rows_at());
    dlogp = stats + 2 * x->n_rows;
  }
  LogpArgs a = logp_args(*x, classes, temperature, ws);
  a.range = p->offsets;
  a.last = 2 * p->n_pairs;
  a.logp = logp;
  a.stats = stats;
  if (x->n_rows > 0) rc = launch_logp<kSums>(x->dtype, a, s);
  if (!rc) rc = launch_pairs(*p, *x, classes, temperature, stats, loss, rewards, dlogp, ws, s);
  if (rc || !step || x->n_rows == 0) return rc;
  a.logp = nullptr;
  a.dlogp = dlogp;
  a.reverse = 1;  // the rows read last are still in the last-level cache
  a.grad = grad;
  a.ldg = grad_stride;
  return launch_logp<kStats>(x->dtype, a, s);
}

}  // namespace

int check_grad(const gbdt_scores& x, const void* grad, int64_t grad_stride) {
  if (!grad) return fail(GBDT_E_ARG, "grad is null");
  if (x.n_rows > 1 && grad_stride < x.n_classes) return fail(GBDT_E_SHAPE, "grad_stride smaller than n_classes");
  const uintptr_t es = x.dtype == GBDT_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(grad) % es) return fail(GBDT_E_ARG, "grad is misaligned");
  return GBDT_OK;
}

}  // namespace gbdt

using namespace gbdt;

extern "C" {

int gbdt_class_logp(const gbdt_scores* x, const int32_t* classes, double temperature, float* logp, float* stats,
                    void* ws, size_t ws_bytes, void* stream) {
  int rc = check_logp(x, temperature);
  if (rc) return rc;
  if (x->n_rows == 0) return GBDT_OK;
  if (!classes || !logp) return fail(GBDT_E_ARG, "classes or logp is null");
  rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  LogpArgs a = logp_args(*x, classes, temperature, ws);
  a.logp = logp;
  a.stats = stats;
  return launch_logp<kSums>(x->dtype, a, reinterpret_cast<hipStream_t>(stream));
}

int gbdt_class_logp_grad(const gbdt_scores* x, const int32_t* classes, double temperature, const float* stats,
                         const float* dlogp, void* grad, int64_t grad_stride, void* ws, size_t ws_bytes,
                         void* stream) {
  int rc = check_logp(x, temperature);
  if (rc) return rc;
  if (x->n_rows == 0) return GBDT_OK;
  if (!classes || !stats || !dlogp) return fail(GBDT_E_ARG, "classes, stats or dlogp is null");
  rc = check_grad(*x, grad, grad_stride);
  if (!rc) rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  LogpArgs a = logp_args(*x, classes, temperature, ws);
  a.stats = const_cast<float*>(stats);  // (read only, as dlogp)
  a.dlogp = const_cast<float*>(dlogp);
  a.grad = grad;
  a.ldg = grad_stride;
  return launch_logp<kStats>(x->dtype, a, reinterpret_cast<hipStream_t>(stream));
}

int gbdt_policy_loss(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_policy* p,
                     float* loss, float* logp, float* dlogp, float* stats, void* ws, size_t ws_bytes,
                     void* stream) {
  return policy(x, classes, temperature, p, loss, logp, dlogp, stats, nullptr, 0, false, ws, ws_bytes,
                reinterpret_cast<hipStream_t>(stream));
}

int gbdt_policy_step(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_policy* p,
                     float* loss, float* logp, void* grad, int64_t grad_stride, void* ws, size_t ws_bytes,
                     void* stream) {
  return policy(x, classes, temperature, p, loss, logp, nullptr, nullptr, grad, grad_stride, true, ws, ws_bytes,
                reinterpret_cast<hipStream_t>(stream));
}

size_t gbdt_preference_workspace_bytes(int64_t n_rows, int32_t n_classes) {
  return gbdt_scores_workspace_bytes(n_rows, n_classes) == 0 ? 0 : preference_rows_at() + size_t(n_rows) * 12;
}

int gbdt_preference_loss(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_pairs* p,
                         float* loss, float* rewards, float* logp, float* dlogp, float* stats, void* ws,
                         size_t ws_bytes, void* stream) {
  return preference(x, classes, temperature, p, loss, rewards, logp, dlogp, stats, nullptr, 0, false, ws, ws_bytes,
                    reinterpret_cast<hipStream_t>(stream));
}

int gbdt_preference_step(const gbdt_scores* x, const int32_t* classes, double temperature, const gbdt_pairs* p,
                         float* loss, float* rewards, void* grad, int64_t grad_stride, void* ws, size_t ws_bytes,
                         void* stream) {
  return preference(x, classes, temperature, p, loss, rewards, nullptr, nullptr, nullptr, grad, grad_stride, true, ws,
                    ws_bytes, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
