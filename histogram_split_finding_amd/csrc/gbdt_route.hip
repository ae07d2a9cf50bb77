// Rows sent to experts: the choice of k experts a row with their weights, the
// weights' gradient, and the experts' lists of places.
//
// With s the softmax or sigmoid values of a row's scores, J the chosen experts and
// d_j = dweight_j:
//   weight_j = scale w_j,  w_j = s_j / sum_J s or s_j,
//   sigmoid:                    dx_j = scale s_j s(-x_j) d_j,
//   sigmoid, renormalised:      dx_j = scale w_j s(-x_j) (d_j - sum_J w d),
//   softmax, renormalised:      dx_j = scale w_j (d_j - sum_J w d),
//   softmax:                    dx_j = scale s_j (d_j - sum_J s d),
//                               dx_c = -scale s_c sum_J s d outside J.
// d_j - sum_J w d cancels where one expert has nearly all: with u the dweight of J's
// largest score and R the softmax mass outside J (0 where renormalised) it is
//   (d_j - u) - sum_J w (d - u) + u R,
// whose terms are as small as the sum itself.  Where R is 1/2 or more nothing cancels,
// and u = 0 keeps small d_j beside a large u.

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

constexpr int kRouteThreads = 256;
constexpr float kMaxF32 = 3.40282346638528859812e38f;

struct RouteArgs {
  const void* x;
  int64_t n, ld;
  int32_t E, k;
  int32_t sigmoid, renorm;
  int32_t groups, kept, top, group_size;
  int32_t per_lane;   // experts of a lane, at most EPL
  int32_t log_lanes;  // lanes of a group of experts, as a power of two
  double scale;
  const float* bias;
  int32_t* classes;
  float* weights;
  const float* dweights;
  void* grad;
  int64_t ldg;
  int32_t* err;
  int64_t row0;  // of this launch
};

// A score as the softmax has it: NaN is out of service, +inf the largest number.
__device__ __forceinline__ float in_service(float f) { return f == f ? __builtin_fminf(f, kMaxF32) : -kInf; }

// 2^y of a score against the largest, y <= 0.  A NaN score has 0; one of +inf, which
// counts as the largest number and is then the largest score, 1.  (One instruction.)
__device__ __forceinline__ float share_32(float y) {
  return __builtin_fminf(__builtin_fmaxf(exp2_32(y), 0.0f), 1.0f);
}

// The choice's keys: the scores themselves, or choice values in FP64.  `taken` is
// below all keys but -inf; an FP64 key is taken by its upper word alone, whatever the
// lower one.  The larger of two keys: no NaN comes here, so FP64 has the bare
// instruction (the compiler's own would quiet both operands first).
template <bool BY_VALUE>
struct RouteKey;
template <>
struct RouteKey<false> {
  using T = float;
  static __device__ __forceinline__ T taken() { return -kInf; }
  static __device__ __forceinline__ T take(T v, bool it) { return it ? -kInf : v; }
  static __device__ __forceinline__ T larger(T a, T b) { return __builtin_fmaxf(a, b); }
  static __device__ __forceinline__ T smaller(T a, T b) { return __builtin_fminf(a, b); }
};
template <>
struct RouteKey<true> {
  using T = double;
  static __device__ __forceinline__ T taken() { return -0x1p1022; }
  static __device__ __forceinline__ T take(T v, bool it) {
    return __hiloint2double(it ? __double2hiint(taken()) : __double2hiint(v), __double2loint(v));
  }
  static __device__ __forceinline__ T larger(T a, T b) {
    T r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ T smaller(T a, T b) {
    T r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
};

__device__ __forceinline__ double sigmoid_64(float x, double* other = nullptr) {  // other: of -x
  const double e = exp2_64(-(double)__builtin_fabsf(x) * kLog2e);
  const double inv = rcp_64(1.0 + e);
  if (other != nullptr) *other = x < 0.0f ? inv : e * inv;
  return x < 0.0f ? e * inv : inv;
}

// NT lanes a row, EPL experts a lane at most, neighbours, and no lane with experts of
// two groups: of equal keys the first is in the lowest lane that has one.  The
// choice takes k rounds: the row's largest key by lane moves, the lane that has it by
// a ballot, its first place there by comparisons.  Round j's score is kept by the lane
// that works out weight j: the key itself, or read again where the key is a value.
//
// Vector instructions are its largest part, 1,584 a wave of four rows of 256 with a bias
// (16,384 rows: 19 us, 11 of them by the counters; 40 % of the instructions the rounds,
// 30 % FP64 sigmoids), 646 a wave of eight rows of 60 without (65,536 rows: 13 us, 8.7 of
// them); the rest are the rounds' dependent steps at 4 and 8 waves a SIMD.  More experts a lane save rounds' lane moves and
// lose waves that cover for each other (8 lanes of 32: 20 us; 32 lanes of 8: 20 us).
// One row takes 5.6 us, with 64 lanes (10 with 16).
template <int DT, int NT, int EPL, bool BY_VALUE>
__global__ void __launch_bounds__(kRouteThreads) k_route(const RouteArgs a) {
  using Elem = typename Score<DT>::Elem;
  using K = RouteKey<BY_VALUE>;
  using Key = typename K::T;
  constexpr int VE = Score<DT>::kVec, V = (EPL + VE - 1) / VE;
  constexpr int kRows = kRouteThreads / NT;
  constexpr int kMost = (GBDT_MAX_ROUTED + NT - 1) / NT;
  __shared__ int32_t all_chosen[kRows][GBDT_MAX_ROUTED];
  const int lane = threadIdx.x & (NT - 1), sub = threadIdx.x / NT;
  const int first_lane = (threadIdx.x & 63) & ~(NT - 1);  // of the row, in the wave
  const uint64_t below = ((uint64_t(1) << lane) - 1) << first_lane;  // the row's lanes below this one
  const int64_t row = a.row0 + int64_t(blockIdx.x) * kRows + sub;
  const bool mine = row < a.n;
  const int64_t i = mine ? row : a.n - 1;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  int32_t* __restrict__ chosen = all_chosen[sub];
  const int32_t group = lane >> a.log_lanes, within = lane & ((1 << a.log_lanes) - 1);
  const int32_t group_end = (group + 1) * a.group_size;
  int32_t e0 = group * a.group_size + within * a.per_lane, e1 = e0 + a.per_lane;
  e1 = e1 < group_end ? e1 : group_end;
  if (group >= a.groups || e0 >= e1) e0 = e1 = 0;
  const int32_t count = e1 - e0;
  float x[V * VE], bias[EPL];
  {
    Vec16<DT> raw[V];
    Vec16<GBDT_DTYPE_F32> raw_bias[EPL / 4];
    load_vecs<DT, V>(xr, e0, VE, a.E, raw);
    if (BY_VALUE && a.bias != nullptr) load_vecs<GBDT_DTYPE_F32, EPL / 4>(a.bias, e0, 4, a.E, raw_bias);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[VE];
      unpack<DT>(raw[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) x[j * VE + q] = __builtin_fmaxf(f[q], -kInf);  // (NaN: -inf)
    }
    if (BY_VALUE && a.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) bias[e] = __uint_as_float(raw_bias[e / 4].w[e % 4]);
    }
  }
  if (__any(count < EPL)) {  // what is another lane's
#pragma unroll
    for (int e = 0; e < EPL; ++e) x[e] = e < count ? x[e] : -kInf;
  }
  // the softmax's maximum and sum
  const bool softmax = !a.sigmoid && (BY_VALUE || !a.renorm);
  double top_x = 0.0, inv_total = 1.0;
  Key v[EPL];
  if (softmax) {
    float m = -kInf;
#pragma unroll
    for (int e = 0; e < EPL; ++e) m = __builtin_fmaxf(m, x[e]);
    m = __builtin_fminf(group_max<NT>(m), kMaxF32);
    top_x = m == -kInf ? 0.0 : (double)m;
    double total = 0.0;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const double w = exp2_64(((double)__builtin_fminf(x[e], kMaxF32) - top_x) * kLog2e);
      total += w;
      if constexpr (BY_VALUE) v[e] = w;
    }
    total = group_sum<NT>(total);
    inv_total = total > 0.0 ? 1.0 / total : 0.0;
    if constexpr (BY_VALUE) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[e] *= inv_total;
    }
  } else if constexpr (BY_VALUE) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = sigmoid_64(x[e]);
  }
  if constexpr (BY_VALUE) {
    if (a.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        v[e] += (double)bias[e];
        v[e] = v[e] == v[e] ? v[e] : -__builtin_inf();
      }
    }
    float least = x[0];
#pragma unroll
    for (int e = 1; e < EPL; ++e) least = __builtin_fminf(least, x[e]);
    if (__any(least == -kInf)) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[e] = x[e] > -kInf ? v[e] : -__builtin_inf();
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = x[e];
  }
  if (a.groups > 1) {
    // a group's two largest: of a lane's, then of its lanes'
    Key t1 = -__builtin_inf(), t2 = t1;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      if (BY_VALUE) t2 = K::larger(t2, K::smaller(t1, v[e]));
      t1 = K::larger(t1, v[e]);
    }
    for (int off = 1; off < 1 << a.log_lanes; off <<= 1) {
      const Key o1 = __shfl_xor(t1, off, 64);
      if (BY_VALUE) t2 = K::larger(K::larger(t2, __shfl_xor(t2, off, 64)), K::smaller(t1, o1));
      t1 = K::larger(t1, o1);
    }
    Key rank = t1;
    if (BY_VALUE && a.top == 2 && t2 > -__builtin_inf()) rank = t1 + t2;
    int32_t before = 0;  // groups ahead of this one
    for (int32_t g = 0; g < a.groups; ++g) {
      const Key other = __shfl(rank, first_lane + (g << a.log_lanes), 64);
      before += other > rank || (other == rank && g < group);
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) v[e] = K::take(v[e], before >= a.kept);
  }
  float xc[kMost], m = -kInf;
#pragma unroll
  for (int u = 0; u < kMost; ++u) xc[u] = -kInf;
  for (int32_t j = 0; j < a.k; ++j) {
    Key part[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) part[e] = v[e];
#pragma unroll
    for (int w = EPL / 2; w > 0; w /= 2) {
#pragma unroll
      for (int e = 0; e < w; ++e) part[e] = K::larger(part[e], part[e + w]);
    }
    const Key top = lanes_reduce<NT>(part[0], [](Key p, Key q) { return K::larger(p, q); });
    const bool left = top > K::taken(), has = part[0] == top && left;
    bool open = has && (__ballot(has) & below) == 0;  // this lane's, and not yet found
    const bool wins = open;
    int32_t at = 0;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
      const bool it = open && v[e] == top;
      v[e] = K::take(v[e], it);
      at = it ? e : at;
      open = open && !it;
    }
    // (class -1 where nothing is left)
    if (left ? wins : lane == 0) chosen[j] = left ? e0 + at : -1;
    if constexpr (!BY_VALUE) {
#pragma unroll
      for (int u = 0; u < kMost; ++u) xc[u] = j == lane + u * NT ? __builtin_fminf(top, kMaxF32) : xc[u];
    }
  }
  // the weights of places lane, lane + NT, ...
  double s[kMost], sum = 0.0;
  int32_t cls[kMost];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int32_t j = lane + u * NT;
    cls[u] = j < a.k ? chosen[j] : -1;
    if (BY_VALUE && cls[u] >= 0) xc[u] = __builtin_fminf(Score<DT>::to_f32(xr[cls[u]]), kMaxF32);
  }
#pragma unroll
  for (int u = 0; u < kMost; ++u) m = __builtin_fmaxf(m, xc[u]);
  if (!a.sigmoid && a.renorm) {
    // of the chosen alone: against the largest of them
    m = group_max<NT>(m);
    top_x = m == -kInf ? 0.0 : (double)m;
    inv_total = 1.0;
  }
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    s[u] = 0.0;
    if (u * NT < a.k && xc[u] > -kInf)
      s[u] = a.sigmoid ? sigmoid_64(xc[u]) : exp2_64(((double)xc[u] - top_x) * kLog2e) * inv_total;
    sum += s[u];
  }
  double inv = 1.0;
  if (a.renorm) {
    sum = group_sum<NT>(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
  }
  if (mine) {
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
      const int32_t j = lane + u * NT;
      if (j < a.k) {
        a.classes[row * a.k + j] = cls[u];
        a.weights[row * a.k + j] = (float)(s[u] * inv * a.scale);  // (scale / sum may overflow)
      }
    }
  }
}

// NT lanes a row that their V vectors of 16 bytes each hold whole.  A byte per
// expert in LDS says which place of the list has it: the mass outside the choice is
// summed by itself (as 1 less the rest it would lose its digits).  65,536 x 128 f32
// softmax: 14.3 us, 4.9 TB/s; all rows are in flight at once, so reads and writes do not
// overlap.  Other forms read the chosen scores alone: 12 us, floor 7.
template <int DT, int NT, int V>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(const RouteArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, kRows = kRouteThreads / NT, W = NT * V * VE;
  constexpr int kMost = (GBDT_MAX_ROUTED + NT - 1) / NT;
  __shared__ uint32_t all_place[kRows][W / 4];  // a byte per expert
  __shared__ float all_value[kRows][GBDT_MAX_ROUTED];
  const int lane = threadIdx.x & (NT - 1), sub = threadIdx.x / NT;
  const int first_lane = (threadIdx.x & 63) & ~(NT - 1);  // of the row, in the wave
  const int64_t row = a.row0 + int64_t(blockIdx.x) * kRows + sub;
  const bool mine = row < a.n;
  const int64_t i = mine ? row : a.n - 1;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  uint32_t* __restrict__ place = all_place[sub];
  float* __restrict__ value = all_value[sub];
  const int32_t E = a.E, c0 = lane * VE;
  const bool whole = !a.sigmoid && !a.renorm;  // all experts have a gradient
  int32_t cls[kMost];
  float xc[kMost], d[kMost];
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int32_t j = lane + u * NT;
    cls[u] = -1;
    d[u] = 0.0f;
    if (j < a.k) cls[u] = a.classes[i * a.k + j];
    if (cls[u] >= E) {
      if (mine) dev_error(a.err, GBDT_E_RANGE);
      cls[u] = -1;
    }
    if (cls[u] >= 0) d[u] = a.dweights[i * a.k + j];
  }
  Vec16<DT> raw[V];
  float m = -kInf, top_d = 0.0f;
  if (whole) load_vecs<DT, V>(xr, c0, NT * VE, E, raw);
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int q = 0; q < VE / 4; ++q) place[(j * NT + lane) * (VE / 4) + q] = 0u;
  }
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    xc[u] = -kInf;
    if (cls[u] >= 0) xc[u] = in_service(Score<DT>::to_f32(xr[cls[u]]));
    top_d = xc[u] > m ? d[u] : top_d;
    m = __builtin_fmaxf(m, xc[u]);
  }
  // of the largest chosen score: the score, and its dweight
  const auto larger = [](float p, float q) { return __builtin_fmaxf(p, q); };
  const auto add = [](double p, double q) { return p + q; };
  const float top = lanes_reduce<NT>(m, larger);
  const uint64_t has = __ballot(m == top) >> first_lane & (~uint64_t(0) >> (64 - NT));
  top_d = __shfl(top_d, first_lane + __ffsll((unsigned long long)has) - 1, 64);
  m = top;
  if (whole) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[VE];
      unpack<DT>(raw[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) m = __builtin_fmaxf(m, f[q]);  // (m is no NaN, so no NaN gets in)
    }
    m = lanes_reduce<NT>(__builtin_fminf(m, kMaxF32), larger);
  }
  const float base = m == -kInf ? 0.0f : m, c = (float)kLog2e;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int32_t j = lane + u * NT;
    if (cls[u] >= 0) {
      uint32_t* word = place + cls[u] / 4;
      const int shift = cls[u] % 4 * 8;
      if (atomicOr(word, (uint32_t)(j + 1) << shift) >> shift & 0xffu && mine) dev_error(a.err, GBDT_E_ARG);
    }
  }
  double rest = 0.0;  // the exponentials outside the choice
  if (whole) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[VE];
      unpack<DT>(raw[j], f);
#pragma unroll
      for (int w = 0; w < VE / 4; ++w) {
        const uint32_t at = place[(j * NT + lane) * (VE / 4) + w];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float e = share_32((f[w * 4 + q] - base) * c);
          f[w * 4 + q] = at >> (8 * q) & 0xffu ? 0.0f : e;
        }
      }
      rest += (double)sum_of(f);
    }
  }
  double s[kMost], away[kMost], sum = 0.0;
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    s[u] = 0.0;
    away[u] = 1.0;
    if (cls[u] >= 0 && !(xc[u] == -kInf)) {
      s[u] = a.sigmoid ? sigmoid_64(xc[u], &away[u]) : exp2_64(((double)xc[u] - (double)base) * kLog2e);
      sum += s[u];
    }
  }
  // w_j, and the share R that is not of the choice
  double inv = 1.0, R = 0.0, from = 0.0, mean = 0.0;
  if (whole || a.renorm) {
    sum = lanes_reduce<NT>(sum, add);
    if (whole) rest = lanes_reduce<NT>(rest, add);
    inv = sum + rest > 0.0 ? rcp_64(sum + rest) : 0.0;
    R = rest * inv;
    from = R < 0.5 ? (double)top_d : 0.0;
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
      if (u * NT >= a.k) break;
      s[u] *= inv;
      mean += s[u] == 0.0 ? 0.0 : s[u] * ((double)d[u] - from);
    }
    mean = lanes_reduce<NT>(mean, add);
  }
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int32_t j = lane + u * NT;
    if (cls[u] >= 0) {
      const double t = (double)d[u] - from - mean + from * R;
      value[j] = (float)(s[u] == 0.0 ? 0.0 : s[u] * away[u] * t * a.scale);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (!mine) return;
  Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
  const float others = (float)(-(mean + from * (1.0 - R)) * inv * a.scale);
  const bool odd = !(__builtin_fabsf(others) < kInf);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int32_t e0 = c0 + j * NT * VE;
    if (e0 >= E) break;
    float f[VE];
    if (whole) {
      unpack<DT>(raw[j], f);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const float e = share_32((f[q] - base) * c) * others;
        f[q] = odd && !(f[q] > -kInf) ? 0.0f : e;  // (out of service: 0, not 0 inf)
      }
    } else {
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < VE / 4; ++w) {
      const uint32_t at = place[(j * NT + lane) * (VE / 4) + w];
      if (at) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t p = at >> (8 * q) & 0xffu;
          // (two places that met in one byte: an error already, but none out of bounds)
          if (p) f[w * 4 + q] = value[(p - 1u) & (GBDT_MAX_ROUTED - 1)];
        }
      }
    }
    store_tail<DT>(gr, e0, E, pack<DT>(f));
  }
}

// ------------------------------------------------------------------- lists --

struct ListArgs {
  const int32_t* classes;
  int64_t n;
  int32_t E, blocks;
  int64_t chunk;  // places of a workgroup
  uint32_t* counts;  // [blocks][E]
  int32_t *offsets, *order, *place, *err;
};

__device__ __forceinline__ int32_t listed_class(const ListArgs& a, int64_t p, bool report) {
  const int32_t c = a.classes[p];
  if (c >= a.E && report) dev_error(a.err, GBDT_E_RANGE);
  return c >= a.E ? -1 : c;
}

constexpr int kCountThreads = 256;
__global__ void __launch_bounds__(kCountThreads) k_list_count(const ListArgs a) {
  __shared__ uint32_t count[GBDT_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.E; e += kCountThreads) count[e] = 0u;
  __syncthreads();
  const int64_t lo = int64_t(blockIdx.x) * a.chunk, hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  for (int64_t p = lo + threadIdx.x; p < hi; p += kCountThreads) {
    const int32_t c = listed_class(a, p, false);
    if (c >= 0) atomicAdd(&count[c], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kCountThreads) a.counts[int64_t(blockIdx.x) * a.E + e] = count[e];
}

// Each workgroup adds up the counts itself (of all workgroups: where the experts'
// lists begin; of those before it: where its own part of each list does), then takes
// its places in order: a wave's 64 at a time, each behind the places before it of
// the same expert, which the wave finds by a ballot per bit of the expert.  Latencies
// bound it (131,072 places of 256 experts: 6.5 us, and 4 us for the counts).
template <int NT>
__global__ void __launch_bounds__(NT) k_list_place(const ListArgs a) {
  constexpr int W = NT / 64, EPT = (GBDT_MAX_EXPERTS + NT - 1) / NT;
  __shared__ uint32_t next[W][GBDT_MAX_EXPERTS];
  __shared__ int32_t total_of[GBDT_MAX_EXPERTS], before_of[GBDT_MAX_EXPERTS];
  __shared__ int32_t sh[32];
  const int tid = threadIdx.x, wid = tid >> 6, lane = tid & 63;
  const int64_t lo = int64_t(blockIdx.x) * a.chunk, hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  const int64_t share = (a.chunk + W * 64 - 1) / (W * 64) * 64;
  const int64_t from_all = lo + wid * share, from = from_all < hi ? from_all : hi;
  const int64_t to = hi - from < share ? hi : from + share;
  // A wave's first places stay in registers; they and the counts are on their way
  // together.  Of the counts a thread adds up some workgroups' of an expert or two (where
  // experts are few, several threads share an expert's workgroups).
  constexpr int kHeld = 2;
  int32_t held[kHeld];
#pragma unroll
  for (int t = 0; t < kHeld; ++t) {
    const int64_t p = from + t * 64 + lane;
    held[t] = p < to ? listed_class(a, p, true) : -1;
  }
  int32_t width = 1;
  while (width < a.E) width *= 2;
  width = width < NT ? width : NT;
  int32_t seen[EPT], ahead_of[EPT];
#pragma unroll
  for (int u = 0; u < EPT; ++u) {
    const int32_t e = (tid & (width - 1)) + u * width;
    seen[u] = ahead_of[u] = 0;
    if (a.blocks > 1 && e < a.E) {
      const int32_t step = NT / width;
#pragma unroll 16
      for (int32_t b = tid / width; b < a.blocks; b += step) {
        const int32_t v = a.counts[b * a.E + e];
        seen[u] += v;
        ahead_of[u] += b < (int32_t)blockIdx.x ? v : 0;
      }
    }
  }
  for (int e = tid; e < a.E; e += NT) {
    for (int w = 0; w < W; ++w) next[w][e] = 0u;
    total_of[e] = before_of[e] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kHeld; ++t)
    if (held[t] >= 0) atomicAdd(&next[wid][held[t]], 1u);
  for (int64_t p = from + kHeld * 64 + lane; p < to; p += 64) {
    const int32_t c = listed_class(a, p, true);
    if (c >= 0) atomicAdd(&next[wid][c], 1u);
  }
#pragma unroll
  for (int u = 0; u < EPT; ++u) {
    const int32_t e = (tid & (width - 1)) + u * width;
    if (a.blocks > 1 && e < a.E) {
      atomicAdd(&total_of[e], seen[u]);
      atomicAdd(&before_of[e], ahead_of[u]);
    }
  }
  __syncthreads();
  int32_t all[EPT], before[EPT], sum = 0;
#pragma unroll
  for (int u = 0; u < EPT; ++u) {
    const int e = tid * EPT + u;
    all[u] = before[u] = 0;
    if (e < a.E) {
      if (a.blocks == 1) {
        for (int w = 0; w < W; ++w) all[u] += next[w][e];
      } else {
        all[u] = total_of[e];
        before[u] = before_of[e];
      }
    }
    sum += all[u];
  }
  int32_t total;
  int32_t at = block_exclusive_scan(sum, &total, sh);
#pragma unroll
  for (int u = 0; u < EPT; ++u) {
    const int e = tid * EPT + u;
    if (e < a.E) {
      if (blockIdx.x == 0) a.offsets[e] = at;
      int32_t pos = at + before[u];
      for (int w = 0; w < W; ++w) {
        const uint32_t c = next[w][e];
        next[w][e] = pos;
        pos += c;
      }
    }
    at += all[u];
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[a.E] = total;
  __syncthreads();
  int bits = 0;
  while (1 << bits < a.E) ++bits;
  auto put = [&](int64_t p, int32_t c) {  // 64 places, by a wave
    uint64_t same = __ballot(c >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(c >> b & 1);
      same &= c >> b & 1 ? set : ~set;
    }
    int32_t pos = -1;
    if (c >= 0) {
      const int ahead = __popcll(same & ((uint64_t(1) << lane) - 1));
      pos = (int32_t)next[wid][c] + ahead;
      a.order[pos] = (int32_t)p;
    }
    // (a wave's LDS accesses keep their order: all reads above come before this write)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (c >= 0 && lane == 63 - __clzll((long long)same)) next[wid][c] = (uint32_t)(pos + 1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (a.place != nullptr && p < to) a.place[p] = pos;
  };
#pragma unroll
  for (int t = 0; t < kHeld; ++t)
    if (from + t * 64 < to) put(from + t * 64 + lane, held[t]);
  for (int64_t p0 = from + kHeld * 64; p0 < to; p0 += 64)
    put(p0 + lane, p0 + lane < to ? listed_class(a, p0 + lane, false) : -1);
}

// -------------------------------------------------------------------- host --

// `launch` for all rows, kRows a workgroup.
template <int64_t kRows, typename Launch>
void each_grid(RouteArgs a, hipStream_t s, Launch launch) {
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid * kRows) {
    const int64_t left = (a.n - a.row0 + kRows - 1) / kRows;
    diag_begin(kDiagRoute, s);
    launch(dim3((unsigned)(left < kMaxRowGrid ? left : kMaxRowGrid)), a);
    diag_end(s);
  }
}

template <int DT, int NT, int EPL, bool BY_VALUE>
void launch_route(const RouteArgs& args, hipStream_t s) {
  each_grid<kRouteThreads / NT>(args, s, [s](dim3 grid, const RouteArgs& a) {
    hipLaunchKernelGGL((k_route<DT, NT, EPL, BY_VALUE>), grid, dim3(kRouteThreads), 0, s, a);
  });
}

template <int DT, int NT, int V>
void launch_route_grad(const RouteArgs& args, hipStream_t s) {
  each_grid<kRouteThreads / NT>(args, s, [s](dim3 grid, const RouteArgs& a) {
    hipLaunchKernelGGL((k_route_grad<DT, NT, V>), grid, dim3(kRouteThreads), 0, s, a);
  });
}

// Rows that all run at once get a wave each: fewer experts a lane, shorter rounds.
constexpr int64_t kRouteFewRows = 1024;

// The lanes of a row: as many as its experts need at EPL each, and at least one a
// group; a group has a power of two of them.
template <int NT, int EPL>
bool route_fits(RouteArgs& a) {
  int32_t log_lanes = 0, groups = 1;
  while (groups < a.groups) groups *= 2;
  if (groups > NT) return false;
  while (groups << (log_lanes + 1) <= NT) ++log_lanes;
  const int32_t lanes = 1 << log_lanes, per = (a.group_size + lanes - 1) / lanes;
  if (per > EPL) return false;
  a.log_lanes = log_lanes;
  a.per_lane = per;
  return true;
}

template <int DT, bool BY_VALUE>
int route_rows(RouteArgs a, hipStream_t s) {
  const bool few = a.n <= kRouteFewRows;
  if (few && route_fits<64, 4>(a)) {
    launch_route<DT, 64, 4, BY_VALUE>(a, s);
  } else if (!few && route_fits<4, 8>(a)) {
    launch_route<DT, 4, 8, BY_VALUE>(a, s);
  } else if (!few && route_fits<8, 8>(a)) {
    launch_route<DT, 8, 8, BY_VALUE>(a, s);
  } else if (!few && route_fits<16, 8>(a)) {
    launch_route<DT, 16, 8, BY_VALUE>(a, s);
  } else if (!few && route_fits<16, 16>(a)) {
    launch_route<DT, 16, 16, BY_VALUE>(a, s);
  } else if (!few && route_fits<32, 16>(a)) {
    launch_route<DT, 32, 16, BY_VALUE>(a, s);
  } else if (route_fits<64, 16>(a)) {
    launch_route<DT, 64, 16, BY_VALUE>(a, s);
  } else {
    // (3, 5, 9, 17, 33 and a few more groups leave lanes over; a lane then has up to 31 experts)
    route_fits<64, 32>(a);
    launch_route<DT, 64, 32, BY_VALUE>(a, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_route");
}

template <int DT>
int route_grad_rows(const RouteArgs& a, hipStream_t s) {
  constexpr int VE = Score<DT>::kVec;
  const int32_t vecs = (a.E + VE - 1) / VE;
  if (vecs <= 8) {
    launch_route_grad<DT, 8, 1>(a, s);
  } else if (vecs <= 16) {
    launch_route_grad<DT, 8, 2>(a, s);
  } else if (vecs <= 32) {
    launch_route_grad<DT, 8, 4>(a, s);
  } else if (vecs <= 64) {
    launch_route_grad<DT, 16, 4>(a, s);
  } else if (vecs <= 128) {
    launch_route_grad<DT, 32, 4>(a, s);
  } else {
    launch_route_grad<DT, 64, 4>(a, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_route_grad");
}

int check_routing(const gbdt_scores& x, const gbdt_routing* r) {
  if (!r) return fail(GBDT_E_ARG, "routing is null");
  if (x.n_classes > GBDT_MAX_EXPERTS) return fail(GBDT_E_UNSUPPORTED, "n_classes above GBDT_MAX_EXPERTS");
  if (r->score != GBDT_ROUTE_SOFTMAX && r->score != GBDT_ROUTE_SIGMOID)
    return fail(GBDT_E_ARG, "score is not a GBDT_ROUTE_*");
  if (!std::isfinite(r->scale)) return fail(GBDT_E_ARG, "scale must be finite");
  if (r->k < 1 || r->k > GBDT_MAX_ROUTED) return fail(GBDT_E_ARG, "k out of [1, GBDT_MAX_ROUTED]");
  if (r->n_groups < 1 || r->n_groups > GBDT_MAX_EXPERT_GROUPS)
    return fail(GBDT_E_ARG, "n_groups out of [1, GBDT_MAX_EXPERT_GROUPS]");
  if (r->groups_kept < 1 || r->groups_kept > r->n_groups) return fail(GBDT_E_ARG, "groups_kept out of [1, n_groups]");
  if (r->group_top != 1 && r->group_top != 2) return fail(GBDT_E_ARG, "group_top is not 1 or 2");
  if (x.n_classes % r->n_groups) return fail(GBDT_E_SHAPE, "n_groups does not divide n_classes");
  if (r->k > x.n_classes / r->n_groups * r->groups_kept)
    return fail(GBDT_E_SHAPE, "k above the experts of the kept groups");
  return GBDT_OK;
}

RouteArgs route_args(const gbdt_scores& x, const gbdt_routing& r, void* ws) {
  RouteArgs a = {};
  a.x = x.data;
  a.n = x.n_rows;
  a.ld = x.row_stride;
  a.E = x.n_classes;
  a.k = r.k;
  a.sigmoid = r.score == GBDT_ROUTE_SIGMOID;
  a.renorm = r.renormalise != 0;
  a.groups = r.n_groups;
  a.kept = r.groups_kept;
  a.top = r.group_top;
  a.group_size = x.n_classes / r.n_groups;
  a.scale = r.scale;
  a.err = &static_cast<WsCtrl*>(ws)->err;
  return a;
}

}  // namespace

}  // namespace gbdt

using namespace gbdt;

extern "C" {

int gbdt_route_classes(const gbdt_scores* x, const gbdt_routing* r, const float* bias, int32_t* classes,
                       float* weights, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_scores(x);
  if (!rc) rc = check_routing(*x, r);
  if (rc) return rc;
  if (x->n_rows == 0) return GBDT_OK;
  if (!classes || !weights) return fail(GBDT_E_ARG, "classes or weights is null");
  rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  RouteArgs a = route_args(*x, *r, ws);
  a.bias = bias;
  a.classes = classes;
  a.weights = weights;
  const bool by_value = bias != nullptr || (r->n_groups > 1 && r->group_top == 2);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (x->dtype) {
    case GBDT_DTYPE_F32:
      return by_value ? route_rows<GBDT_DTYPE_F32, true>(a, s) : route_rows<GBDT_DTYPE_F32, false>(a, s);
    case GBDT_DTYPE_BF16:
      return by_value ? route_rows<GBDT_DTYPE_BF16, true>(a, s) : route_rows<GBDT_DTYPE_BF16, false>(a, s);
    default: return by_value ? route_rows<GBDT_DTYPE_F16, true>(a, s) : route_rows<GBDT_DTYPE_F16, false>(a, s);
  }
}

int gbdt_route_grad(const gbdt_scores* x, const gbdt_routing* r, const int32_t* classes, const float* dweights,
                    void* grad, int64_t grad_stride, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_scores(x);
  if (!rc) rc = check_routing(*x, r);
  if (rc) return rc;
  if (x->n_rows == 0) return GBDT_OK;
  if (!classes || !dweights) return fail(GBDT_E_ARG, "classes or dweights is null");
  rc = check_grad(*x, grad, grad_stride);
  if (!rc) rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  RouteArgs a = route_args(*x, *r, ws);
  a.classes = const_cast<int32_t*>(classes);  // (read only)
  a.dweights = dweights;
  a.grad = grad;
  a.ldg = grad_stride;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (x->dtype) {
    case GBDT_DTYPE_F32: return route_grad_rows<GBDT_DTYPE_F32>(a, s);
    case GBDT_DTYPE_BF16: return route_grad_rows<GBDT_DTYPE_BF16>(a, s);
    default: return route_grad_rows<GBDT_DTYPE_F16>(a, s);
  }
}

int gbdt_route_lists(const int32_t* classes, int64_t n_places, int32_t n_experts, int32_t* offsets, int32_t* order,
                     int32_t* place, void* ws, size_t ws_bytes, void* stream) {
  if (n_places < 0 || n_places > INT32_MAX) return fail(GBDT_E_ARG, "n_places out of [0, 2^31)");
  if (n_experts < 1 || n_experts > GBDT_MAX_EXPERTS) return fail(GBDT_E_ARG, "n_experts out of [1, GBDT_MAX_EXPERTS]");
  if (!offsets) return fail(GBDT_E_ARG, "offsets is null");
  if (n_places > 0 && (!classes || !order)) return fail(GBDT_E_ARG, "classes or order is null");
  gbdt_scores x = {};
  x.n_classes = n_experts;
  const int rc = check_scores_ws(x, ws, ws_bytes);
  if (rc) return rc;
  ListArgs a = {};
  a.classes = classes;
  a.n = n_places;
  a.E = n_experts;
  a.counts = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + sizeof(WsCtrl));
  a.offsets = offsets;
  a.order = order;
  a.place = place;
  a.err = &static_cast<WsCtrl*>(ws)->err;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // Up to kAlone places one workgroup does it all (3,000 places of 64 and of 1,024 experts
  // alone 7.0 and 8.8 us, with counts 10.0 and 9.5; 6,000: 11.7 and 15.1, 9.1 and 10.7).
  // More go to workgroups of kChunk places or more (65,536 places of 64 and of 1,024
  // experts with 512, 1,024, 2,048 and 4,096: 9.5, 9.3, 10.0, 13.6 and 15.8, 12.5, 13.2,
  // 17.5 us), as many as the counts have room for.
  constexpr int64_t kAlone = 4096, kChunk = 1024, kMostBlocks = 256;
  static_assert(kMostBlocks * GBDT_MAX_EXPERTS * 4 <= kScoresPartBytes, "the counts fit the workspace");
  a.blocks = 1;
  a.chunk = n_places;
  if (n_places > kAlone) {
    a.chunk = (n_places + kMostBlocks - 1) / kMostBlocks;
    if (a.chunk < kChunk) a.chunk = kChunk;
    a.blocks = (int32_t)((n_places + a.chunk - 1) / a.chunk);
    diag_begin(kDiagRouteLists, s);
    hipLaunchKernelGGL(k_list_count, dim3(a.blocks), dim3(kCountThreads), 0, s, a);
    diag_end(s);
  }
  diag_begin(kDiagRouteLists, s);
  hipLaunchKernelGGL(k_list_place<512>, dim3(a.blocks), dim3(512), 0, s, a);
  diag_end(s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_list_place");
}

}  // extern "C"
