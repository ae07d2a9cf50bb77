// Distillation of a student's rows of class scores from a teacher's records
// (the listed classes with their scores, and the mass of the rest): the loss,
// its gradient, and both in one pass.
//
// With w_c = exp((x_c - m) / T), m = max x, S the listed classes,
// s_in = sum_S w, s_out = sum_{not S} w, s = s_in + s_out, e_j =
// exp((t_j - t_max) / T), z = sum e_j, r the rest and p_j = (1 - r) e_j / z:
//   loss / T^2 = sum_j p_j ((t_j - t_max) - (x_j - m)) / T
//                + (1 - r) log((1 - r) s / z) + r log(r s / s_out),
// which is sum p log(p / q) with the logarithms of the sums taken out: their
// arguments are near 1 when the student is near the teacher, so the loss keeps
// its digits where it is small.  s_out is kept as a sum against the largest
// score outside S, m_out (v_c = exp((x_c - m_out) / T), o = sum_{not S} v, which
// is at least 1): a student that is certain of a listed class has all others so
// far below m that their w underflow.  s_out = o exp((m_out - m) / T), and
//   log(r s / s_out) = log(r s / o) + (m - m_out) / T.
//   gradient: weight T (w_c / s - p_c) in S, weight T v_c (a / s - r / o) outside,
//   a = exp((m_out - m) / T): every factor is at most 1, whatever the gap.

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

// What a launch does: write the statistics, write the loss, write the gradient;
// of rows shared by several workgroups, write the part's sums or read them.
constexpr int kStats = 1, kLoss = 2, kGrad = 4, kPart = 8, kJoin = 16;

struct PartSum {
  double o;
  float m_out;
  uint32_t pad;
};

struct DistillArgs {
  const void* x;
  int64_t n, ld;
  int32_t C, k;
  const float* tv;
  const int32_t* tc;
  const float* tr;
  float T;
  double c, inv_T;  // log2(e) / T, 1 / T
  const float* weight;
  float* stats_out;
  const float* stats_in;
  float* loss;
  void* grad;
  int64_t ldg;
  int32_t* err;
  PartSum* parts;  // [n][n_joined]
  int32_t n_parts, part_len, n_joined;
  int64_t row0;  // of this launch
};

// The rest's mass of row i, clamped to [0, 1].
__device__ __forceinline__ double row_rest(const DistillArgs& a, int64_t i, bool report) {
  if (a.tr == nullptr) return 0.0;
  const float r = a.tr[i];
  if (r >= 0.0f && r <= 1.0f) return (double)r;
  if (report) dev_error(a.err, GBDT_E_RANGE);
  return r > 1.0f ? 1.0 : 0.0;
}

// The loss from the row's sums; kd = sum_j e_j ((t_j - t_max) - (x_j - m)),
// gap = m - m_out.
__device__ __forceinline__ double row_loss(double T, double inv_T, double r, double z, double kd, double s, double o,
                                           double gap) {
  double l = 0.0;
  if (r < 1.0) {
    const double iz = rcp_64(z);
    l += (1.0 - r) * (kd * iz * inv_T + log_64((1.0 - r) * s * iz));
  }
  if (r > 0.0) l += o == 0.0 ? __builtin_inf() : r * (log_64(r * s * rcp_64(o)) + gap * inv_T);
  return T * T * l;
}

// Statistics are FP32.  Below its normal numbers s_out has lost digits, or is 0:
// the gradient then takes m_out and o from the scores again.  Otherwise s_out =
// o 2^e with o in [1/2, 1) serves: v = w 2^-e = exp2((x - m) c + up), up = -e.
constexpr float kLeastStat = 0x1p-126f;
__device__ __forceinline__ void stat_sum(float s_out, double& o, float& up) {
  const uint32_t b = __float_as_uint(s_out);
  o = (double)__uint_as_float((b & 0x7fffffu) | 0x3f000000u);
  up = (float)(126 - (int32_t)(b >> 23));
}

// a / s - r / o = (s_out / s - r) / o; 0 without mass outside S.
__device__ __forceinline__ double outside_factor(double s_out_s, double r, double o) {
  return o > 0.0 ? (s_out_s - r) * rcp_64(o) : (o == 0.0 ? 0.0 : o);
}

// One thread per row of at most CMAX classes, R rows a workgroup; k <= C.  Rows,
// records and gradients pass through LDS, so that global memory sees whole
// lines (a thread's own row is a stride of 4 C bytes from its neighbours'), in
// rows of C | 1 words, which spreads the threads over the banks.  All loads are
// in flight at once: the rows are few microseconds in all, one memory latency
// each way.  The exponentials that the loss needs are in FP64 (a row's few
// terms do not average rounding errors away, and a small loss is what is left
// when terms of order 1 cancel).  Vector instructions bound it, about 940 a row
// of seven classes: step of 581,012 rows 23 us, 12 without its arithmetic.
template <int DT, int R, int CMAX, int MODE>
__global__ void __launch_bounds__(R, CMAX == 8 ? 1 : 4) k_distill_rows(const DistillArgs a) {
  using Elem = typename Score<DT>::Elem;
  extern __shared__ float lds[];
  const int tid = threadIdx.x;
  const int64_t i0 = int64_t(blockIdx.x) * R, i = i0 + tid;
  const int32_t rows = (int32_t)(a.n - i0 < R ? a.n - i0 : R);
  const int32_t C = a.C, k = a.k, P = C | 1, PK = k | 1;
  const RowDiv by_c(C), by_k(k);
  float* __restrict__ all_t = lds + R * P;
  int32_t* __restrict__ all_c = reinterpret_cast<int32_t*>(all_t + R * PK);
  const Elem* __restrict__ xg = static_cast<const Elem*>(a.x) + i0 * a.ld;
  {
    Staged<R, CMAX, float> xs, ts;
    Staged<R, CMAX, int32_t> cs;
    xs.load(
        rows, C, a.ld == C, by_c, [&](int32_t e) { return Score<DT>::to_f32(xg[(uint32_t)e]); },
        [&](int32_t row, int32_t c) { return Score<DT>::to_f32(xg[row * a.ld + c]); });
    const float* __restrict__ tg = a.tv + i0 * k;
    const int32_t* __restrict__ cg = a.tc + i0 * k;
    ts.load(rows, k, true, by_k, [&](int32_t e) { return tg[(uint32_t)e]; }, [](int32_t, int32_t) { return 0.0f; });
    cs.load(rows, k, true, by_k, [&](int32_t e) { return cg[(uint32_t)e]; }, [](int32_t, int32_t) { return 0; });
    ts.put(rows, k, by_k, all_t);
    cs.put(rows, k, by_k, all_c);
    xs.put(rows, C, by_c, lds);
  }
  const bool mine = tid < rows;
  const double r = mine ? row_rest(a, i, true) : 0.0;
  float wt = 1.0f, m = -kInf, m_out = -kInf, tm = -kInf;
  double s_in = 0.0, s_out = 0.0, o = 0.0;
  if (mine && (MODE & kGrad) && a.weight != nullptr) wt = a.weight[i];
  if (mine && !(MODE & kStats)) {
    m = a.stats_in[3 * i];
    s_in = a.stats_in[3 * i + 1];
    s_out = a.stats_in[3 * i + 2];
  }
  __syncthreads();
  float* __restrict__ x = lds + tid * P;
  float* __restrict__ tv = all_t + tid * PK;
  const int32_t* __restrict__ tc = all_c + tid * PK;
  if (mine) {
    uint32_t in_s = 0u;
    bool has = false;
    for (int32_t j = 0; j < k; ++j) {
      const int32_t cls = tc[j];
      if (cls < 0) continue;
      if (cls >= C) {
        dev_error(a.err, GBDT_E_RANGE);
        continue;
      }
      if (in_s >> cls & 1u) dev_error(a.err, GBDT_E_ARG);
      in_s |= 1u << cls;
      const float t = tv[j];
      tm = __builtin_fmaxf(tm, t);
      has = has || !(t == -kInf);
    }
    if (MODE & kStats) {
#pragma unroll
      for (int c = 0; c < CMAX; ++c) {
        if (c < C) {
          m = __builtin_fmaxf(m, x[c]);
          m_out = in_s >> c & 1u ? m_out : __builtin_fmaxf(m_out, x[c]);
        }
      }
    }
    const double ms = m == -kInf ? 0.0 : (double)m;
    double mos = m_out == -kInf ? 0.0 : (double)m_out;
    const double ts = tm == -kInf ? 0.0 : (double)tm;
    double z = 0.0, kd = 0.0;
    for (int32_t j = 0; j < k; ++j) {
      const int32_t cls = tc[j];
      if (cls < 0 || cls >= C) continue;
      const double d = (double)tv[j] - ts;
      const double e = exp2_64(d * a.c);
      z += e;
      if ((MODE & kLoss) && !(e == 0.0)) kd += e * (d - ((double)x[cls] - ms));
      if (MODE & kGrad) tv[j] = (float)e;
    }
    if (MODE & kStats) {
      const double of_m = exp2_64(((double)m_out - ms) * a.c);  // w / v
#pragma unroll
      for (int c = 0; c < CMAX; ++c) {
        if (c < C) {
          const bool in = in_s >> c & 1u;
          const double w = exp2_64(((double)x[c] - (in ? ms : mos)) * a.c);
          if (in) s_in += w; else o += w;
          if (MODE & kGrad) x[c] = (float)w;
        }
      }
      s_out = o * of_m;
    }
    const double s = s_in + s_out;
    const bool live = has && !(s == 0.0);
    if ((MODE & kStats) && a.stats_out != nullptr) {
      a.stats_out[3 * i] = m;
      a.stats_out[3 * i + 1] = (float)s_in;
      a.stats_out[3 * i + 2] = (float)s_out;
    }
    if (MODE & kLoss) a.loss[i] = live ? (float)row_loss(a.T, a.inv_T, r, z, kd, s, o, ms - mos) : 0.0f;
    if (MODE & kGrad) {
      const bool counts = live && !(wt == 0.0f);
      const double g = (double)wt * (double)a.T;
      const double inv = rcp_64(s);
      float up = 0.0f;  // v = exp2((x - m_out) c + up)
      if (!(MODE & kStats)) {
        if (r > 0.0 && (float)s_out < kLeastStat) {
#pragma unroll 1
          for (int c = 0; c < C; ++c) m_out = in_s >> c & 1u ? m_out : __builtin_fmaxf(m_out, x[c]);
          mos = m_out == -kInf ? 0.0 : (double)m_out;
#pragma unroll 1
          for (int c = 0; c < C; ++c) o += in_s >> c & 1u ? 0.0 : exp2_64(((double)x[c] - mos) * a.c);
        } else {
          stat_sum((float)s_out, o, up);
          mos = ms;
        }
      }
      const float in = (float)inv, out = (float)(g * outside_factor(s_out * inv, r, o));
      const float cf = exponent_scale(a.c), mf = (float)ms, mof = (float)mos;
#pragma unroll
      for (int c = 0; c < CMAX; ++c) {
        if (c < C) {
          const bool in_c = in_s >> c & 1u;
          const float w = MODE & kStats
                              ? x[c]
                              : exp2_32(__builtin_fmaf(x[c] - (in_c ? mf : mof), cf, in_c ? 0.0f : up));
          x[c] = counts ? w * (in_c ? in : out) : 0.0f;
        }
      }
      if (counts) {
        const double pz = (1.0 - r) * rcp_64(z);
        for (int32_t j = 0; j < k; ++j) {
          const int32_t cls = tc[j];
          if (cls < 0 || cls >= C) continue;
          x[cls] = (float)(g * ((double)x[cls] - (double)tv[j] * pz));
        }
      }
    }
  }
  if (MODE & kGrad) {
    __syncthreads();
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i0 * a.ldg;
    unstage<R, CMAX>(
        rows, C, a.ldg == C, by_c, lds, [&](int32_t e, float v) { gr[(uint32_t)e] = Score<DT>::from_f32(v); },
        [&](int32_t row, int32_t c, float v) { gr[row * a.ldg + c] = Score<DT>::from_f32(v); });
  }
}

// One workgroup per row, or per part of one: `part_len` classes (a multiple of
// NT * kBlk) of a row that n_parts workgroups share; a first launch (kPart)
// leaves each part's sums, a second (kJoin) adds them up.
//
// Memory bounds it where rows are many: step of 4,096 x 131,072 bf16 443 us
// (4.9 TB/s of what has to move; the second read of the scores comes from the
// last-level cache), gradient of 2,048 x 50,001 f32 152 us (5.4 TB/s).
//
// One pass takes the sum outside S against a reference that is the first
// maximum the thread meets there and moves only when a score is above it by
// 2^20 in the exponential, so a vector costs no rescaling; the second writes the
// gradient.
// LDS: a bit per class (set: listed), laid out so that a thread's part of a
// block is one word (or half of one).  Thread j of the first k owns entry j
// (and j + NT, ...) of the record; its class's gradient replaces, behind a
// barrier, what the vector stores left there.
//
// With fewer than 64 threads a row, a wave holds several rows (the last one's
// spare threads do the last row again): step of 300,000 rows of 100 bf16 152
// us, 520 with a wave each.
//
// A gradient from statistics reads a row three times where the sum outside has
// to be taken again: 2,048 x 50,001 f32 with all rows 200 T apart 262 us, 168
// with none.
constexpr int kNarrowThreads = 16, kNarrowClasses = 256, kNarrowListed = 64;

template <int DT, int NT, int MODE>
__global__ void __launch_bounds__(NT < 64 ? 64 : NT, NT <= 64 ? 6 : 8) k_distill_block(const DistillArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec, BLK = kBlk<DT>, W = NT < 64 ? 1 : NT / 64;
  constexpr int KPT = NT < 64 ? kNarrowListed / NT : (GBDT_MAX_LISTED + NT - 1) / NT;
  constexpr bool kSums = (MODE & kStats) && !(MODE & kJoin);
  extern __shared__ uint32_t all_bits[];
  __shared__ float sh_m[W], sh_o[W], sh_t[W];
  __shared__ double sh_d[4][W];
  const int tid = threadIdx.x & (NT - 1), wid = threadIdx.x >> 6;
  const int sub = NT < 64 ? threadIdx.x / NT : 0;  // the row's place in the wave
  const float cf = exponent_scale(a.c);
  const uint32_t in_launch = a.n_parts > 1 ? blockIdx.x / (uint32_t)a.n_parts : blockIdx.x;
  const int32_t part = (int32_t)(blockIdx.x - in_launch * (uint32_t)a.n_parts);
  const int64_t i_all = NT < 64 ? a.row0 + int64_t(in_launch) * (64 / NT) + sub : a.row0 + in_launch;
  const int64_t i = NT < 64 && i_all >= a.n ? a.n - 1 : i_all;
  const int32_t lo = part * a.part_len;
  const int32_t hi = a.C - lo < a.part_len ? a.C : lo + a.part_len;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  RawBlock<DT> raw;
  if (kSums) raw = load_block<DT, NT>(xr, lo, hi);
  const int32_t words = ((hi - lo + NT * BLK - 1) / (NT * BLK) * BLK + 31) / 32 * NT;
  uint32_t* __restrict__ bits = all_bits + sub * words;
  for (int32_t w = tid; w < words; w += NT) bits[w] = 0u;
  const double r = row_rest(a, i, tid == 0);
  const float wt = (MODE & kGrad) && a.weight != nullptr ? a.weight[i] : 1.0f;
  int32_t cls[KPT];
  float t[KPT], xj[KPT];
#pragma unroll
  for (int u = 0; u < KPT; ++u) {
    const int32_t j = tid + u * NT;
    cls[u] = -1;
    t[u] = -kInf;
    xj[u] = -kInf;
    if (j < a.k) {
      cls[u] = a.tc[i * a.k + j];
      if (cls[u] >= a.C) {
        dev_error(a.err, GBDT_E_RANGE);
        cls[u] = -1;
      }
      if (cls[u] >= 0) {
        t[u] = a.tv[i * a.k + j];
        xj[u] = Score<DT>::to_f32(xr[cls[u]]);
      }
    }
  }
  __syncthreads();
  // the bits of the record's classes in [from, to)
  auto mark_listed = [&](int32_t from, int32_t to) {
#pragma unroll
    for (int u = 0; u < KPT; ++u) {
      if (cls[u] >= from && cls[u] < to) {
        // (block, vector, thread, element) of the class
        const int32_t e = cls[u] - from, in = e % (NT * BLK), blk = e / (NT * BLK);
        const int32_t bit = blk * BLK % 32 + in / (NT * VE) * VE + in % VE;
        const int32_t word = blk * BLK / 32 * NT + in / VE % NT;
        if (atomicOr(&bits[word], 1u << bit) >> bit & 1u) dev_error(a.err, GBDT_E_ARG);
      }
    }
  };
  mark_listed(lo, hi);
  float tm = -kInf;
  bool has = false;
#pragma unroll
  for (int u = 0; u < KPT; ++u) {
    tm = __builtin_fmaxf(tm, t[u]);
    has = has || !(t[u] == -kInf);
  }
  __syncthreads();
  float m = -kInf, m_out = -kInf, ref = -kInf;
  double o = 0.0;
  // of a gradient from statistics: v = exp2((x - mf) c + up), and its sum
  float mf = 0.0f, up = 0.0f;
  double s_in = 0.0, s_out = 0.0, o_stat = 0.0;
  if (kSums) {
    for (int32_t base = lo, b = 0;; b += BLK) {
      const uint32_t in_s = bits[(b / 32) * NT + tid] >> (b % 32);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float f[VE];
        unpack<DT>(raw.v[j], f);
        const uint32_t in_v = in_s >> (j * VE) & ((1u << VE) - 1u);
        if (in_v) {
#pragma unroll
          for (int q = 0; q < VE; ++q) f[q] = in_v >> q & 1u ? -kInf : f[q];
        }
        const float vm = max_of(f);
        m_out = __builtin_fmaxf(m_out, vm);
        if ((vm - ref) * cf > 20.0f) {  // (the first finite score among them)
          o *= exp2_64(((double)ref - (double)vm) * a.c);
          ref = vm;
        }
        const float rf = ref == -kInf ? 0.0f : ref;
#pragma unroll
        for (int q = 0; q < VE; ++q) f[q] = exp2_32((f[q] - rf) * cf);
        o += (double)sum_of(f);
        __builtin_amdgcn_sched_barrier(0);  // (vector by vector: fewer registers)
      }
      base += NT * BLK;
      if (base >= hi) break;
      raw = load_block<DT, NT>(xr, base, hi);
    }
  } else if (MODE & kJoin) {
    if (tid < a.n_joined) {
      const PartSum p = a.parts[i * a.n_joined + tid];
      m_out = ref = p.m_out;
      o = p.o;
    }
  } else {
    s_in = a.stats_in[3 * i + 1];
    s_out = a.stats_in[3 * i + 2];
    m = a.stats_in[3 * i];
    stat_sum((float)s_out, o_stat, up);
    mf = m;
    const bool lost = r > 0.0 && !(wt == 0.0f) && (float)s_out < kLeastStat;
    if (NT <= 64 ? __any(lost) : lost) {
      // All threads of a row, and all rows of a wave, come here together; a part
      // at a time, as the bits have room for one; vector by vector: few registers
      // for what few rows need.
      double again = 0.0, mos = 0.0;
      for (int pass = 0; pass < 2; ++pass) {
        for (int32_t from = 0; from < a.C; from += a.part_len) {
          const int32_t to = a.C - from < a.part_len ? a.C : from + a.part_len;
          __syncthreads();
          for (int32_t w = tid; w < (a.part_len / (NT * BLK) * BLK + 31) / 32 * NT; w += NT) bits[w] = 0u;
          __syncthreads();
          mark_listed(from, to);
          __syncthreads();
#pragma unroll 1
          for (int32_t c = from + tid * VE, b = 0; c - tid * VE < to; c += NT * VE, b += VE) {
            float f[VE];
            load_chunk<DT>(xr, c, to, f);
            const uint32_t in_v = bits[b / 32 * NT + tid] >> b % 32 & ((1u << VE) - 1u);
#pragma unroll
            for (int q = 0; q < VE; ++q) f[q] = in_v >> q & 1u ? -kInf : f[q];
            if (pass == 0) {
              m_out = __builtin_fmaxf(m_out, max_of(f));
            } else {
#pragma unroll
              for (int q = 0; q < VE; ++q) again += exp2_64(((double)f[q] - mos) * a.c);
            }
          }
        }
        if (pass == 0) {
          m_out = NT <= 64 ? group_max<NT>(m_out) : block_max<NT>(m_out, sh_o);
          mos = m_out == -kInf ? 0.0 : (double)m_out;
        }
      }
      again = NT <= 64 ? group_sum<NT>(again) : block_sum<NT>(again, sh_d[0]);
      if (lost) {
        o_stat = again;
        up = 0.0f;
        mf = (float)mos;
      }
    }
  }
  // the row's maxima; NaN in the record counts as an entry
  if (MODE & kStats) {
#pragma unroll
    for (int u = 0; u < KPT; ++u) m = __builtin_fmaxf(m, xj[u]);
    m = group_max<NT>(__builtin_fmaxf(m, m_out));
    m_out = group_max<NT>(m_out);
  }
  tm = group_max<NT>(tm);
  if (NT <= 64) {
    has = (__ballot(has) >> (sub * NT) & (~uint64_t(0) >> (64 - (NT < 64 ? NT : 64)))) != 0;
  } else {
    if ((tid & 63) == 0) {
      if (MODE & kStats) {
        sh_m[wid] = m;
        sh_o[wid] = m_out;
      }
      sh_t[wid] = tm;
    }
    has = __syncthreads_or(has);
    if (MODE & kStats) {
      m = across_waves<W>(sh_m, [](float u, float v) { return __builtin_fmaxf(u, v); });
      m_out = across_waves<W>(sh_o, [](float u, float v) { return __builtin_fmaxf(u, v); });
    }
    tm = across_waves<W>(sh_t, [](float u, float v) { return __builtin_fmaxf(u, v); });
  }
  const double ms = m == -kInf ? 0.0 : (double)m;
  const double mos = m_out == -kInf ? 0.0 : (double)m_out;
  const double ts = tm == -kInf ? 0.0 : (double)tm;
  if ((MODE & kStats) && ref != m_out) o *= exp2_64(((double)ref - mos) * a.c);
  if constexpr ((MODE & kPart) != 0) {
    o = block_sum<NT>(o, sh_d[0]);
    if (tid == 0) a.parts[i * a.n_parts + part] = PartSum{o, m_out, 0u};
    return;
  }
  double e[KPT], wj[KPT], z = 0.0, kd = 0.0, si = 0.0;
#pragma unroll
  for (int u = 0; u < KPT; ++u) {
    const double d = (double)t[u] - ts, dx = (double)xj[u] - ms;
    e[u] = exp2_64(d * a.c);
    wj[u] = exp2_64(dx * a.c);
    z += e[u];
    if (!(e[u] == 0.0)) kd += e[u] * (d - dx);
    si += wj[u];
  }
  double sum[4] = {z, kd, si, o};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    sum[v] = group_sum<NT>(sum[v]);
    if (NT > 64 && (tid & 63) == 0) sh_d[v][wid] = sum[v];
  }
  if (NT > 64) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v) sum[v] = across_waves<W>(sh_d[v], [](double p, double q) { return p + q; });
  }
  z = sum[0];
  kd = sum[1];
  if (MODE & kStats) {
    o = sum[3];
    s_in = sum[2];
    s_out = o * exp2_64(((double)m_out - ms) * a.c);
    mf = (float)mos;
  } else {
    o = o_stat;
  }
  const double s = s_in + s_out;
  const bool live = has && !(s == 0.0);
  if (tid == 0 && part == 0) {
    if ((MODE & kStats) && a.stats_out != nullptr) {
      a.stats_out[3 * i] = m;
      a.stats_out[3 * i + 1] = (float)s_in;
      a.stats_out[3 * i + 2] = (float)s_out;
    }
    if (MODE & kLoss) a.loss[i] = live ? (float)row_loss(a.T, a.inv_T, r, z, kd, s, o, ms - mos) : 0.0f;
  }
  if (MODE & kGrad) {
    const bool counts = live && !(wt == 0.0f);
    const double g = (double)wt * (double)a.T;
    const double inv = rcp_64(s);
    const float scale = (float)(g * outside_factor(s_out * inv, r, o));
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
    for (int32_t base = lo; base < hi; base += NT * BLK) {
      RawBlock<DT> out;
      if (counts) {
        raw = load_block<DT, NT>(xr, base, hi);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[VE];
          unpack<DT>(raw.v[j], f);
#pragma unroll
          for (int q = 0; q < VE; ++q)
            f[q] = exp2_32(MODE & kStats ? (f[q] - mf) * cf : __builtin_fmaf(f[q] - mf, cf, up)) * scale;
          out.v[j] = pack<DT>(f);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        out = RawBlock<DT>{};
      }
      store_block<DT, NT>(gr, base, hi, out);
    }
    __syncthreads();
    if (counts) {
#pragma unroll
      for (int u = 0; u < KPT; ++u)
        if (cls[u] >= lo && cls[u] < hi)
          gr[cls[u]] = Score<DT>::from_f32((float)(g * (wj[u] * inv - e[u] * ((1.0 - r) * rcp_64(z)))));
    }
  }
}

template <int DT, int R, int CMAX, int MODE>
void launch_rows(const DistillArgs& a, hipStream_t s) {
  const size_t lds = size_t(R) * 4 * ((a.C | 1) + 2 * (a.k | 1));
  const dim3 grid((unsigned)((a.n + R - 1) / R));
  diag_begin(kDiagDistill, s);
  hipLaunchKernelGGL((k_distill_rows<DT, R, CMAX, MODE>), grid, dim3(R), lds, s, a);
  diag_end(s);
}

template <int DT, int NT, int MODE>
void launch_block(DistillArgs a, hipStream_t s) {
  constexpr int32_t kStep = NT * kBlk<DT>;
  if (a.n_parts == 1) a.part_len = (a.C + kStep - 1) / kStep * kStep;
  constexpr int kRows = NT < 64 ? 64 / NT : 1;  // of a workgroup
  const size_t lds = size_t((a.part_len / kStep * kBlk<DT> + 31) / 32) * NT * 4 * kRows;
  for (a.row0 = 0; a.row0 < a.n; a.row0 += kMaxRowGrid) {
    const int64_t n = a.n - a.row0 < kMaxRowGrid ? a.n - a.row0 : kMaxRowGrid;
    diag_begin(kDiagDistill, s);
    hipLaunchKernelGGL((k_distill_block<DT, NT, MODE>), dim3((unsigned)((n + kRows - 1) / kRows * a.n_parts)),
                       dim3(kRows * NT), lds, s, a);
    diag_end(s);
  }
}

// Threads for a row: a wave up to 2,048 classes (no barrier waits for others),
// 1,024 threads where a row is long enough to be read twice from memory: then
// fewer rows are between their two reads at a time, and more of them are still
// in the last-level cache (step, 4,096 x 131,072 bf16: 445 us with 1,024
// threads, 485 with 512, 578 with 256; grad, 2,048 x 50,001 f32: 155, 163, 166;
// the loss alone, which reads once, 2,048 x 131,072 bf16: 105, 100, 101).
// In between 256: more rows side by side hide the rows' own latencies (loss,
// 1,000 x 32,003 f16: 21 us with 256 threads, 23 with 512, 35 with 1,024).
// Few rows are split: 1 x 131,072 f32 takes 13 us with 32 workgroups and 28 with
// one, 64 rows bf16 19 and 27; at 128 rows both take 28.
template <int DT, int MODE>
int launch_distill(const DistillArgs& args, hipStream_t s) {
  DistillArgs a = args;
  a.n_parts = a.n_joined = 1;
  a.part_len = 0;
  constexpr int32_t kPartStep = 256 * kBlk<DT>;
  const int32_t steps = (a.C + kPartStep - 1) / kPartStep;
  const bool short_rows = a.C <= kRowsMaxClasses && a.k <= a.C;
  if (short_rows && a.C <= 8) {
    launch_rows<DT, 64, 8, MODE>(a, s);
  } else if (short_rows && a.C <= 16) {
    launch_rows<DT, 128, 16, MODE>(a, s);
  } else if (short_rows) {
    launch_rows<DT, 64, 32, MODE>(a, s);
  } else if (a.n <= kSplitRows && steps >= 4) {
    const int32_t want = (int32_t)(kSplitGrid / a.n);
    const int32_t per = (steps + want - 1) / want;
    const int32_t parts = (steps + per - 1) / per;
    a.part_len = per * kPartStep;
    a.n_parts = a.n_joined = parts;
    if constexpr ((MODE & kStats) != 0) {
      launch_block<DT, 256, kStats | kPart>(a, s);
      if (!(MODE & kGrad)) a.n_parts = 1;
      launch_block<DT, 256, MODE | kJoin>(a, s);
    } else {
      launch_block<DT, 256, MODE>(a, s);
    }
  } else if (a.C <= kNarrowClasses && a.k <= kNarrowListed) {
    launch_block<DT, kNarrowThreads, MODE>(a, s);
  } else if (a.C <= 2048) {
    launch_block<DT, 64, MODE>(a, s);
  } else if (a.C <= 40000) {
    launch_block<DT, 256, MODE>(a, s);
  } else {
    launch_block<DT, 1024, MODE>(a, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GBDT_OK : hip_fail(e, "k_distill");
}

template <int MODE>
int distill(const gbdt_scores* x, const gbdt_teacher* t, float temperature, const float* stats_in,
            const float* weight, float* loss, float* stats_out, void* grad, int64_t grad_stride, void* ws,
            size_t ws_bytes, hipStream_t s) {
  int rc = check_scores(x);
  if (rc) return rc;
  if (!t) return fail(GBDT_E_ARG, "teacher is null");
  if (t->k < 1 || t->k > GBDT_MAX_LISTED) return fail(GBDT_E_ARG, "teacher k out of [1, GBDT_MAX_LISTED]");
  if (!std::isfinite(temperature) || !(temperature > 0.0f))
    return fail(GBDT_E_ARG, "temperature must be finite and > 0");
  if (x->n_rows == 0) return GBDT_OK;
  if (!t->values || !t->classes) return fail(GBDT_E_ARG, "teacher values or classes is null");
  if ((MODE & kLoss) && !loss) return fail(GBDT_E_ARG, "loss is null");
  if (MODE == (kStats | kLoss) && !stats_out) return fail(GBDT_E_ARG, "stats is null");
  if (!(MODE & kStats) && !stats_in) return fail(GBDT_E_ARG, "stats is null");
  if (MODE & kGrad) rc = check_grad(*x, grad, grad_stride);
  if (!rc) rc = check_scores_ws(*x, ws, ws_bytes);
  if (rc) return rc;
  DistillArgs a;
  a.x = x->data;
  a.n = x->n_rows;
  a.ld = x->row_stride;
  a.C = x->n_classes;
  a.k = t->k;
  a.tv = t->values;
  a.tc = t->classes;
  a.tr = t->rest;
  a.T = temperature;
  a.c = kLog2e / (double)temperature;
  a.inv_T = 1.0 / (double)temperature;
  a.weight = weight;
  a.stats_out = stats_out;
  a.stats_in = stats_in;
  a.loss = loss;
  a.grad = grad;
  a.ldg = grad_stride;
  a.parts = reinterpret_cast<PartSum*>(static_cast<char*>(ws) + sizeof(WsCtrl));
  a.err = &static_cast<WsCtrl*>(ws)->err;
  switch (x->dtype) {
    case GBDT_DTYPE_F32: return launch_distill<GBDT_DTYPE_F32, MODE>(a, s);
    case GBDT_DTYPE_BF16: return launch_distill<GBDT_DTYPE_BF16, MODE>(a, s);
    default: return launch_distill<GBDT_DTYPE_F16, MODE>(a, s);
  }
}

}  // namespace

int check_scores(const gbdt_scores* x) {
  if (!x) return fail(GBDT_E_ARG, "scores is null");
  if (x->dtype != GBDT_DTYPE_F32 && x->dtype != GBDT_DTYPE_BF16 && x->dtype != GBDT_DTYPE_F16)
    return fail(GBDT_E_ARG, "dtype is not a GBDT_DTYPE_*");
  if (x->n_rows < 0 || x->n_rows > (int64_t(1) << 31)) return fail(GBDT_E_ARG, "n_rows out of [0, 2^31]");
  if (x->n_classes < 1 || x->n_classes > GBDT_MAX_CLASSES)
    return fail(GBDT_E_ARG, "n_classes out of [1, GBDT_MAX_CLASSES]");
  if (x->n_rows > 1 && x->row_stride < x->n_classes)
    return fail(GBDT_E_SHAPE, "row_stride smaller than n_classes");
  if (x->n_rows > 0) {
    if (!x->data) return fail(GBDT_E_ARG, "scores data is null");
    if (reinterpret_cast<uintptr_t>(x->data) % (x->dtype == GBDT_DTYPE_F32 ? 4 : 2))
      return fail(GBDT_E_ARG, "scores data is misaligned");
  }
  return GBDT_OK;
}

int check_scores_ws(const gbdt_scores& x, const void* ws, size_t ws_bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return fail(GBDT_E_ARG, "workspace is null or misaligned");
  if (ws_bytes < gbdt_scores_workspace_bytes(x.n_rows, x.n_classes))
    return fail(GBDT_E_ARG, "workspace smaller than gbdt_scores_workspace_bytes()");
  return GBDT_OK;
}

}  // namespace gbdt

using namespace gbdt;

extern "C" {

size_t gbdt_scores_workspace_bytes(int64_t n_rows, int32_t n_classes) {
  if (n_rows < 0 || n_rows > (int64_t(1) << 31) || n_classes < 1 || n_classes > GBDT_MAX_CLASSES) return 0;
  return sizeof(WsCtrl) + kScoresPartBytes;
}

int gbdt_distill_loss(const gbdt_scores* x, const gbdt_teacher* t, float temperature, float* loss,
                      float* stats, void* ws, size_t ws_bytes, void* stream) {
  return distill<kStats | kLoss>(x, t, temperature, nullptr, nullptr, loss, stats, nullptr, 0, ws, ws_bytes,
                                 reinterpret_cast<hipStream_t>(stream));
}

int gbdt_distill_grad(const gbdt_scores* x, const gbdt_teacher* t, float temperature, const float* stats,
                      const float* weight, void* grad, int64_t grad_stride, void* ws, size_t ws_bytes,
                      void* stream) {
  return distill<kGrad>(x, t, temperature, stats, weight, nullptr, nullptr, grad, grad_stride, ws, ws_bytes,
                        reinterpret_cast<hipStream_t>(stream));
}

int gbdt_distill_step(const gbdt_scores* x, const gbdt_teacher* t, float temperature, const float* weight,
                      float* loss, void* grad, int64_t grad_stride, void* ws, size_t ws_bytes, void* stream) {
  return distill<kStats | kLoss | kGrad>(x, t, temperature, nullptr, weight, loss, nullptr, grad, grad_stride,
                                         ws, ws_bytes, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
