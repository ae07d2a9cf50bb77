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
// its digits where it is small.
//   gradient: weight T (w_c / s - p_c) in S, weight T (w_c / s)(1 - r s / s_out)
//   outside.

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

// What a launch does: write the statistics, write the loss, write the gradient.
constexpr int kStats = 1, kLoss = 2, kGrad = 4;

struct DistillArgs {
  const void* x;
  int64_t n, ld;
  int32_t C, k;
  const float* tv;
  const int32_t* tc;
  const float* tr;
  float T;
  double c;  // log2(e) / T
  const float* weight;
  float* stats_out;
  const float* stats_in;
  float* loss;
  void* grad;
  int64_t ldg;
  int32_t* err;
};

// The rest's mass of row i, clamped to [0, 1].
__device__ __forceinline__ double row_rest(const DistillArgs& a, int64_t i, bool report) {
  if (a.tr == nullptr) return 0.0;
  const float r = a.tr[i];
  if (r >= 0.0f && r <= 1.0f) return (double)r;
  if (report) dev_error(a.err, GBDT_E_RANGE);
  return r > 1.0f ? 1.0 : 0.0;
}

// The loss from the row's sums; k_sum = sum_j p_j ((t_j - t_max) - (x_j - m)).
__device__ __forceinline__ double row_loss(double T, double r, double z, double k_sum, double s_in,
                                           double s_out) {
  const double s = s_in + s_out;
  double l = k_sum / T;
  if (r < 1.0) l += (1.0 - r) * log((1.0 - r) * s / z);
  if (r > 0.0) l += r * log(r * s / s_out);
  return T * T * l;
}

// One thread per row of at most CMAX classes; every exponential in FP64 (a
// row's few terms do not average rounding errors away, and a small loss is
// what is left when terms of order 1 cancel).
template <int DT, int CMAX, int MODE>
__global__ void __launch_bounds__(256) k_distill_rows(const DistillArgs a) {
  using Elem = typename Score<DT>::Elem;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.n) return;
  const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
  float x[CMAX], t[CMAX];
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    x[c] = c < a.C ? Score<DT>::to_f32(xr[c]) : -kInf;
    t[c] = -kInf;
  }
  uint32_t in_s = 0u;
  for (int32_t j = 0; j < a.k; ++j) {
    const int32_t cls = a.tc[i * a.k + j];
    if (cls < 0) continue;
    if (cls >= a.C) {
      dev_error(a.err, GBDT_E_RANGE);
      continue;
    }
    if (in_s >> cls & 1u) dev_error(a.err, GBDT_E_ARG);
    in_s |= 1u << cls;
    const float tv = a.tv[i * a.k + j];
#pragma unroll
    for (int c = 0; c < CMAX; ++c) t[c] = c == cls ? tv : t[c];
  }
  const double r = row_rest(a, i, true);
  float m = -kInf, tm = -kInf;
  bool has = false;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    m = __builtin_fmaxf(m, x[c]);
    tm = __builtin_fmaxf(tm, t[c]);
    has = has || !(t[c] == -kInf);
  }
  if (!(MODE & kStats)) m = a.stats_in[3 * i];
  const double ms = m == -kInf ? 0.0 : (double)m;
  const double ts = tm == -kInf ? 0.0 : (double)tm;
  double w[CMAX], p[CMAX], z = 0.0, s_in = 0.0, s_out = 0.0;
#pragma unroll
  for (int c = 0; c < CMAX; ++c) {
    w[c] = exp2_64(((double)x[c] - ms) * a.c);
    p[c] = exp2_64(((double)t[c] - ts) * a.c);
    z += p[c];
    if (in_s >> c & 1u) s_in += w[c]; else s_out += w[c];
  }
  if (!(MODE & kStats)) {
    s_in = a.stats_in[3 * i + 1];
    s_out = a.stats_in[3 * i + 2];
  }
  const double s = s_in + s_out;
  const bool live = has && !(s == 0.0);
  const double pz = live ? (1.0 - r) / z : 0.0;
  if ((MODE & kStats) && a.stats_out != nullptr) {
    a.stats_out[3 * i] = m;
    a.stats_out[3 * i + 1] = (float)s_in;
    a.stats_out[3 * i + 2] = (float)s_out;
  }
  if (MODE & kLoss) {
    double k_sum = 0.0;
#pragma unroll
    for (int c = 0; c < CMAX; ++c) {
      const double pc = p[c] * pz;
      if (!(pc == 0.0)) k_sum += pc * (((double)t[c] - ts) - ((double)x[c] - ms));
    }
    a.loss[i] = live ? (float)row_loss(a.T, r, z, k_sum, s_in, s_out) : 0.0f;
  }
  if (MODE & kGrad) {
    const float wt = a.weight != nullptr ? a.weight[i] : 1.0f;
    const bool counts = live && !(wt == 0.0f);
    const double g = (double)wt * (double)a.T;
    const double inv = 1.0 / s;
    const double share = s_out > 0.0 ? 1.0 - r * s / s_out : (s_out == 0.0 ? 0.0 : s_out);
    Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
#pragma unroll
    for (int c = 0; c < CMAX; ++c) {
      const double q = w[c] * inv;
      const double d = (in_s >> c & 1u) ? q - p[c] * pz : q * share;
      if (c < a.C) gr[c] = Score<DT>::from_f32(counts ? (float)(g * d) : 0.0f);
    }
  }
}

// One workgroup per row.  LDS: a bit per class (set: listed).  Thread j < k
// owns entry j of the record: its class's gradient is its to write, and the
// vector stores leave the listed classes out, so no element is written twice.
template <int DT, int NT, int MODE>
__global__ void __launch_bounds__(NT) k_distill_block(const DistillArgs a) {
  using Elem = typename Score<DT>::Elem;
  constexpr int VE = Score<DT>::kVec;
  extern __shared__ uint32_t bits[];
  __shared__ float shf[NT / 64];
  __shared__ double shd[NT / 64];
  const int tid = threadIdx.x;
  const int32_t C = a.C;
  const float cf = (float)a.c;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    const Elem* __restrict__ xr = static_cast<const Elem*>(a.x) + i * a.ld;
    for (int32_t wd = tid; wd < (C + 31) / 32; wd += NT) bits[wd] = 0u;
    __syncthreads();
    int32_t cls = -1;
    float t = -kInf, xj = -kInf;
    if (tid < a.k) {
      cls = a.tc[i * a.k + tid];
      if (cls >= C) {
        dev_error(a.err, GBDT_E_RANGE);
        cls = -1;
      }
      if (cls >= 0) {
        const uint32_t b = 1u << (cls & 31);
        if (atomicOr(&bits[cls >> 5], b) & b) dev_error(a.err, GBDT_E_ARG);
        t = a.tv[i * a.k + tid];
        xj = Score<DT>::to_f32(xr[cls]);
      }
    }
    const double r = row_rest(a, i, tid == 0);
    const bool has = __syncthreads_or(!(t == -kInf));
    const float tm = block_max<NT>(t, shf);
    const double ts = tm == -kInf ? 0.0 : (double)tm;
    const double e = exp2_64(((double)t - ts) * a.c);
    const double z = block_sum<NT>(e, shd);
    float m = -kInf;
    double s_in, s_out;
    if (MODE & kStats) {
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
#pragma unroll
        for (int q = 0; q < VE; ++q) m = __builtin_fmaxf(m, f[q]);
      }
      m = block_max<NT>(m, shf);
    } else {
      m = a.stats_in[3 * i];
    }
    const float mf = m == -kInf ? 0.0f : m;
    const double ms = (double)mf;
    const double wj = cls >= 0 ? exp2_64(((double)xj - ms) * a.c) : 0.0;
    if (MODE & kStats) {
      s_in = block_sum<NT>(wj, shd);
      double so = 0.0;
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
        const uint32_t in_s = bits[c0 >> 5] >> (c0 & 31);
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          const float wq = exp2_32((f[q] - mf) * cf);
          so += (in_s >> q & 1u) ? 0.0 : (double)wq;
        }
      }
      s_out = block_sum<NT>(so, shd);
    } else {
      s_in = a.stats_in[3 * i + 1];
      s_out = a.stats_in[3 * i + 2];
    }
    const double s = s_in + s_out;
    const bool live = has && !(s == 0.0);
    const double pj = live ? e * (1.0 - r) / z : 0.0;
    if ((MODE & kStats) && a.stats_out != nullptr && tid == 0) {
      a.stats_out[3 * i] = m;
      a.stats_out[3 * i + 1] = (float)s_in;
      a.stats_out[3 * i + 2] = (float)s_out;
    }
    if (MODE & kLoss) {
      const double d = (((double)t - ts) - ((double)xj - ms));
      const double k_sum = block_sum<NT>(pj == 0.0 ? 0.0 : pj * d, shd);
      if (tid == 0) a.loss[i] = live ? (float)row_loss(a.T, r, z, k_sum, s_in, s_out) : 0.0f;
    }
    if (MODE & kGrad) {
      const float wt = a.weight != nullptr ? a.weight[i] : 1.0f;
      const bool counts = live && !(wt == 0.0f);
      const double g = (double)wt * (double)a.T;
      const double share = s_out > 0.0 ? 1.0 - r * s / s_out : (s_out == 0.0 ? 0.0 : s_out);
      const float scale = counts ? (float)(g * share / s) : 0.0f;
      Elem* __restrict__ gr = static_cast<Elem*>(a.grad) + i * a.ldg;
      for (int32_t c0 = tid * VE; c0 < C; c0 += NT * VE) {
        float f[VE];
        load_chunk<DT>(xr, c0, C, f);
        const uint32_t in_s = (bits[c0 >> 5] >> (c0 & 31)) & ((1u << VE) - 1u);
        Vec16<DT> o;
#pragma unroll
        for (int q = 0; q < VE; ++q)
          o.e[q] = Score<DT>::from_f32(counts ? exp2_32((f[q] - mf) * cf) * scale : 0.0f);
        if (in_s == 0u && c0 + VE <= C) {
          __builtin_memcpy(gr + c0, &o, 16);
        } else {
#pragma unroll
          for (int q = 0; q < VE; ++q)
            if (c0 + q < C && !(in_s >> q & 1u)) gr[c0 + q] = o.e[q];
        }
      }
      if (cls >= 0) gr[cls] = Score<DT>::from_f32(counts ? (float)(g * (wj / s - pj)) : 0.0f);
    }
    __syncthreads();  // (the bits are free)
  }
}

constexpr int64_t kMaxRowGrid = 1 << 20;  // workgroups of a row launch, at most

template <int DT, int MODE>
int launch_distill(const DistillArgs& a, hipStream_t s) {
  diag_begin(kDiagDistill, s);
  if (a.C <= kRowsMaxClasses) {
    const dim3 grid((unsigned)((a.n + 255) / 256));
    if (a.C <= 8)
      hipLaunchKernelGGL((k_distill_rows<DT, 8, MODE>), grid, dim3(256), 0, s, a);
    else if (a.C <= 16)
      hipLaunchKernelGGL((k_distill_rows<DT, 16, MODE>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((k_distill_rows<DT, 32, MODE>), grid, dim3(256), 0, s, a);
  } else {
    const dim3 grid((unsigned)(a.n < kMaxRowGrid ? a.n : kMaxRowGrid));
    const size_t lds = size_t((a.C + 31) / 32) * 4;
    if (a.C <= 8192)
      hipLaunchKernelGGL((k_distill_block<DT, 256, MODE>), grid, dim3(256), lds, s, a);
    else
      hipLaunchKernelGGL((k_distill_block<DT, 1024, MODE>), grid, dim3(1024), lds, s, a);
  }
  diag_end(s);
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
  if (MODE & kGrad) {
    if (!grad) return fail(GBDT_E_ARG, "grad is null");
    if (x->n_rows > 1 && grad_stride < x->n_classes)
      return fail(GBDT_E_SHAPE, "grad_stride smaller than n_classes");
    const uintptr_t es = x->dtype == GBDT_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(grad) % es) return fail(GBDT_E_ARG, "grad is misaligned");
  }
  rc = check_scores_ws(*x, ws, ws_bytes);
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
  a.weight = weight;
  a.stats_out = stats_out;
  a.stats_in = stats_in;
  a.loss = loss;
  a.grad = grad;
  a.ldg = grad_stride;
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
  return sizeof(WsCtrl);
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
