// Distillation from a teacher's top logits: the loss of a row and its
// gradient (see lopt_train.h).
//
// With m = max z and s = sum exp((z - m) / T), log q_j = (z_j - m) / T - log s.
// The exponents are taken of z - m, not of z / T - m / T: masks of the type's
// lowest value stay finite that way, and the terms near the maximum exact.
// The dense part of the gradient, w T q_j, is written for every column and
// the listed columns are then written again with their p taken off.
#include <algorithm>

#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

struct Distill {
  const void *logits, *top_logits, *top_index;
  const float* row_weight;
  float* loss;
  void* grad;
  int32_t* status;
  int64_t rows, cols, ls, ts, is, gs;
  int top, ttype, itype;
  float temperature, inv_t, log2e_t;   // T, 1 / T, log2(e) / T
};

// 2^x: the ex2.approx instruction (relative error below 2^-22).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int W>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t += red[k];
  return t;
}
template <int W>
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t = fmaxf(t, red[k]);
  return t;
}

// One block per row, which is read from memory for each of the three passes.
template <typename T>
__global__ void __launch_bounds__(512) k_distill_rows(const Distill a) {
  constexpr int L = 512, W = L / 32;
  __shared__ float red[W];
  __shared__ int32_t id[LOPT_MAX_TOP];
  __shared__ float p[LOPT_MAX_TOP], zi[LOPT_MAX_TOP];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + row * a.ls;
  T* g = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  float tmax = -INFINITY;
  bool any = false;
  if (w != 0.f) {
    for (int k = tid; k < a.top; k += L) {
      const int64_t i = load_index(a.top_index, row * a.is + k, a.itype);
      float t = load_as_f(a.top_logits, row * a.ts + k, a.ttype);
      if (i >= a.cols && a.status) atomicOr(a.status, 1);
      const bool counts = i >= 0 && i < a.cols && t != -INFINITY;
      id[k] = counts ? (int32_t)i : -1;
      p[k] = t;
      any |= counts;
      if (counts) tmax = fmaxf(tmax, t);
    }
  }
  if (!__syncthreads_or(any)) {   // nothing to learn from this row
    if (tid == 0) a.loss[row] = 0.f;
    if (g)
      for (int64_t j = tid; j < a.cols; j += L) g[j] = from_f<T>(0.f);
    return;
  }
  tmax = block_max<W>(tmax, red);
  float ps = 0.f;
  for (int k = tid; k < a.top; k += L) {
    if (id[k] < 0) continue;
    ps += ex2((p[k] - tmax) * a.log2e_t);
    zi[k] = to_f(z[id[k]]);
  }
  ps = block_sum<W>(ps, red);
  float m = -INFINITY;
  for (int64_t j = tid; j < a.cols; j += L) m = fmaxf(m, to_f(z[j]));
  m = block_max<W>(m, red);
  float s = 0.f;
  for (int64_t j = tid; j < a.cols; j += L) s += ex2((to_f(z[j]) - m) * a.log2e_t);
  s = block_sum<W>(s, red);
  const float log_s = logf(s), log_ps = logf(ps), inv_ps = 1.f / ps;
  float kl = 0.f;
  for (int k = tid; k < a.top; k += L) {
    if (id[k] < 0) continue;
    const float d = p[k] - tmax;
    const float pk = ex2(d * a.log2e_t) * inv_ps;
    const float term = pk * ((d * a.inv_t - log_ps) - ((zi[k] - m) * a.inv_t - log_s));
    if (pk != 0.f) kl += term;   // 0 log 0 = 0
    p[k] = pk;
  }
  kl = block_sum<W>(kl, red);
  if (tid == 0) a.loss[row] = w * a.temperature * a.temperature * kl;
  if (!g) return;
  const float wt = w * a.temperature, f = wt / s;
  for (int64_t j = tid; j < a.cols; j += L) g[j] = from_f<T>(ex2((to_f(z[j]) - m) * a.log2e_t) * f);
  __syncthreads();
  // A class listed more than once is written by its first slot.
  for (int k = tid; k < a.top; k += L) {
    if (id[k] < 0) continue;
    bool first = true;
    for (int o = 0; o < k && first; ++o) first = id[o] != id[k];
    if (!first) continue;
    float pk = p[k];
    for (int o = k + 1; o < a.top; ++o)
      if (id[o] == id[k]) pk += p[o];
    g[id[k]] = from_f<T>(fmaf(ex2((zi[k] - m) * a.log2e_t), f, -wt * pk));
  }
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" int lopt_distill(const void* logits, int type, int64_t rows, int64_t cols, int64_t logits_stride,
                            const void* top_logits, int top_type, int64_t top_logits_stride, const void* top_index,
                            int index_type, int64_t top_index_stride, int64_t top, float temperature,
                            const float* row_weight, float* loss, void* grad, int64_t grad_stride, int32_t* status,
                            void* stream) {
  const int es = type_size(type), ts = type_size(top_type), is = index_size(index_type);
  if (!es || !ts || !is || (top_type != LOPT_F32 && top_type != type)) return LOPT_E_ARG;
  // T, 1 / T and log2(e) / T are finite and not zero.
  if (!(temperature >= 1e-30f && temperature <= 1e30f)) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols || top < 1 || top > LOPT_MAX_TOP) return LOPT_E_SHAPE;
  if (rows == 0) return LOPT_OK;
  const Span mz{logits, rows, cols, logits_stride, es}, mt{top_logits, rows, top, top_logits_stride, ts};
  const Span mi{top_index, rows, top, top_index_stride, is}, mw{row_weight, 1, rows, rows, 4};
  const Span ml{loss, 1, rows, rows, 4}, mg{grad, rows, cols, grad_stride, es};
  int rc;
  if ((rc = check_matrix(mz, false)) || (rc = check_matrix(mt, false)) || (rc = check_matrix(mi, false)) ||
      (rc = check_matrix(ml, true)))
    return rc;
  if (grad && (rc = check_matrix(mg, true))) return rc;
  if (row_weight && (rc = check_matrix(mw, false))) return rc;
  if (status && (uintptr_t)status % 4) return LOPT_E_ALIGN;
  if (overlap(ml, mg) || (overlap(mg, mz) && !mg.same_place(mz))) return LOPT_E_ALIAS;
  for (const Span* in : {&mt, &mi, &mw})
    if (overlap(ml, *in) || overlap(mg, *in)) return LOPT_E_ALIAS;
  if (overlap(ml, mz)) return LOPT_E_ALIAS;
  const Distill a{logits, top_logits, top_index, row_weight, loss, grad, status, rows, cols, logits_stride,
                  top_logits_stride, top_index_stride, grad_stride, (int)top, top_type, index_type, temperature,
                  1.f / temperature, 1.4426950408889634f / temperature};
  cudaStream_t s = (cudaStream_t)stream;
  const dim3 grid((unsigned)rows);
  switch (type) {
    case LOPT_F32: return done(launch(k_distill_rows<float>, grid, dim3(512), 0, s, false, 1, a));
    case LOPT_F16: return done(launch(k_distill_rows<__half>, grid, dim3(512), 0, s, false, 1, a));
    default: return done(launch(k_distill_rows<__nv_bfloat16>, grid, dim3(512), 0, s, false, 1, a));
  }
}
