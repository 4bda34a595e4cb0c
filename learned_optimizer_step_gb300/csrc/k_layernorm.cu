// Layer norm over rows, forward and backward (see lopt_train.h).
//
// Forward, s = x + residual:  y = (s - mean) * rstd * w + b.  A row is read
// once into registers; mean and variance are two sums over them (the variance
// about the mean, not E[s^2] - mean^2, which cancels for rows far from 0).
// Backward, with xhat = (x - mean) * rstd and g = dy * w:
//   dx = rstd * (g - <g> - xhat * <g xhat>),   dw = sum dy * xhat,  db = sum dy.
// Each thread keeps the sums over rows of its own columns in registers; the
// blocks' sums go to the workspace and a second kernel adds them in block
// order.  Both directions are bound by HBM bytes.
#include <algorithm>

#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

struct NormFwd {
  const void *x, *residual, *weight, *bias;
  void *y, *summed;
  float *mean, *rstd;
  int64_t rows, cols, xs, rs, ys, ss;
  int wtype;
  float eps;
};

struct NormBwd {
  const void *dy, *x, *weight, *dres;
  const float *mean, *rstd;
  void* dx;
  float* part;      // [2][gridDim.x][cols]: sums of dy * xhat, then of dy
  int64_t rows, cols, dys, xs, drs, dxs;
  int wtype;
};

// Sum over the L threads of a row; L == 32: a warp, else the whole block.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (L == 32) return v;
  constexpr int W = L / 32;
  const int w = threadIdx.x / 32;
  __syncthreads();                      // the previous use of red is over
  if (threadIdx.x % 32 == 0) red[w] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t += red[k];
  return t;
}

template <int L>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (L == 32) return make_float2(a, b);
  constexpr int W = L / 32;
  const int w = threadIdx.x / 32;
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[w] = make_float2(a, b);
  __syncthreads();
  float2 t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) {
    t.x += red[k].x;
    t.y += red[k].y;
  }
  return t;
}

// VEC consecutive weights from column j on.
template <typename T, int VEC>
__device__ __forceinline__ void load_weights(const void* p, int wtype, int64_t j, float out[VEC]) {
  if (wtype == LOPT_F32) {
    constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
    for (int k = 0; k < VEC; k += V4) {
      const Pack<float, V4> q = *reinterpret_cast<const Pack<float, V4>*>(static_cast<const float*>(p) + j + k);
#pragma unroll
      for (int e = 0; e < V4; ++e) out[k + e] = q.v[e];
    }
  } else {
    const Pack<T, VEC> q = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(p) + j);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = to_f(q.v[e]);
  }
}

__host__ __device__ constexpr int row_threads(int L) { return L == 32 ? 256 : L; }

// L threads per row, each with SLOTS accesses of VEC elements.
template <typename T, int VEC, int SLOTS, int L>
__global__ void __launch_bounds__(row_threads(L)) k_norm_fwd(const NormFwd a) {
  constexpr int R = row_threads(L) / L;
  __shared__ float red[L / 32];
  const int lane = threadIdx.x % L;
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / L;
  if (row >= a.rows) return;            // whole warps when L == 32, else never
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.rs : nullptr;
  const int cols = (int)a.cols;
  Pack<T, VEC> px[SLOTS], pr[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int j = (s * L + lane) * VEC;
    if (j < cols) {
      px[s] = *reinterpret_cast<const Pack<T, VEC>*>(x + j);
      if (r) pr[s] = *reinterpret_cast<const Pack<T, VEC>*>(r + j);
    }
  }
  float v[SLOTS][VEC];
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const bool in = (s * L + lane) * VEC < cols;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[s][e] = in ? to_f(px[s].v[e]) + (r ? to_f(pr[s].v[e]) : 0.f) : 0.f;
      sum += v[s][e];
    }
  }
  const float inv = 1.f / (float)cols;
  const float mean = row_sum<L>(sum, red) * inv;
  float sq = 0.f;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if ((s * L + lane) * VEC < cols) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = v[s][e] - mean;
        sq = fmaf(d, d, sq);
      }
    }
  }
  const float rstd = rsqrtf(row_sum<L>(sq, red) * inv + a.eps);
  if (lane == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ys;
  T* sm = a.summed ? static_cast<T*>(a.summed) + row * a.ss : nullptr;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int j = (s * L + lane) * VEC;
    if (j >= cols) continue;
    float w[VEC], b[VEC];
    load_weights<T, VEC>(a.weight, a.wtype, j, w);
    if (a.bias) {
      load_weights<T, VEC>(a.bias, a.wtype, j, b);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
    }
    Pack<T, VEC> o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o.v[e] = from_f<T>(fmaf((v[s][e] - mean) * rstd, w[e], b[e]));
    if (sm) {
      Pack<T, VEC> q;
#pragma unroll
      for (int e = 0; e < VEC; ++e) q.v[e] = from_f<T>(v[s][e]);
      *reinterpret_cast<Pack<T, VEC>*>(sm + j) = q;
    }
    *reinterpret_cast<Pack<T, VEC>*>(y + j) = o;
  }
}

// Rows too long for registers: one block per row, which reads the row three
// times (from L2 after the first).
template <typename T>
__global__ void __launch_bounds__(512) k_norm_fwd_long(const NormFwd a) {
  constexpr int L = 512;
  __shared__ float red[L / 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.rs : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ys;
  T* sm = a.summed ? static_cast<T*>(a.summed) + row * a.ss : nullptr;
  float sum = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) sum += to_f(x[j]) + (r ? to_f(r[j]) : 0.f);
  const float inv = 1.f / (float)a.cols;
  const float mean = row_sum<L>(sum, red) * inv;
  float sq = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    const float d = to_f(x[j]) + (r ? to_f(r[j]) : 0.f) - mean;
    sq = fmaf(d, d, sq);
  }
  const float rstd = rsqrtf(row_sum<L>(sq, red) * inv + a.eps);
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    const float s = to_f(x[j]) + (r ? to_f(r[j]) : 0.f);
    float w, b = 0.f;
    load_weights<T, 1>(a.weight, a.wtype, j, &w);
    if (a.bias) load_weights<T, 1>(a.bias, a.wtype, j, &b);
    if (sm) sm[j] = from_f<T>(s);
    y[j] = from_f<T>(fmaf((s - mean) * rstd, w, b));
  }
}

// Persistent: a block's row groups take rows blockIdx.x * R + group,
// striding by gridDim.x * R, and keep the column sums of their columns.
template <typename T, int VEC, int SLOTS, int L>
__global__ void __launch_bounds__(row_threads(L)) k_norm_bwd(const NormBwd a) {
  constexpr int TH = row_threads(L), R = TH / L;
  __shared__ float2 red[L / 32];
  __shared__ float comb[R > 1 ? TH * VEC : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int cols = (int)a.cols;
  const float inv = 1.f / (float)cols;
  float dw[SLOTS][VEC], db[SLOTS][VEC];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[s][e] = db[s][e] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * R + group; row < a.rows; row += (int64_t)gridDim.x * R) {
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dys;
    Pack<T, VEC> px[SLOTS], pd[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = (s * L + lane) * VEC;
      if (j < cols) {
        px[s] = *reinterpret_cast<const Pack<T, VEC>*>(x + j);
        pd[s] = *reinterpret_cast<const Pack<T, VEC>*>(dy + j);
      }
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = (s * L + lane) * VEC;
      if (j >= cols) continue;
      float w[VEC];
      load_weights<T, VEC>(a.weight, a.wtype, j, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = to_f(pd[s].v[e]);
        const float xh = (to_f(px[s].v[e]) - mean) * rstd;
        const float g = d * w[e];
        sg += g;
        sgx = fmaf(g, xh, sgx);
        dw[s][e] = fmaf(d, xh, dw[s][e]);
        db[s][e] += d;
      }
    }
    const float2 t = row_sum2<L>(sg, sgx, red);
    const float mg = t.x * inv, mgx = t.y * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.dxs;
    const T* dr = a.dres ? static_cast<const T*>(a.dres) + row * a.drs : nullptr;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = (s * L + lane) * VEC;
      if (j >= cols) continue;
      float w[VEC];
      load_weights<T, VEC>(a.weight, a.wtype, j, w);
      Pack<T, VEC> o, q;
      if (dr) q = *reinterpret_cast<const Pack<T, VEC>*>(dr + j);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (to_f(px[s].v[e]) - mean) * rstd;
        const float g = to_f(pd[s].v[e]) * w[e];
        const float v = rstd * (g - mg - xh * mgx);
        o.v[e] = from_f<T>(dr ? v + to_f(q.v[e]) : v);
      }
      *reinterpret_cast<Pack<T, VEC>*>(dx + j) = o;
    }
  }
  // The block's sums: over its row groups in order.
  float* pw = a.part + (int64_t)blockIdx.x * cols;
  float* pb = a.part + ((int64_t)gridDim.x + blockIdx.x) * cols;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int j = (s * L + lane) * VEC;
    if (R == 1) {
      if (j < cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          pw[j + e] = dw[s][e];
          pb[j + e] = db[s][e];
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) comb[group * L * VEC + e * L + lane] = h ? db[s][e] : dw[s][e];
        __syncthreads();
        for (int c = threadIdx.x; c < L * VEC; c += TH) {   // c = e * L + lane of the column
          float t = 0.f;
#pragma unroll
          for (int g = 0; g < R; ++g) t += comb[g * L * VEC + c];
          const int col = (s * L + c % L) * VEC + c / L;
          if (col < cols) (h ? pb : pw)[col] = t;
        }
      }
    }
  }
}

// Rows too long for registers: dx row by row; the column sums are another
// kernel's.
template <typename T>
__global__ void __launch_bounds__(512) k_norm_bwd_long(const NormBwd a) {
  constexpr int L = 512;
  __shared__ float2 red[L / 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* dy = static_cast<const T*>(a.dy) + row * a.dys;
  const T* dr = a.dres ? static_cast<const T*>(a.dres) + row * a.drs : nullptr;
  T* dx = static_cast<T*>(a.dx) + row * a.dxs;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float sg = 0.f, sgx = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    float w;
    load_weights<T, 1>(a.weight, a.wtype, j, &w);
    const float g = to_f(dy[j]) * w;
    sg += g;
    sgx = fmaf(g, (to_f(x[j]) - mean) * rstd, sgx);
  }
  const float2 t = row_sum2<L>(sg, sgx, red);
  const float inv = 1.f / (float)a.cols;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    float w;
    load_weights<T, 1>(a.weight, a.wtype, j, &w);
    const float v = rstd * (to_f(dy[j]) * w - t.x * inv - (to_f(x[j]) - mean) * rstd * (t.y * inv));
    dx[j] = from_f<T>(dr ? v + to_f(dr[j]) : v);
  }
}

// Column sums of long rows, before dx may overwrite its inputs: each thread
// one column, each blockIdx.y a run of rows.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_cols_long(const NormBwd a) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= a.cols) return;
  const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
  const int64_t end = min(a.rows, per * (blockIdx.y + 1));
  float dw = 0.f, db = 0.f;
  for (int64_t row = per * blockIdx.y; row < end; ++row) {
    const float d = to_f(static_cast<const T*>(a.dy)[row * a.dys + j]);
    dw = fmaf(d, (to_f(static_cast<const T*>(a.x)[row * a.xs + j]) - a.mean[row]) * a.rstd[row], dw);
    db += d;
  }
  a.part[(int64_t)blockIdx.y * a.cols + j] = dw;
  a.part[((int64_t)gridDim.y + blockIdx.y) * a.cols + j] = db;
}

// The blocks' sums of 32 columns: warp w adds blocks w, w + 32, ..., then one
// warp the 32 sums in order.  blockIdx.y: 0 the weight's, 1 the bias's.
__global__ void __launch_bounds__(1024) k_norm_finish(const float* part, int blocks, int64_t cols, float* dw, float* db,
                                                      int accumulate) {
  __shared__ float red[32][33];
  wait_for_previous();
  float* out = blockIdx.y ? db : dw;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  const float* p = part + (int64_t)blockIdx.y * blocks * cols;
  float t = 0.f;
  if (j < cols)
    for (int b = w; b < blocks; b += 32) t += p[(int64_t)b * cols + j];
  red[w][lane] = t;
  __syncthreads();
  if (w == 0 && j < cols) {
    t = red[0][lane];
#pragma unroll
    for (int k = 1; k < 32; ++k) t += red[k][lane];
    out[j] = accumulate ? out[j] + t : t;
  }
}

// ---- choice of the kernel -------------------------------------------------------
// nvec accesses of VEC elements per row.  A warp per row while a lane holds
// at most 32 elements, then 256 and 512 threads; longer rows read again.
constexpr int kMaxBlocks = 1216;   // partial sums in the workspace

template <typename T, int VEC, int SLOTS, int L>
cudaError_t fwd_as(const NormFwd& a, cudaStream_t s) {
  constexpr int R = row_threads(L) / L;
  const int64_t grid = (a.rows + R - 1) / R;
  return launch(k_norm_fwd<T, VEC, SLOTS, L>, dim3((unsigned)grid), dim3(row_threads(L)), 0, s, false, 1, a);
}

template <typename T, int VEC, int SLOTS, int L>
cudaError_t bwd_as(const NormBwd& a, int sms, cudaStream_t s, int* blocks) {
  constexpr int R = row_threads(L) / L;
  int per_sm = 1;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_norm_bwd<T, VEC, SLOTS, L>, row_threads(L), 0);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>({(a.rows + R - 1) / R, (int64_t)sms * std::max(per_sm, 1), kMaxBlocks});
  *blocks = (int)grid;
  return launch(k_norm_bwd<T, VEC, SLOTS, L>, dim3((unsigned)grid), dim3(row_threads(L)), 0, s, false, 1, a);
}

// f.template operator()<VEC, SLOTS, L>() for the shape of a row.
#define LOPT_NORM_CASE(V, S, L_) if (nvec <= (int64_t)(S) * (L_)) return f.template run<V, S, L_>()
template <int FULL, typename F>
cudaError_t pick(int64_t cols, bool vec, F f) {
  if (vec) {
    const int64_t nvec = (cols + FULL - 1) / FULL;
    LOPT_NORM_CASE(FULL, 1, 32);
    LOPT_NORM_CASE(FULL, 2, 32);
    LOPT_NORM_CASE(FULL, 3, 32);
    LOPT_NORM_CASE(FULL, 4, 32);
    if constexpr (FULL == 4) {
      LOPT_NORM_CASE(FULL, 6, 32);
      LOPT_NORM_CASE(FULL, 8, 32);
    }
    LOPT_NORM_CASE(FULL, 1, 256);
    LOPT_NORM_CASE(FULL, 2, 256);
    LOPT_NORM_CASE(FULL, 4, 256);
    if constexpr (FULL == 4) {
      LOPT_NORM_CASE(FULL, 8, 256);
    }
    LOPT_NORM_CASE(FULL, 32 / FULL, 512);
  } else {
    const int64_t nvec = cols;
    LOPT_NORM_CASE(1, 4, 32);
    LOPT_NORM_CASE(1, 8, 32);
    LOPT_NORM_CASE(1, 16, 32);
    LOPT_NORM_CASE(1, 4, 256);
    LOPT_NORM_CASE(1, 8, 256);
    LOPT_NORM_CASE(1, 16, 256);
    LOPT_NORM_CASE(1, 32, 512);
  }
  return f.long_rows();
}

template <typename T> struct FwdRun {
  const NormFwd& a;
  cudaStream_t s;
  template <int V, int S, int L> cudaError_t run() { return fwd_as<T, V, S, L>(a, s); }
  cudaError_t long_rows() {
    return launch(k_norm_fwd_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
  }
};

template <typename T> struct BwdRun {
  const NormBwd& a;
  int sms;
  cudaStream_t s;
  int* blocks;
  template <int V, int S, int L> cudaError_t run() { return bwd_as<T, V, S, L>(a, sms, s, blocks); }
  cudaError_t long_rows() {
    *blocks = (int)std::min<int64_t>(a.rows, 32);
    const dim3 grid((unsigned)((a.cols + 255) / 256), (unsigned)*blocks);
    cudaError_t e = launch(k_norm_cols_long<T>, grid, dim3(256), 0, s, false, 1, a);
    if (e != cudaSuccess) return e;
    return launch(k_norm_bwd_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
  }
};

// Vector accesses need whole vectors in a row and aligned rows.
bool vec_ok(int64_t cols, int es, std::initializer_list<Span> ms, const void* w, const void* b, int wsize) {
  if ((cols * es) % 16) return false;
  for (const Span& m : ms)
    if (!rows_aligned(m, 16)) return false;
  (void)wsize;
  return (uintptr_t)w % 16 == 0 && (uintptr_t)b % 16 == 0;
}

int check_weight(const void* w, int wtype, int type) {
  if (!w) return LOPT_E_ARG;
  if (wtype != LOPT_F32 && wtype != type) return LOPT_E_ARG;
  return (uintptr_t)w % type_size(wtype) ? LOPT_E_ALIGN : LOPT_OK;
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_layernorm_forward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* residual,
                           int64_t residual_stride, const void* weight, const void* bias, int weight_type, float eps,
                           void* y, int64_t y_stride, void* summed, int64_t summed_stride, float* mean, float* rstd,
                           void* stream) {
  const int es = type_size(type);
  if (!es || !(eps >= 0.f) || (summed && !residual)) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols) return LOPT_E_SHAPE;
  if (rows == 0) return LOPT_OK;
  const Span mx{x, rows, cols, x_stride, es}, mr{residual, rows, cols, residual_stride, es};
  const Span my{y, rows, cols, y_stride, es}, ms{summed, rows, cols, summed_stride, es};
  const Span sm{mean, 1, rows, rows, 4}, sr{rstd, 1, rows, rows, 4};
  int rc;
  if ((rc = check_matrix(mx, false)) || (rc = check_matrix(my, true))) return rc;
  if (residual && (rc = check_matrix(mr, false))) return rc;
  if (summed && (rc = check_matrix(ms, true))) return rc;
  if ((rc = check_matrix(sm, true)) || (rc = check_matrix(sr, true)) || (rc = check_weight(weight, weight_type, type)))
    return rc;
  if (bias && (rc = check_weight(bias, weight_type, type))) return rc;
  const Span sw{weight, 1, cols, cols, type_size(weight_type)}, sb{bias, 1, cols, cols, type_size(weight_type)};
  const Span* outs[4] = {&my, &ms, &sm, &sr};
  for (int i = 0; i < 4; ++i) {
    for (int k = i + 1; k < 4; ++k)
      if (overlap(*outs[i], *outs[k])) return LOPT_E_ALIAS;
    for (const Span* in : {&mx, &mr})
      if (overlap(*outs[i], *in) && !(i < 2 && outs[i]->same_place(*in))) return LOPT_E_ALIAS;
    if (overlap(*outs[i], sw) || overlap(*outs[i], sb)) return LOPT_E_ALIAS;
  }
  const NormFwd a{x, residual, weight, bias, y, summed, mean, rstd, rows, cols, x_stride, residual_stride,
                  y_stride, summed_stride, weight_type, eps};
  const bool vec = vec_ok(cols, es, {mx, mr, my, ms}, weight, bias, type_size(weight_type));
  cudaStream_t s = (cudaStream_t)stream;
  switch (type) {
    case LOPT_F32: return done(pick<4>(cols, vec, FwdRun<float>{a, s}));
    case LOPT_F16: return done(pick<8>(cols, vec, FwdRun<__half>{a, s}));
    default: return done(pick<8>(cols, vec, FwdRun<__nv_bfloat16>{a, s}));
  }
}

int lopt_layernorm_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols) return LOPT_E_SHAPE;
  *bytes = 2 * std::min<int64_t>(std::max<int64_t>(rows, 1), kMaxBlocks) * cols * 4;
  return LOPT_OK;
}

int lopt_layernorm_backward(const void* grad_out, int type, int64_t rows, int64_t cols, int64_t grad_out_stride,
                            const void* x, int64_t x_stride, const float* mean, const float* rstd, const void* weight,
                            int weight_type, const void* grad_residual, int64_t grad_residual_stride, void* grad_x,
                            int64_t grad_x_stride, float* grad_weight, float* grad_bias, int accumulate,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  const int es = type_size(type);
  if (!es || !grad_weight || (accumulate != 0 && accumulate != 1)) return LOPT_E_ARG;
  int64_t need = 0;
  int rc = lopt_layernorm_workspace(rows, cols, &need);
  if (rc) return rc;
  const Span gw{grad_weight, 1, cols, cols, 4}, gb{grad_bias, 1, cols, cols, 4};
  if ((rc = check_matrix(gw, true)) || (grad_bias && (rc = check_matrix(gb, true)))) return rc;
  if (overlap(gw, gb)) return LOPT_E_ALIAS;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    if (accumulate) return LOPT_OK;
    cudaError_t e = cudaMemsetAsync(grad_weight, 0, cols * 4, s);
    if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, cols * 4, s);
    return done(e);
  }
  const Span md{grad_out, rows, cols, grad_out_stride, es}, mx{x, rows, cols, x_stride, es};
  const Span mr{grad_residual, rows, cols, grad_residual_stride, es}, mo{grad_x, rows, cols, grad_x_stride, es};
  const Span sm{mean, 1, rows, rows, 4}, sr{rstd, 1, rows, rows, 4};
  const Span sw{weight, 1, cols, cols, type_size(weight_type)};
  const Span ws{workspace, 1, need, need, 1};
  if ((rc = check_matrix(md, false)) || (rc = check_matrix(mx, false)) || (rc = check_matrix(mo, true)) ||
      (rc = check_matrix(sm, false)) || (rc = check_matrix(sr, false)) || (rc = check_weight(weight, weight_type, type)))
    return rc;
  if (grad_residual && (rc = check_matrix(mr, false))) return rc;
  if (!workspace || workspace_bytes < need) return LOPT_E_ARG;
  if ((uintptr_t)workspace % 256) return LOPT_E_ALIGN;
  const Span* outs[4] = {&mo, &gw, &gb, &ws};
  for (int i = 0; i < 4; ++i) {
    for (int k = i + 1; k < 4; ++k)
      if (overlap(*outs[i], *outs[k])) return LOPT_E_ALIAS;
    for (const Span* in : {&md, &mx, &mr})
      if (overlap(*outs[i], *in) && !(i == 0 && mo.same_place(*in))) return LOPT_E_ALIAS;
    for (const Span* in : {&sm, &sr, &sw})
      if (overlap(*outs[i], *in)) return LOPT_E_ALIAS;
  }
  const NormBwd a{grad_out, x, weight, grad_residual, mean, rstd, grad_x, (float*)workspace, rows, cols,
                  grad_out_stride, x_stride, grad_residual_stride, grad_x_stride, weight_type};
  const bool vec = vec_ok(cols, es, {md, mx, mr, mo}, weight, nullptr, type_size(weight_type));
  const int sms = sm_count();
  int blocks = 0;
  cudaError_t e;
  switch (type) {
    case LOPT_F32: e = pick<4>(cols, vec, BwdRun<float>{a, sms, s, &blocks}); break;
    case LOPT_F16: e = pick<8>(cols, vec, BwdRun<__half>{a, sms, s, &blocks}); break;
    default: e = pick<8>(cols, vec, BwdRun<__nv_bfloat16>{a, sms, s, &blocks}); break;
  }
  if (e != cudaSuccess) return done(e);
  return done(launch(k_norm_finish, dim3((unsigned)((cols + 31) / 32), grad_bias ? 2u : 1u), dim3(1024), 0, s, true, 1,
                     (const float*)workspace, blocks, cols, grad_weight, grad_bias, accumulate));
}

}  // extern "C"
