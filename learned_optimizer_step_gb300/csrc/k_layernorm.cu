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
#include <cstring>

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

// Sum over the L threads of a row that are a whole block (L > 32), a warp or
// half of one.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (L <= 32) return v;
  constexpr int W = L <= 32 ? 1 : L / 32;
  __syncthreads();                      // the previous use of red is over
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t += red[k];
  return t;
}

// Two sums over the L threads of group `group` of a block; red alternates
// between two areas from row to row, so one barrier does.
template <int L>
__device__ __forceinline__ float2 group_sum2(float2 v, float2* red, int group) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1)
    v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if (L <= 32) return v;
  constexpr int W = L <= 32 ? 1 : L / 32;
  red += group * W;
  if (threadIdx.x % 32 == 0) red[threadIdx.x % L / 32] = v;
  asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "n"(L) : "memory");
  float2 t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t = __fadd2_rn(t, red[k]);
  return t;
}

// VEC consecutive weights from column j on.
template <typename T, int VEC>
__device__ __forceinline__ void load_weights(const void* p, int wtype, int64_t j, float (&out)[VEC]) {
  if (wtype == LOPT_F32) {
    constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
    for (int k = 0; k < VEC; k += V4) {
      const Pack<float, V4> q = *reinterpret_cast<const Pack<float, V4>*>(static_cast<const float*>(p) + j + k);
#pragma unroll
      for (int e = 0; e < V4; ++e) out[k + e] = q.v[e];
    }
  } else {
    to_floats(*reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(p) + j), out);
  }
}

// Elementwise arithmetic on a lane's V elements: two at a time, by one
// instruction for both, where V is even.
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
#define LOPT_EACH(V, PAIRS, SINGLE)                                     \
  if constexpr ((V) % 2 == 0) {                                         \
    _Pragma("unroll") for (int k = 0; k < (V); k += 2) { PAIRS; }       \
  } else {                                                              \
    _Pragma("unroll") for (int k = 0; k < (V); ++k) { SINGLE; }         \
  }
template <int V> __device__ __forceinline__ float2 at2(const float (&v)[V], int k) { return make_float2(v[k], v[k + 1]); }
template <int V> __device__ __forceinline__ void set2(float (&v)[V], int k, float2 x) {
  v[k] = x.x;
  v[k + 1] = x.y;
}
// o = (x + a) * b
template <int V> __device__ __forceinline__ void add_mul(const float (&x)[V], float a, float b, float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __fmul2_rn(__fadd2_rn(at2(x, k), two(a)), two(b))), o[k] = (x[k] + a) * b)
}
// o += a;  o *= a
template <int V> __device__ __forceinline__ void add_one(float a, float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __fadd2_rn(at2(o, k), two(a))), o[k] += a)
}
template <int V> __device__ __forceinline__ void mul_one(float a, float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __fmul2_rn(at2(o, k), two(a))), o[k] *= a)
}
// o = x * y
template <int V> __device__ __forceinline__ void mul(const float (&x)[V], const float (&y)[V], float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __fmul2_rn(at2(x, k), at2(y, k))), o[k] = x[k] * y[k])
}
// o += x
template <int V> __device__ __forceinline__ void add_to(const float (&x)[V], float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __fadd2_rn(at2(o, k), at2(x, k))), o[k] += x[k])
}
// o += x * y
template <int V> __device__ __forceinline__ void fma_to(const float (&x)[V], const float (&y)[V], float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __ffma2_rn(at2(x, k), at2(y, k), at2(o, k))), o[k] = fmaf(x[k], y[k], o[k]))
}
// o = x * a + (y * b + c)
template <int V> __device__ __forceinline__ void fma_fma(const float (&x)[V], float a, const float (&y)[V], float b, float c, float (&o)[V]) {
  LOPT_EACH(V, set2(o, k, __ffma2_rn(at2(x, k), two(a), __ffma2_rn(at2(y, k), two(b), two(c)))),
            o[k] = fmaf(x[k], a, fmaf(y[k], b, c)))
}
template <int V> __device__ __forceinline__ float sum_of(const float (&x)[V]) {
  if constexpr (V % 2 == 0) {
    float2 t = at2(x, 0);
#pragma unroll
    for (int k = 2; k < V; k += 2) t = __fadd2_rn(t, at2(x, k));
    return t.x + t.y;
  } else {
    float t = x[0];
#pragma unroll
    for (int k = 1; k < V; ++k) t += x[k];
    return t;
  }
}

constexpr int kFetchBlocks = 256;
__device__ __forceinline__ void fetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__host__ __device__ constexpr int fwd_threads(int L) { return L <= 32 ? 128 : L; }

// L threads per row, each with SLOTS accesses of VEC elements.  Bound by HBM
// bytes: 33.5M float32 elements with a residual take 84.6 us at any width from
// 64 to 2048 (6.3 TB/s, what an elementwise sum of three such arrays takes);
// 16,421 rows of 768 bfloat16 with a residual 21.0 us (4.8 TB/s: launch, first
// loads and last stores are a sixth of it).  Small blocks that take one row
// and end: a persistent form with the next row's loads ahead took 23.1 us
// there, since its few rows per warp do not come out even.
template <typename T, int VEC, int SLOTS, int L, bool RES>
__global__ void __launch_bounds__(fwd_threads(L), 1024 / fwd_threads(L)) k_norm_fwd(const NormFwd a) {
  constexpr int TH = fwd_threads(L), R = TH / L;
  __shared__ float red[L <= 32 ? 1 : L / 32];
  const int lane = threadIdx.x % L;
  const int cols = (int)a.cols;
  const float inv = 1.f / (float)cols;
  int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / L;
  const bool live = row < a.rows;
  if (L >= 32 && !live) return;         // whole warps when L == 32, else never
  if (!live) row = a.rows - 1;          // half a warp: reads, and writes nothing
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* r = RES ? static_cast<const T*>(a.residual) + row * a.rs : nullptr;
  Pack<T, VEC> px[SLOTS], pr[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int j = (s * L + lane) * VEC;
    if (j >= cols) continue;
    px[s] = *reinterpret_cast<const Pack<T, VEC>*>(x + j);
    if (RES) pr[s] = *reinterpret_cast<const Pack<T, VEC>*>(r + j);
  }
  // The weights are wanted after two sums: a small call fetches them from HBM
  // meanwhile (16 rows of 768 float32, all cold: 5.3 us, 5.9 without; 16,421
  // rows, had their first blocks fetched: 22.6 us, 21.1 without).
  if (gridDim.x <= kFetchBlocks) {
    const size_t size = a.wtype == LOPT_F32 ? 4 : sizeof(T);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = (s * L + lane) * VEC;
      if (j >= cols) continue;
      fetch_line(static_cast<const char*>(a.weight) + j * size);
      if (a.bias) fetch_line(static_cast<const char*>(a.bias) + j * size);
    }
  }
  {
    float v[SLOTS][VEC], sum[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum[k] = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      to_floats(px[s], v[s]);
      if (RES) {
        float t[VEC];
        to_floats(pr[s], t);
        add_to(t, v[s]);
      }
      if ((s * L + lane) * VEC < cols) add_to(v[s], sum);
    }
    if (RES && a.summed && live) {
      T* sm = static_cast<T*>(a.summed) + row * a.ss;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int j = (s * L + lane) * VEC;
        if (j < cols) *reinterpret_cast<Pack<T, VEC>*>(sm + j) = from_floats<T, VEC>(v[s]);
      }
    }
    const float mean = row_sum<L>(sum_of(sum), red) * inv;
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum[k] = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      add_one(-mean, v[s]);
      if ((s * L + lane) * VEC < cols) fma_to(v[s], v[s], sum);
    }
    const float rstd = rsqrtf(row_sum<L>(sum_of(sum), red) * inv + a.eps);
    if (lane == 0 && live) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    if (!live) return;
    T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = (s * L + lane) * VEC;
      if (j >= cols) continue;
      float w[VEC];
      load_weights<T, VEC>(a.weight, a.wtype, j, w);
      mul_one(rstd, v[s]);
      mul(v[s], w, w);
      if (a.bias) {
        float b[VEC];
        load_weights<T, VEC>(a.bias, a.wtype, j, b);
        add_to(b, w);
      }
      *reinterpret_cast<Pack<T, VEC>*>(y + j) = from_floats<T, VEC>(w);
    }
  }
}

// Rows too long for registers: one block per row, which reads the row three
// times (from L2 after the first).  1,520 rows of 20,001 bfloat16: 74 us.
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
    float w[1], b[1] = {0.f};
    load_weights<T, 1>(a.weight, a.wtype, j, w);
    if (a.bias) load_weights<T, 1>(a.bias, a.wtype, j, b);
    if (sm) sm[j] = from_f<T>(s);
    y[j] = from_f<T>(fmaf((s - mean) * rstd, w[0], b[0]));
  }
}

// Threads of a backward block, of which an SM takes one: 24 warps of lanes
// with 8 elements of 16 bits (80 registers) where rows take 32 to 256 threads,
// else 16 warps (128 registers): with 64 or 80 registers the others spill
// (bfloat16 with a residual gradient, 8,192 rows of 4096: 74 us with one group
// of 512 threads, 107 with two; 524,288 rows of 64: 130 us with 16 warps, 197
// with 24).
__host__ __device__ constexpr int bwd_threads(int E, int L, int es) {
  return L == 1024 ? 1024 : L % 96 == 0 ? (es == 2 ? 768 : 480) : E <= 8 && es == 2 && L >= 32 && L <= 256 ? 768 : 512;
}

// Persistent: a block's groups of L threads take rows blockIdx.x * R + group,
// striding by gridDim.x * R, and keep the column sums of their columns.  With
// AHEAD, the next row's x and dy are loaded before the current row is reduced;
// with KEEP, xhat and g stay in registers over the reduction, else they are
// made again.  32,768 rows of 2048 bfloat16 with a residual gradient: 98 us
// (5.5 TB/s; 85 us is what an elementwise operation on as many arrays takes).
// Not the loads bound it but a row's chain of sum, barrier and store: rows
// copied to shared memory five ahead 104 to 108 us, pairs of elements per
// instruction 106 to 113 (fewer instructions, more conversions between pairs),
// two groups with all weights in registers 111, 16 elements a thread 118.
template <typename T, int VEC, int SLOTS, int L, bool AHEAD, bool KEEP>
__global__ void __launch_bounds__(bwd_threads(VEC * SLOTS, L, sizeof(T)), 1) k_norm_bwd(const NormBwd a) {
  constexpr int E = VEC * SLOTS, TH = bwd_threads(E, L, sizeof(T)), R = TH / L, W = L * E;
  using P = Pack<T, VEC>;
  __shared__ float2 red[2][TH / 32];
  extern __shared__ __align__(16) float comb[];   // the groups' sums, at the end: [2][R][W]
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int cols = (int)a.cols;
  const float inv = 1.f / (float)cols;
  const int64_t stride = (int64_t)gridDim.x * R;
  const bool res = a.dres != nullptr;
  let_next_start();
  auto in = [&](int s) { return (s * L + lane) * VEC < cols; };
  float dw[SLOTS][VEC], db[SLOTS][VEC];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[s][k] = db[s][k] = 0.f;
  P px[SLOTS], pd[SLOTS];
  float mean = 0.f, rstd = 0.f;
  // A warp that holds two rows goes on while the first is one: the other's
  // lanes then see a row of zeros and write nothing.
  const int second = L < 32 ? group % 2 : 0;
  auto load = [&](int64_t r, P (&x)[SLOTS], P (&d)[SLOTS], float& m, float& rs) {
    if (L < 32 && r >= a.rows) {
      m = rs = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) x[s] = d[s] = P{};
      return;
    }
    const T* xp = static_cast<const T*>(a.x) + r * a.xs + lane * VEC;
    const T* dp = static_cast<const T*>(a.dy) + r * a.dys + lane * VEC;
    m = a.mean[r];
    rs = a.rstd[r];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (!in(s)) continue;
      x[s] = *reinterpret_cast<const P*>(xp + s * L * VEC);
      d[s] = *reinterpret_cast<const P*>(dp + s * L * VEC);
    }
  };
  int64_t row = (int64_t)blockIdx.x * R + group;
  if (row - second < a.rows) load(row, px, pd, mean, rstd);
  for (int par = 0; row - second < a.rows; row += stride, par ^= 1) {
    const bool live = L >= 32 || row < a.rows;
    P pr[SLOTS];
    if (res && live) {
      const T* rp = static_cast<const T*>(a.dres) + row * a.drs + lane * VEC;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
        if (in(s)) pr[s] = *reinterpret_cast<const P*>(rp + s * L * VEC);
    }
    P nx[SLOTS], nd[SLOTS];
    float nmean = 0.f, nrstd = 0.f;
    if (AHEAD && row - second + stride < a.rows) load(row + stride, nx, nd, nmean, nrstd);
    float kx[SLOTS][VEC], kg[SLOTS][VEC];
    auto make = [&](int s, float (&d)[VEC]) {
      float w[VEC];
      load_weights<T, VEC>(a.weight, a.wtype, (s * L + lane) * VEC, w);
      to_floats(px[s], kx[s]);
      to_floats(pd[s], d);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        kx[s][k] = (kx[s][k] - mean) * rstd;
        kg[s][k] = d[k] * w[k];
      }
    };
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (!in(s)) continue;
      float d[VEC];
      make(s, d);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        sg += kg[s][k];
        sgx = fmaf(kg[s][k], kx[s][k], sgx);
        dw[s][k] = fmaf(d[k], kx[s][k], dw[s][k]);
        db[s][k] += d[k];
      }
    }
    const float2 t = group_sum2<L>(make_float2(sg, sgx), red[par], group);
    const float c1 = -rstd * (t.x * inv), c2 = -rstd * (t.y * inv);
    T* op = static_cast<T*>(a.dx) + row * a.dxs + lane * VEC;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (!in(s) || !live) continue;
      float o[VEC];
      if (!KEEP) make(s, o);
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = fmaf(kx[s][k], c2, fmaf(kg[s][k], rstd, c1));
      if (res) {
        float q[VEC];
        to_floats(pr[s], q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] += q[k];
      }
      *reinterpret_cast<P*>(op + s * L * VEC) = from_floats<T, VEC>(o);
    }
    if (AHEAD) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        px[s] = nx[s];
        pd[s] = nd[s];
      }
      mean = nmean;
      rstd = nrstd;
    } else if (row - second + stride < a.rows) {
      load(row + stride, px, pd, mean, rstd);
    }
  }
  // The block's sums: over its groups in order.
  float* pw = a.part + (int64_t)blockIdx.x * cols;
  const int64_t pb = (int64_t)gridDim.x * cols;   // the bias's sums lie so far behind the weight's
  float* to_w = R == 1 ? pw : comb + group * W;
  float* to_b = R == 1 ? pw + pb : comb + (R + group) * W;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      to_w[(s * L + lane) * VEC + k] = dw[s][k];
      to_b[(s * L + lane) * VEC + k] = db[s][k];
    }
  }
  if (R > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * W; c += TH) {
      const int h = c / W, j = c % W;
      if (j >= cols) continue;
      float t = 0.f;
#pragma unroll
      for (int g = 0; g < R; ++g) t += comb[(h * R + g) * W + j];
      pw[h * pb + j] = t;
    }
  }
}

// Rows too long for registers: dx row by row; the column sums are another
// kernel's.  1,520 rows of 20,001 bfloat16: 101 us with those.
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
    float w[1];
    load_weights<T, 1>(a.weight, a.wtype, j, w);
    const float g = to_f(dy[j]) * w[0];
    sg += g;
    sgx = fmaf(g, (to_f(x[j]) - mean) * rstd, sgx);
  }
  const float2 t = group_sum2<L>(make_float2(sg, sgx), red, 0);
  const float inv = 1.f / (float)a.cols;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    float w[1];
    load_weights<T, 1>(a.weight, a.wtype, j, w);
    const float v = rstd * (to_f(dy[j]) * w[0] - t.x * inv - (to_f(x[j]) - mean) * rstd * (t.y * inv));
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

// The blocks' sums of 32 columns: warp w adds blocks w, w + 8, ..., then one
// warp the eight sums in order.  blockIdx.y: 0 the weight's, 1 the bias's.  One
// latency, all of a warp's loads side by side: 5.5 us for 152 blocks' sums of
// 2048 columns, set up while the kernel before it still runs.
__global__ void __launch_bounds__(256) k_norm_finish(const float* part, int blocks, int64_t cols, float* dw, float* db,
                                                     int accumulate) {
  __shared__ float red[8][32];
  float* out = blockIdx.y ? db : dw;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  const float* p = part + (int64_t)blockIdx.y * blocks * cols + j;
  wait_for_previous();
  float t = 0.f;
  if (j < cols) {
    constexpr int U = 20;   // 152 blocks in one go
    for (int b0 = w; b0 < blocks; b0 += 8 * U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = b0 + 8 * u < blocks ? __ldcg(p + (int64_t)(b0 + 8 * u) * cols) : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) t += v[u];
    }
  }
  red[w][lane] = t;
  __syncthreads();
  if (w == 0 && j < cols) {
    t = red[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) t += red[k][lane];
    out[j] = accumulate ? out[j] + t : t;
  }
}

// ---- choice of the kernel -------------------------------------------------------
constexpr int kMaxBlocks = 192;   // blocks' sums in the workspace

template <typename T, int VEC, int SLOTS, int L>
cudaError_t fwd_as(const NormFwd& a, cudaStream_t s) {
  constexpr int R = fwd_threads(L) / L;
  const int64_t grid = (a.rows + R - 1) / R;
  return launch(a.residual ? k_norm_fwd<T, VEC, SLOTS, L, true> : k_norm_fwd<T, VEC, SLOTS, L, false>, dim3((unsigned)grid),
                dim3(fwd_threads(L)), 0, s, false, 1, a);
}

template <typename T, int VEC, int SLOTS, int L>
cudaError_t bwd_as(const NormBwd& a, int sms, cudaStream_t s, int* blocks) {
  constexpr int E = VEC * SLOTS, TH = bwd_threads(E, L, sizeof(T)), R = TH / L;
  constexpr bool kAhead = VEC > 1 && E <= 16, kKeep = VEC > 1 && E <= 8;   // what the registers hold beside the sums
  const size_t smem = R > 1 ? (size_t)TH * E * 8 : 0;
  auto* k = &k_norm_bwd<T, VEC, SLOTS, L, kAhead, kKeep>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  *blocks = (int)std::min<int64_t>({(a.rows + R - 1) / R, (int64_t)sms, kMaxBlocks});
  return launch(k, dim3((unsigned)*blocks), dim3(TH), smem, s, false, 1, a);
}

// Threads and slots for rows of nvec accesses of VEC elements: half a warp
// for the shortest, then as few threads as keep 8 elements each (the forward
// direction in 16 bits: a warp up to 24), for wide rows 16 where that leaves an
// SM several rows (forward, and backward in float32: in 16 bits its loads a row
// ahead and xhat in registers count for more); then 512 threads with 32
// elements each; longer rows are read again.  33.5M elements with a residual,
// us: forward, rows of 128 bfloat16 by half warps 48, by warps 74; of 768
// float32 by 96 threads 85, by 256 117; of 4512 by 384 threads with 16 elements
// 60 bfloat16, 91 float32, by 1024 with 8 136, 158; backward, rows of 768
// bfloat16 by 96 threads 62, by 128 69; of 3000 by 384 68, by 512 83; of 4512
// by 768 threads with 8 elements 88, by 512 with 16 117 (float32: 137 with 16,
// 178 with 8).
#define LOPT_NORM_CASE(V, S, L_) if (nvec <= (int64_t)(S) * (L_)) return f.template run<V, S, L_>()
template <int FULL, typename F>
cudaError_t pick(int64_t cols, bool vec, F f) {
  if (vec) {
    const int64_t nvec = (cols + FULL - 1) / FULL;
    constexpr int B = 8 / FULL;   // slots of 8 elements
    if constexpr (F::kForward && FULL == 8) {
      LOPT_NORM_CASE(FULL, 1, 16);
      LOPT_NORM_CASE(FULL, 1, 32);
      LOPT_NORM_CASE(FULL, 2, 32);
      LOPT_NORM_CASE(FULL, 3, 32);
      LOPT_NORM_CASE(FULL, 2, 64);
    } else if constexpr (F::kForward) {
      LOPT_NORM_CASE(FULL, 1, 16);
      LOPT_NORM_CASE(FULL, 1, 32);
      LOPT_NORM_CASE(FULL, B, 32);
      LOPT_NORM_CASE(FULL, B, 64);
      LOPT_NORM_CASE(FULL, B, 96);
      LOPT_NORM_CASE(FULL, B, 128);
    } else {
      LOPT_NORM_CASE(FULL, 1, 16);
      LOPT_NORM_CASE(FULL, 1, 32);
      LOPT_NORM_CASE(FULL, B, 32);
      LOPT_NORM_CASE(FULL, B, 64);
      LOPT_NORM_CASE(FULL, B, 96);
      LOPT_NORM_CASE(FULL, B, 128);
    }
    LOPT_NORM_CASE(FULL, B, 256);
    if constexpr (F::kForward) {
      LOPT_NORM_CASE(FULL, 2 * B, 192);
      LOPT_NORM_CASE(FULL, 2 * B, 256);
      LOPT_NORM_CASE(FULL, 2 * B, 384);
      LOPT_NORM_CASE(FULL, 2 * B, 512);
    } else if constexpr (FULL == 8) {
      LOPT_NORM_CASE(FULL, B, 384);
      LOPT_NORM_CASE(FULL, B, 512);
      LOPT_NORM_CASE(FULL, B, 768);
      LOPT_NORM_CASE(FULL, B, 1024);
    } else {
      LOPT_NORM_CASE(FULL, 2 * B, 256);
      LOPT_NORM_CASE(FULL, 2 * B, 512);
    }
    LOPT_NORM_CASE(FULL, 4 * B, 512);
  } else {
    const int64_t nvec = cols;
    LOPT_NORM_CASE(1, 4, 32);
    LOPT_NORM_CASE(1, 8, 32);
    LOPT_NORM_CASE(1, 16, 32);
    LOPT_NORM_CASE(1, 8, 128);
    LOPT_NORM_CASE(1, 8, 256);
    LOPT_NORM_CASE(1, 8, 512);
    LOPT_NORM_CASE(1, 16, 512);
    LOPT_NORM_CASE(1, 32, 512);
  }
  return f.long_rows();
}

template <typename T> struct FwdRun {
  static constexpr bool kForward = true;
  const NormFwd& a;
  cudaStream_t s;
  template <int V, int S, int L> cudaError_t run() { return fwd_as<T, V, S, L>(a, s); }
  cudaError_t long_rows() {
    return launch(k_norm_fwd_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
  }
};

template <typename T> struct BwdRun {
  static constexpr bool kForward = false;
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
bool vec_ok(int64_t cols, int es, std::initializer_list<Span> ms, const void* w, const void* b) {
  if ((cols * es) % 16) return false;
  for (const Span& m : ms)
    if (!rows_aligned(m, 16)) return false;
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
  const bool vec = vec_ok(cols, es, {mx, mr, my, ms}, weight, bias);
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
  const bool vec = vec_ok(cols, es, {md, mx, mr, mo}, weight, nullptr);
  const int sms = sm_count();
  int blocks = 0;
  cudaError_t e;
  switch (type) {
    case LOPT_F32: e = pick<4>(cols, vec, BwdRun<float>{a, sms, s, &blocks}); break;
    case LOPT_F16: e = pick<8>(cols, vec, BwdRun<__half>{a, sms, s, &blocks}); break;
    default: e = pick<8>(cols, vec, BwdRun<__nv_bfloat16>{a, sms, s, &blocks}); break;
  }
  if (e != cudaSuccess) return done(e);
  return done(launch(k_norm_finish, dim3((unsigned)((cols + 31) / 32), grad_bias ? 2u : 1u), dim3(256), 0, s, true, 1,
                     (const float*)workspace, blocks, cols, grad_weight, grad_bias, accumulate));
}

}  // extern "C"
