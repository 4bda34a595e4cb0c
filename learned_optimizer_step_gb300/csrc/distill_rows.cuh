// Distillation from a teacher's top logits: the loss of a row and its
// gradient (see lopt_train.h).
//
// With m = max z and s = sum exp((z - m) / T), log q_j = (z_j - m) / T - log s.
// The exponents are taken of z - m, not of z / T - m / T: masks of the type's
// lowest value stay finite that way, and the terms near the maximum exact.
// The dense part of the gradient, w T q_j, is written for every column and
// the listed columns are then written again with their p taken off.
#pragma once

#include <algorithm>

#include "train_common.cuh"

namespace lopt {
namespace train {
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

// One per element type, each in a source of its own (they compile side by side).
cudaError_t distill_f32(const Distill& a, int sms, cudaStream_t s);
cudaError_t distill_f16(const Distill& a, int sms, cudaStream_t s);
cudaError_t distill_bf16(const Distill& a, int sms, cudaStream_t s);

#ifdef LOPT_DISTILL_KERNELS
namespace {

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

// ---- 16 bytes of a row ---------------------------------------------------------
// Rows start where they start: a 50257-wide row of 2-byte logits begins on any
// even address.  So a row is taken as the aligned 16-byte slots that cover
// it; only its first and last slot can hold foreign elements, and those two
// are read and written element by element.
template <typename T> struct Slots;
template <> struct Slots<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int k) {   // elements 2k, 2k + 1
    return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
  }
  static __device__ __forceinline__ void put(uint32_t* w, int k, float2 v) {
    w[2 * k] = __float_as_uint(v.x);
    w[2 * k + 1] = __float_as_uint(v.y);
  }
  static __device__ __forceinline__ float max_of(const uint32_t* w, float m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, __uint_as_float(w[k]));
    return m;
  }
};
template <> struct Slots<__half> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int k) { return __half22float2(h2(w[k])); }
  static __device__ __forceinline__ void put(uint32_t* w, int k, float2 v) {
    const __half2 h = __float22half2_rn(v);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float max_of(const uint32_t* w, float m) {
    const __half2 t = __hmax2(__hmax2(h2(w[0]), h2(w[1])), __hmax2(h2(w[2]), h2(w[3])));
    return fmaxf(m, fmaxf(__low2float(t), __high2float(t)));
  }
};
template <> struct Slots<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ __nv_bfloat162 b2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
  static __device__ __forceinline__ float2 pair(const uint32_t* w, int k) {
    return make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  }
  static __device__ __forceinline__ void put(uint32_t* w, int k, float2 v) {
    const __nv_bfloat162 b = __float22bfloat162_rn(v);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  static __device__ __forceinline__ float max_of(const uint32_t* w, float m) {
    const __nv_bfloat162 t = __hmax2(__hmax2(b2(w[0]), b2(w[1])), __hmax2(b2(w[2]), b2(w[3])));
    return fmaxf(m, fmaxf(__low2float(t), __high2float(t)));
  }
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void put_pair(uint32_t addr, int rank, float m, float s) {   // into block `rank` of the cluster
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(remote), "f"(m), "f"(s) : "memory");
}

constexpr int kMaxCluster = 8;

// The dense part's factor 2^((z - m) log2e / T) of two elements.
__device__ __forceinline__ float2 ex2_pair(float2 z, float neg_m, float c) {
  const float2 d = __fmul2_rn(__fadd2_rn(z, make_float2(neg_m, neg_m)), make_float2(c, c));
  return make_float2(ex2(d.x), ex2(d.y));
}

// One row per group of G threads (a warp, or the block), or per cluster of C
// blocks whose slices follow each other.  A thread holds NV slots of 16 bytes
// of the row in registers from the first read to the gradient's store, so
// memory is touched once each way.  The one exchange is of (m, s): every
// warp takes its own maximum and its sum about that, and all pairs of the
// row meet in shared memory (every block's copy, written across the cluster).
template <typename T, int NV, int G, bool GRAD>
__global__ void __launch_bounds__(G == 32 ? 256 : G, G == 512 ? 2 : 4) k_distill(const Distill a, const int C) {
  using S = Slots<T>;
  constexpr int N = S::N, GW = G / 32;                  // warps of a group
  constexpr int TH = G == 32 ? 256 : G, ROWS = TH / G;
  extern __shared__ int32_t lists[];                    // per group: class, p, z, teacher's logit of the slots
  __shared__ float2 pairs[ROWS][GW * kMaxCluster];      // (m, s) of the row's warps
  const int lane = threadIdx.x % 32, t = threadIdx.x % G, group = threadIdx.x / G, gw = t / 32;
  const int rank = G == 32 || C == 1 ? 0 : (int)cluster_rank();
  if (G != 32 && C > 1) cluster_arrive();               // that all blocks of the row run, before their memory is written
  const int64_t row = G == 32 ? (int64_t)blockIdx.x * ROWS + group : (int64_t)(blockIdx.x / (unsigned)C);
  if (row >= a.rows) return;                            // whole warps of a one-warp group
  const T* z = static_cast<const T*>(a.logits) + row * a.ls;
  T* g = GRAD ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
  const int cols = (int)a.cols;
  const int mis = (int)(((uintptr_t)z / sizeof(T)) % N);
  const uint4* z16 = reinterpret_cast<const uint4*>(z - mis);
  const int total = (mis + cols + N - 1) / N;           // slots that cover the row
  const int per = (total + C - 1) / C, beg = rank * per, end = min(beg + per, total);
  int32_t* id = lists + group * a.top * 4;
  float* p = reinterpret_cast<float*>(id + a.top);
  float* zi = p + a.top;
  float* tl = zi + a.top;
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  const bool same = !GRAD || (int)(((uintptr_t)g / sizeof(T)) % N) == mis;   // grad's rows start alike

  // The slot at index q of the row: whole, or element by element.
  auto whole = [&](int q) { return q * N >= mis && (q + 1) * N <= mis + cols; };
  auto store = [&](int q, const uint32_t v[4]) {
    if (same && whole(q)) {
      reinterpret_cast<uint4*>(g - mis)[q] = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      const T* e = reinterpret_cast<const T*>(v);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int j = q * N + k - mis;
        if (j >= 0 && j < cols) g[j] = e[k];
      }
    }
  };
  auto zero_row = [&]() {
    if (rank == 0 && t == 0) a.loss[row] = 0.f;
    if (GRAD) {
      const uint32_t v[4] = {0, 0, 0, 0};
      for (int q = beg + t; q < end; q += G) store(q, v);
    }
  };
  if (w == 0.f) {   // the same for all blocks of the row
    if (G != 32 && C > 1) cluster_wait();
    zero_row();
    return;
  }

  uint32_t v[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = beg + i * G + t;
    if (q < end && whole(q)) {
      const uint4 x = z16[q];
      v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = S::kNegInf;
      if (q < end) {
        T* e = reinterpret_cast<T*>(v[i]);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int j = q * N + k - mis;
          if (j >= 0 && j < cols) e[k] = z[j];
        }
      }
    }
  }

  // The teacher's list, one slot per thread, beside the row's loads.
  for (int k = t; k < a.top; k += G) {
    const int64_t i = load_index(a.top_index, row * a.is + k, a.itype);
    const float tk = load_as_f(a.top_logits, row * a.ts + k, a.ttype);
    if (i >= a.cols && a.status && rank == 0) atomicOr(a.status, 1);
    const bool counts = i >= 0 && i < a.cols && tk != -INFINITY;
    id[k] = counts ? (int32_t)i : -1;
    tl[k] = tk;
    if (counts) zi[k] = to_f(z[i]);
  }

  // This warp's maximum, and its sum about it (about 0 where all is masked).
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) m = S::max_of(v[i], m);
  m = warp_max(m);
  float neg_m = m == -INFINITY ? 0.f : -m;
  const float c = a.log2e_t;
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < N / 2; ++k) s2 = __fadd2_rn(s2, ex2_pair(S::pair(v[i], k), neg_m, c));
  float s = warp_sum(s2.x + s2.y);
  if (G == 32) {
    __syncwarp();
  } else {
    if (C == 1) {
      if (lane == 0) pairs[0][gw] = make_float2(m, s);
      __syncthreads();
    } else {
      cluster_wait();
      if (lane < C) put_pair(smem_addr(&pairs[0][rank * GW + gw]), lane, m, s);
      cluster_arrive();
      cluster_wait();
    }
    // Every warp joins all pairs, in the same order.
    const int n = GW * C;
    float mj = -INFINITY, sj = 0.f;
    float2 q[GW * kMaxCluster / 32 > 0 ? GW * kMaxCluster / 32 : 1];
#pragma unroll
    for (int k = 0; k < (int)(sizeof(q) / sizeof(q[0])); ++k) {
      q[k] = k * 32 + lane < n ? pairs[0][k * 32 + lane] : make_float2(-INFINITY, 0.f);
      mj = fmaxf(mj, q[k].x);
    }
    m = warp_max(mj);
#pragma unroll
    for (int k = 0; k < (int)(sizeof(q) / sizeof(q[0])); ++k)
      if (k * 32 + lane < n) sj += q[k].y * ex2((q[k].x - m) * c);
    s = warp_sum(sj);
    neg_m = -m;
  }
  // The teacher's softmax: every warp its maximum and sum, each thread the p
  // of its own slots.
  float tmax = -INFINITY, ps = 0.f;
  bool any = false;
  for (int k = lane; k < a.top; k += 32) {
    if (id[k] < 0) continue;
    any = true;
    tmax = fmaxf(tmax, tl[k]);
  }
  if (!__any_sync(0xffffffffu, any)) {   // nothing to learn from this row
    zero_row();
    return;
  }
  tmax = warp_max(tmax);
  for (int k = lane; k < a.top; k += 32)
    if (id[k] >= 0) ps += ex2((tl[k] - tmax) * c);
  ps = warp_sum(ps);
  const float inv_ps = 1.f / ps;
  if (rank == 0 && gw == 0) {
    const float log_s = logf(s), log_ps = logf(ps);
    float kl = 0.f;
    for (int k = lane; k < a.top; k += 32) {
      if (id[k] < 0) continue;
      const float d = tl[k] - tmax, pk = ex2(d * c) * inv_ps;
      if (pk == 0.f) continue;   // 0 log 0 = 0
      kl += pk * ((d * a.inv_t - log_ps) - ((zi[k] - m) * a.inv_t - log_s));
    }
    kl = warp_sum(kl);
    if (lane == 0) a.loss[row] = w * a.temperature * a.temperature * kl;
  }
  if (!GRAD) return;
  const float wt = w * a.temperature, f = wt / s;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = beg + i * G + t;
    if (q >= end) continue;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < N / 2; ++k)
      S::put(o, k, __fmul2_rn(ex2_pair(S::pair(v[i], k), neg_m, c), make_float2(f, f)));
    store(q, o);
  }
  for (int k = t; k < a.top; k += G) p[k] = id[k] < 0 ? 0.f : ex2((tl[k] - tmax) * c) * inv_ps;
  if (G == 32) __syncwarp();
  else __syncthreads();
  // The listed classes of this slice, again: a class listed more than once
  // by its first slot, with the sum of its p.
  for (int k = t; k < a.top; k += G) {
    const int j = id[k];
    const int q = (j + mis) / N;
    if (j < 0 || q < beg || q >= end) continue;
    bool first = true;
    float pk = 0.f;
#pragma unroll 4
    for (int o = 0; o < a.top; ++o) {
      const bool same_class = id[o] == j;
      first &= !same_class || o >= k;
      pk += same_class ? p[o] : 0.f;
    }
    if (first) g[j] = from_f<T>(fmaf(ex2((zi[k] - m) * c), f, -wt * pk));
  }
}

// Rows beyond a cluster's registers: one block per row, which is read for
// each of the three passes.
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

// ---- choice of the kernel -------------------------------------------------------
template <typename T, int NV, int G>
cudaError_t rows_as(const Distill& a, int C, cudaStream_t s) {
  constexpr int ROWS = G == 32 ? 8 : 1;
  const int64_t grid = G == 32 ? (a.rows + 7) / 8 : a.rows * C;
  const size_t smem = (size_t)ROWS * a.top * 4 * 4;
  const dim3 block(G == 32 ? 256 : G);
  if (a.grad) return launch(k_distill<T, NV, G, true>, dim3((unsigned)grid), block, smem, s, false, C, a, C);
  return launch(k_distill<T, NV, G, false>, dim3((unsigned)grid), block, smem, s, false, C, a, C);
}

// NV is the next of these that holds a thread's slots.
template <typename T, int G>
cudaError_t rows_with(const Distill& a, int64_t nv, int C, cudaStream_t s) {
  if constexpr (G == 512) return nv <= 6 ? rows_as<T, 6, G>(a, C, s) : rows_as<T, 8, G>(a, C, s);
  if (nv <= 1) return rows_as<T, 1, G>(a, C, s);
  if (nv <= 2) return rows_as<T, 2, G>(a, C, s);
  if (nv <= 3) return rows_as<T, 3, G>(a, C, s);
  if (nv <= 4) return rows_as<T, 4, G>(a, C, s);
  if constexpr (G == 256) {
    if (nv <= 5) return rows_as<T, 5, G>(a, C, s);
  }
  if (nv <= 6) return rows_as<T, 6, G>(a, C, s);
  if constexpr (G == 256) {
    if (nv <= 7) return rows_as<T, 7, G>(a, C, s);
  }
  return rows_as<T, 8, G>(a, C, s);
}

template <typename T>
cudaError_t distill_rows(const Distill& a, int sms, cudaStream_t s) {
  constexpr int N = Slots<T>::N, kMaxNV = 8;
  // Most slots that cover a row, wherever it starts.
  const bool aligned = (uintptr_t)a.logits % 16 == 0 && (a.rows == 1 || (a.ls * (int64_t)sizeof(T)) % 16 == 0);
  const int64_t slots = (a.cols + (aligned ? 0 : N - 1) + N - 1) / N;
  auto ceil = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  if (slots <= 32 * kMaxNV && a.top <= 256) return rows_with<T, 32>(a, ceil(slots, 32), 1, s);
  int C = 1;
  while (C < kMaxCluster && ceil(slots, C) > 256 * kMaxNV) C *= 2;
  // Few rows: more blocks for each, while they have a slot per thread.
  while (C < kMaxCluster && a.rows * C < sms && ceil(slots, 2 * C) >= 256) C *= 2;
  if (a.rows * C < kMaxRows) {
    if (ceil(slots, C) <= 256 * kMaxNV) return rows_with<T, 256>(a, ceil(ceil(slots, C), 256), C, s);
    if (ceil(slots, C) <= 512 * kMaxNV) return rows_with<T, 512>(a, ceil(ceil(slots, C), 512), C, s);
  }
  return launch(k_distill_rows<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
}

}  // namespace
#endif
}  // namespace train
}  // namespace lopt
