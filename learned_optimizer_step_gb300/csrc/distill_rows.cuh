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

#include "tc_layout.cuh"
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

// The maximum, which keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
  template <int U> static __device__ __forceinline__ float max_of(const uint32_t (&v)[U][4]) {
    float m = __uint_as_float(v[0][0]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) m = max_nan(m, __uint_as_float(v[u][k]));
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
  template <int U> static __device__ __forceinline__ float max_of(const uint32_t (&v)[U][4]) {
    __half2 t = h2(v[0][0]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) t = __hmax2_nan(t, h2(v[u][k]));
    return max_nan(__low2float(t), __high2float(t));
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
  template <int U> static __device__ __forceinline__ float max_of(const uint32_t (&v)[U][4]) {
    __nv_bfloat162 t = b2(v[0][0]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) t = __hmax2_nan(t, b2(v[u][k]));
    return max_nan(__low2float(t), __high2float(t));
  }
};

// Sums of 2^((z - m) c) over slots, m a running maximum: one thread's part.
//
// The exponent is fma(z, c, -mc) with mc = m c rounded once; `fix` takes off
// what that rounding left, so the sum is about m exactly.  Where m c could
// overflow (rows of the type's lowest value), (z - m) c is taken instead,
// which is slower by an addition.
constexpr float kSafe = 1e38f;

template <typename T> struct Partial {
  float m = -INFINITY, s = 0.f;

  template <int U> __device__ __forceinline__ void add(const uint32_t (&v)[U][4], float c) {
    using S = Slots<T>;
    const float top = S::template max_of<U>(v);
    if (!(top <= m)) {   // a NaN too
      if (s != 0.f) s *= ex2((m - top) * c);
      m = top;
    }
    if (m == -INFINITY) return;   // nothing but -inf so far
    const float mc = m * c;
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (fabsf(mc) <= kSafe) {
      const float2 c2 = make_float2(c, c), n2 = make_float2(-mc, -mc);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < S::N / 2; ++k) {
          const float2 d = __ffma2_rn(S::pair(v[u], k), c2, n2);
          acc[k & 1] = __fadd2_rn(acc[k & 1], make_float2(ex2(d.x), ex2(d.y)));
        }
      acc[0] = __fadd2_rn(acc[0], acc[1]);
      s = fmaf(acc[0].x + acc[0].y, ex2(-fmaf(m, c, -mc)), s);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < S::N / 2; ++k) {
          const float2 z = S::pair(v[u], k);
          s += ex2((z.x - m) * c) + ex2((z.y - m) * c);
        }
    }
  }
};

// Joins the lanes' (m, s): all lanes end with the same.  A part with m ==
// -inf is empty.
__device__ __forceinline__ void join_warp(float& m, float& s, float c) {
  const float top = warp_max(m);
  s = warp_sum(m == -INFINITY ? s : s * ex2((m - top) * c));
  m = top;
}

// f 2^((z - m) c) for the slots of a row, by the same two forms.
template <typename T> struct Dense {
  float m, c, mc, f, f_fast;
  bool fast;
  __device__ __forceinline__ Dense(float m_, float c_, float f_) : m(m_), c(c_), mc(m_ * c_), f(f_) {
    fast = fabsf(mc) <= kSafe;
    f_fast = f * ex2(-fmaf(m, c, -mc));
  }
  __device__ __forceinline__ void of(const uint32_t v[4], uint32_t o[4]) const {
    using S = Slots<T>;
    if (fast) {
#pragma unroll
      for (int k = 0; k < S::N / 2; ++k) {
        const float2 d = __ffma2_rn(S::pair(v, k), make_float2(c, c), make_float2(-mc, -mc));
        S::put(o, k, __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)), make_float2(f_fast, f_fast)));
      }
    } else {
#pragma unroll
      for (int k = 0; k < S::N / 2; ++k) {
        const float2 z = S::pair(v, k);
        S::put(o, k, make_float2(ex2((z.x - m) * c) * f, ex2((z.y - m) * c) * f));
      }
    }
  }
};

// The part of a row that a group of threads holds: slots [beg, beg + cnt) of
// the aligned 16-byte slots that cover the row.
template <typename T> struct Slice {
  static constexpr int N = Slots<T>::N;
  const T* z;
  T* g;
  int cols, mis, beg, cnt;
  int first, last;     // the slice's slots that are not whole, or -1
  bool same;           // the gradient's row starts alike
  __device__ __forceinline__ Slice(const Distill& a, int64_t row, int rank, int C) {
    z = static_cast<const T*>(a.logits) + row * a.ls;
    g = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
    cols = (int)a.cols;
    mis = (int)(((uintptr_t)z / sizeof(T)) % N);
    const int total = (mis + cols + N - 1) / N, per = (total + C - 1) / C;
    beg = min(rank * per, total);
    cnt = min(per, total - beg);
    same = (int)(((uintptr_t)g / sizeof(T)) % N) == mis;
    first = beg == 0 && cnt > 0 && (mis > 0 || cols < N) ? 0 : -1;
    last = cnt > 0 && beg + cnt == total && (mis + cols) % N ? cnt - 1 : -1;
  }
  __device__ __forceinline__ const uint4* z16() const { return reinterpret_cast<const uint4*>(z - mis) + beg; }
  __device__ __forceinline__ bool whole(int q) const { return q != first && q != last; }
  // A slot that is not whole, -inf outside the row.
  __device__ __forceinline__ void read_edge(int q, uint32_t v[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = Slots<T>::kNegInf;
    T* e = reinterpret_cast<T*>(v);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int j = (beg + q) * N + k - mis;
      if (j >= 0 && j < cols) e[k] = z[j];
    }
  }
  __device__ __forceinline__ void write(int q, const uint32_t v[4]) const {
    if (same && whole(q)) {
      reinterpret_cast<uint4*>(g - mis)[beg + q] = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      const T* e = reinterpret_cast<const T*>(v);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int j = (beg + q) * N + k - mis;
        if (j >= 0 && j < cols) g[j] = e[k];
      }
    }
  }
  __device__ __forceinline__ bool holds(int j) const {   // column j
    const int q = (j + mis) / N - beg;
    return j >= 0 && q >= 0 && q < cnt;
  }
};

// One slot of the teacher's list: its class (-1: does not count) and logit.
__device__ __forceinline__ void load_top(const Distill& a, int64_t row, int k, bool report, int32_t& id, float& t) {
  const int64_t i = load_index(a.top_index, row * a.is + k, a.itype);
  t = load_as_f(a.top_logits, row * a.ts + k, a.ttype);
  if (i >= a.cols && a.status && report) atomicOr(a.status, kStatusIndex);
  id = i >= 0 && i < a.cols && t != -INFINITY ? (int32_t)i : -1;
}

// The teacher's maximum and sum over a list in shared memory, by one warp;
// false if no slot counts.
__device__ __forceinline__ bool top_softmax(const int32_t* id, const float* tl, int top, float c, float& tmax, float& ps) {
  const int lane = threadIdx.x % 32;
  bool any = false;
  tmax = -INFINITY;
  ps = 0.f;
  for (int k = lane; k < top; k += 32) {
    if (id[k] < 0) continue;
    any = true;
    tmax = fmaxf(tmax, tl[k]);
  }
  if (!__any_sync(0xffffffffu, any)) return false;
  tmax = warp_max(tmax);
  for (int k = lane; k < top; k += 32)
    if (id[k] >= 0) ps += ex2((tl[k] - tmax) * c);
  ps = warp_sum(ps);
  return true;
}

// The row's loss, by one warp.
__device__ __forceinline__ float top_loss(const Distill& a, const int32_t* id, const float* tl, const float* zi, float tmax,
                                          float ps, float m, float s) {
  const float log_s = logf(s), log_ps = logf(ps), inv_ps = 1.f / ps;
  float kl = 0.f;
  for (int k = threadIdx.x % 32; k < a.top; k += 32) {
    if (id[k] < 0) continue;
    const float d = tl[k] - tmax, pk = ex2(d * a.log2e_t) * inv_ps;
    if (pk == 0.f) continue;   // 0 log 0 = 0
    kl += pk * ((d * a.inv_t - log_ps) - ((zi[k] - m) * a.inv_t - log_s));
  }
  return warp_sum(kl) * a.temperature * a.temperature;
}

// The gradient of slot k's class, if slot k is the first that lists it.
__device__ __forceinline__ bool top_grad(const Distill& a, const int32_t* id, const float* p, const float* zi, int k, float m,
                                         float f, float wt, float& v) {
  const int j = id[k];
  bool first = true;
  float pk = 0.f;
#pragma unroll 4
  for (int o = 0; o < a.top; ++o) {
    const bool alike = id[o] == j;
    first &= !alike || o >= k;
    pk += alike ? p[o] : 0.f;
  }
  v = fmaf(ex2((zi[k] - m) * a.log2e_t), f, -wt * pk);
  return first;
}

// ---- short rows: a warp per row ----------------------------------------------------
// The row stays in registers, NV slots per lane.
template <typename T, int NV, bool GRAD>
__global__ void __launch_bounds__(256) k_distill_warp(const Distill a) {
  using S = Slots<T>;
  extern __shared__ int32_t lists[];                    // per warp: class, p, z, teacher's logit of the slots
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * 8 + warp;
  if (row >= a.rows) return;
  int32_t* id = lists + warp * a.top * 4;
  float* p = reinterpret_cast<float*>(id + a.top);
  float* zi = p + a.top;
  float* tl = zi + a.top;
  const Slice<T> r(a, row, 0, 1);
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  uint32_t v[NV][4];
  float tmax, ps;
  bool learn = w != 0.f;
  if (learn) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = i * 32 + lane;
      if (q < r.cnt && r.whole(q)) {
        const uint4 x = r.z16()[q];
        v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
      } else if (q < r.cnt) {
        r.read_edge(q, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = S::kNegInf;
      }
    }
    for (int k = lane; k < a.top; k += 32) {
      load_top(a, row, k, true, id[k], tl[k]);
      if (id[k] >= 0) zi[k] = to_f(r.z[id[k]]);
    }
    __syncwarp();
    learn = top_softmax(id, tl, a.top, a.log2e_t, tmax, ps);
  }
  if (!learn) {
    if (lane == 0) a.loss[row] = 0.f;
    if (GRAD) {
      const uint32_t o[4] = {0, 0, 0, 0};
      for (int q = lane; q < r.cnt; q += 32) r.write(q, o);
    }
    return;
  }
  const float c = a.log2e_t;
  Partial<T> part;
  part.template add<NV>(v, c);
  float m = part.m, s = part.s;
  join_warp(m, s, c);
  const float loss = top_loss(a, id, tl, zi, tmax, ps, m, s);
  if (lane == 0) a.loss[row] = w * loss;
  if (!GRAD) return;
  const float wt = w * a.temperature, f = wt / s, inv_ps = 1.f / ps;
  const Dense<T> dense(m, c, f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = i * 32 + lane;
    if (q >= r.cnt) continue;
    uint32_t o[4];
    dense.of(v[i], o);
    r.write(q, o);
  }
  for (int k = lane; k < a.top; k += 32) p[k] = id[k] < 0 ? 0.f : ex2((tl[k] - tmax) * c) * inv_ps;
  __syncwarp();
  for (int k = lane; k < a.top; k += 32) {
    float g;
    if (id[k] >= 0 && top_grad(a, id, p, zi, k, m, f, wt, g)) r.g[id[k]] = from_f<T>(g);
  }
}

// ---- long rows: a block, or a cluster of blocks, per row -----------------------------
constexpr int kMaxCluster = 8;
constexpr uint64_t kWaitNs = 1000000000ull;   // 1 s: a wait that long has failed

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// (m, s) into block `rank` of the cluster, counted on its barrier.
__device__ __forceinline__ void send_pair(const float2* at, const uint64_t* bar, int rank, float m, float s) {
  uint32_t ra, rb;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
               :: "r"(ra), "r"(__float_as_uint(m)), "r"(__float_as_uint(s)), "r"(rb) : "memory");
}

// Persistent: cluster i takes rows i, i + clusters, ...  Each block's slice
// of the next row lands in shared memory by a bulk copy, issued as soon as
// the last read of the current row is done, so that loads run while the
// block still stores and another block of the SM computes.  A thread reads
// its slots twice: for its part of (m, s), and for the dense gradient.
//
// Hand-offs, per row: the block barrier after the sums publishes the lists
// and (one block per row) the warps' pairs; the barrier after the dense part
// frees the landing buffer and publishes p.  Between blocks only the pairs
// move, by stores that count on the receiver's barrier; two sets of pairs
// alternate, and a block cannot be two rows ahead of another, since it needs
// the other's pairs for the row between.  Every block of a cluster sees the
// same rows and weights and so makes the same number of exchanges.
template <typename T, int TH, bool GRAD>
__global__ void __launch_bounds__(TH, 1024 / TH) k_distill_ring(const Distill a, const int C, const int slice_slots) {
  using S = Slots<T>;
  constexpr int GW = TH / 32, U = 4;
  extern __shared__ __align__(128) unsigned char sm[];
  uint4* buf = reinterpret_cast<uint4*>(sm);
  int32_t* ids = reinterpret_cast<int32_t*>(sm + (size_t)slice_slots * 16);   // [2][top]: rows alternate
  float* zis = reinterpret_cast<float*>(ids + 2 * a.top);                      // [2][top]
  float* tl = zis + 2 * a.top;
  float* p = tl + a.top;
  __shared__ float2 pairs[2][GW * kMaxCluster];
  __shared__ uint64_t full, xch[2];
  __shared__ int gave_up;
  const int t = threadIdx.x, lane = t % 32, gw = t / 32;
  const int rank = C == 1 ? 0 : (int)cluster_rank();
  const int64_t clusters = gridDim.x / (unsigned)C;
  int64_t row = blockIdx.x / (unsigned)C;
  if (t == 0) {
    mbar_init(&full, 1);
    mbar_init(&xch[0], 1);
    mbar_init(&xch[1], 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (C > 1) cluster_sync();

  // The whole slots of a row's slice, by one thread, once the buffer is free.
  auto fetch = [&](int64_t r) {
    const Slice<T> n(a, r, rank, C);
    const int lo = n.first == 0 ? 1 : 0, hi = n.last >= 0 ? n.last : n.cnt;
    const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16 : 0;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // after the block's reads of the last row
    mbar_arrive_expect_tx(&full, bytes);
    if (bytes) bulk_g2s(buf + lo, n.z16() + lo, bytes, &full);
  };
  auto weight = [&](int64_t r) { return r >= a.rows ? 0.f : a.row_weight ? a.row_weight[r] : 1.f; };

  float w = weight(row);
  int32_t next_id = -1;
  float next_t = 0.f;
  if (w != 0.f) {
    if (t == 0) fetch(row);
    if (t < a.top) load_top(a, row, t, rank == 0, next_id, next_t);
  }
  uint32_t fetched = 0, exchanged = 0;
  const float c = a.log2e_t;
  for (int par = 0; row < a.rows; par ^= 1) {
    const int64_t next = row + clusters;
    const float w_next = weight(next);
    const Slice<T> r(a, row, rank, C);
    int32_t* id = ids + par * a.top;
    float* zi = zis + par * a.top;
    const float wt = w * a.temperature;
    float m = 0.f, s = 1.f, f = 0.f;
    bool learn = w != 0.f;
    if (learn) {
      for (int k = t; k < a.top; k += TH) {
        if (k != t) load_top(a, row, k, rank == 0, next_id, next_t);
        id[k] = next_id;
        tl[k] = next_t;
        if (next_id >= 0) zi[k] = to_f(r.z[next_id]);
      }
      // Slots that are not whole, by the threads that will use them.
      if (r.first == 0 && t == 0) r.read_edge(0, reinterpret_cast<uint32_t*>(buf));
      if (r.last > 0 && t == r.last % TH) r.read_edge(r.last, reinterpret_cast<uint32_t*>(buf + r.last));
      if (r.last == 0 && r.first != 0 && t == 0) r.read_edge(0, reinterpret_cast<uint32_t*>(buf));
      mbar_wait_or_abort(&full, fetched++ & 1, kWaitNs, &gave_up);
      Partial<T> part;
      for (int q0 = t; q0 < r.cnt; q0 += U * TH) {
        uint32_t v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = q0 + u * TH;
          const uint4 x = q < r.cnt ? buf[q] : make_uint4(S::kNegInf, S::kNegInf, S::kNegInf, S::kNegInf);
          v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
        }
        part.template add<U>(v, c);
      }
      m = part.m;
      s = part.s;
      join_warp(m, s, c);
      const float2* got = pairs[0];
      if (C == 1) {
        if (lane == 0) pairs[0][gw] = make_float2(m, s);
        __syncthreads();
      } else {
        const int b = exchanged & 1;
        got = pairs[b];
        if (t == 0) mbar_arrive_expect_tx(&xch[b], (uint32_t)(GW * C * sizeof(float2)));
        if (lane < C) send_pair(&pairs[b][rank * GW + gw], &xch[b], lane, m, s);
        __syncthreads();
        mbar_wait_or_abort(&xch[b], exchanged++ >> 1 & 1, kWaitNs, &gave_up);
      }
      // Every warp joins all pairs, in the same order.
      Partial<T> all;
#pragma unroll
      for (int k = 0; k < GW * kMaxCluster; k += 32) {
        if (k + lane >= GW * C) continue;
        const float2 x = got[k + lane];
        if (x.x == -INFINITY) {
          all.s += x.y;
        } else if (!(x.x <= all.m)) {
          all.s = fmaf(all.s, all.m == -INFINITY ? 1.f : ex2((all.m - x.x) * c), x.y);
          all.m = x.x;
        } else {
          all.s = fmaf(x.y, ex2((x.x - all.m) * c), all.s);
        }
      }
      m = all.m;
      s = all.s;
      join_warp(m, s, c);
      float tmax, ps;
      learn = top_softmax(id, tl, a.top, c, tmax, ps);
      if (learn) {
        f = wt / s;
        if (rank == 0 && gw == GW - 1) {
          const float loss = top_loss(a, id, tl, zi, tmax, ps, m, s);
          if (lane == 0) a.loss[row] = w * loss;
        }
        if (GRAD) {
          const float inv_ps = 1.f / ps;
          for (int k = t; k < a.top; k += TH) p[k] = id[k] < 0 ? 0.f : ex2((tl[k] - tmax) * c) * inv_ps;
          const Dense<T> dense(m, c, f);
#pragma unroll 4
          for (int q = t; q < r.cnt; q += TH) {
            const uint4 x = buf[q];
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
            uint32_t o[4];
            dense.of(v, o);
            r.write(q, o);
          }
        }
      }
    }
    if (!learn) {   // nothing to learn from this row
      if (rank == 0 && t == 0) a.loss[row] = 0.f;
      if (GRAD) {
        const uint32_t o[4] = {0, 0, 0, 0};
        for (int q = t; q < r.cnt; q += TH) r.write(q, o);
      }
    }
    __syncthreads();
    if (w_next != 0.f) {
      if (t == 0) fetch(next);
      if (t < a.top) load_top(a, next, t, rank == 0, next_id, next_t);
    }
    if (GRAD && learn) {   // the listed classes of this slice, again
      for (int k = t; k < a.top; k += TH) {
        float g;
        if (r.holds(id[k]) && top_grad(a, id, p, zi, k, m, f, wt, g)) r.g[id[k]] = from_f<T>(g);
      }
    }
    row = next;
    w = w_next;
  }
  if (gave_up && t == 0 && a.status) atomicOr(a.status, kStatusGaveUp);
}

// Rows beyond a cluster's shared memory: one block per row, which is read for
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
      if (i >= a.cols && a.status) atomicOr(a.status, kStatusIndex);
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
template <typename T, int NV>
cudaError_t warp_as(const Distill& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.rows + 7) / 8)), block(256);
  const size_t smem = (size_t)8 * a.top * 4 * 4;
  if (a.grad) return launch(k_distill_warp<T, NV, true>, grid, block, smem, s, false, 1, a);
  return launch(k_distill_warp<T, NV, false>, grid, block, smem, s, false, 1, a);
}

template <typename T, int TH, bool GRAD>
cudaError_t ring_as(const Distill& a, int C, int slice_slots, size_t smem, int blocks, cudaStream_t s) {
  auto* k = &k_distill_ring<T, TH, GRAD>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t clusters = std::min<int64_t>(a.rows, blocks / C);
  return launch(k, dim3((unsigned)(clusters * C)), dim3(TH), smem, s, false, C, a, C, slice_slots);
}

template <typename T>
cudaError_t distill_rows(const Distill& a, int sms, cudaStream_t s) {
  constexpr int N = Slots<T>::N;
  // Most slots that cover a row, wherever it starts.
  const bool aligned = (uintptr_t)a.logits % 16 == 0 && (a.rows == 1 || (a.ls * (int64_t)sizeof(T)) % 16 == 0);
  const int64_t slots = (a.cols + (aligned ? 0 : N - 1) + N - 1) / N;
  auto ceil = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  if (slots <= 32 * 8 && a.top <= 256) {   // 4 KB
    if (slots <= 32 * 1) return warp_as<T, 1>(a, s);
    if (slots <= 32 * 2) return warp_as<T, 2>(a, s);
    if (slots <= 32 * 3) return warp_as<T, 3>(a, s);
    if (slots <= 32 * 4) return warp_as<T, 4>(a, s);
    if (slots <= 32 * 6) return warp_as<T, 6>(a, s);
    return warp_as<T, 8>(a, s);
  }
  // Shared memory of a block: its slice of the row and the lists; two blocks
  // of 512 threads (four of 256) per SM while they fit, one at most beyond.
  constexpr int64_t kFour = 54 * 1024, kTwo = 110 * 1024, kOne = 220 * 1024;
  const int64_t list_bytes = (int64_t)a.top * 6 * 4;
  auto bytes = [&](int64_t C) { return ceil(slots, C) * 16 + list_bytes; };
  int64_t C = 1;
  while (C < kMaxCluster && bytes(C) > kTwo) C *= 2;
  if (bytes(C) <= kOne) {
    // Few rows: more blocks for each, while a slice is 8 KB.
    while (C < kMaxCluster && a.rows * C * 2 <= sms && ceil(slots, 2 * C) >= 512) C *= 2;
    const bool small = bytes(C) <= kFour;
    const int per_sm = small ? 4 : bytes(C) <= kTwo ? 2 : 1;
    const int slice = (int)ceil(slots, C), blocks = sms * per_sm;
    const size_t smem = (size_t)bytes(C);
    if (a.grad)
      return small ? ring_as<T, 256, true>(a, (int)C, slice, smem, blocks, s) : ring_as<T, 512, true>(a, (int)C, slice, smem, blocks, s);
    return small ? ring_as<T, 256, false>(a, (int)C, slice, smem, blocks, s) : ring_as<T, 512, false>(a, (int)C, slice, smem, blocks, s);
  }
  return launch(k_distill_rows<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
}

}  // namespace
#endif
}  // namespace train
}  // namespace lopt
