// Distillation from a teacher's top logits: the loss of a row and its
// gradient (see lopt_train.h).
//
// With m = max z and s = sum exp((z - m) / T), log q_j = (z_j - m) / T - log s.
// The exponents are taken of z - m, not of z / T - m / T: masks of the type's
// lowest value stay finite that way, and the terms near the maximum exact.
// The loss, with d = t - max t and es = sum 2^(d log2e / T) over the slots, is
//   w T (sum p d - sum p (z - m) + T (log s - log es)):
// no quotient by T, which could overflow for a small one, and no T^2.
// The dense part of the gradient, w T q_j, is written for every column and
// the listed columns are then written again with their p taken off.
#pragma once

#include <algorithm>
#include <type_traits>

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
  float temperature, log2e_t;   // T, log2(e) / T
};

// One per element type, each in a source of its own (they compile side by side).
// A wait that lasts longer than wait_ns has failed.
cudaError_t distill_f32(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s);
cudaError_t distill_f16(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s);
cudaError_t distill_bf16(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s);

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

// The loss of a row from the sums over its slots and its own; wt = w T.  pz is
// half the sum of p (z - m): z = -3.4e38 and p rounded up to more than 1 in
// total would overflow where the loss, for w T < 1, does not.
__device__ __forceinline__ float half_distance(float z, float m) { return 0.5f * z - 0.5f * m; }
__device__ __forceinline__ float loss_of(const Distill& a, float wt, float p_d, float log_e, float pz, float s) {
  return 2.f * (wt * fmaf(0.5f * a.temperature, logf(s) - log_e, fmaf(0.5f, p_d, -pz)));
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
// The exponent is fma(z, c, -mc) with mc = m c rounded once; a factor takes off
// what that rounding left, so the sum is about m exactly.  What it left is at
// most half a unit in the last place of mc: up to 2^24 that is 1/2, and all
// terms stay below 2.  Beyond (rows, or a thread's first classes, that are
// masked by -1e10 or the type's lowest value) it would grow past what 2^x can
// hold, so (z - m) c is taken there, which is slower by an addition.
constexpr float kSafe = 16777216.f;

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
  // One of 2^log_c slices.
  __device__ __forceinline__ Slice(const Distill& a, int64_t row, int rank, int log_c) {
    z = static_cast<const T*>(a.logits) + row * a.ls;
    g = a.grad ? static_cast<T*>(a.grad) + row * a.gs : nullptr;
    cols = (int)a.cols;
    mis = (int)(((uintptr_t)z / sizeof(T)) % N);
    const int total = (mis + cols + N - 1) / N, per = (total + (1 << log_c) - 1) >> log_c;
    beg = min(rank * per, total);
    cnt = min(per, total - beg);
    same = (int)(((uintptr_t)g / sizeof(T)) % N) == mis;
    first = beg == 0 && cnt > 0 && (mis > 0 || cols < N) ? 0 : -1;
    last = cnt > 0 && beg + cnt == total && (mis + cols) % N ? cnt - 1 : -1;
  }
  __device__ __forceinline__ const uint4* z16() const { return reinterpret_cast<const uint4*>(z - mis) + beg; }
  __device__ __forceinline__ bool whole(int q) const { return q != first && q != last; }
  // A slot that is not whole, -inf outside the row.
  __device__ __forceinline__ uint4 read_edge(int q) const { return read_elements(z, (beg + q) * N - mis, cols); }
  static __device__ __noinline__ uint4 read_elements(const T* z, int j, int cols) {
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = Slots<T>::kNegInf;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (j + k < 0 || j + k >= cols) continue;
      if constexpr (sizeof(T) == 4) {
        v[k] = reinterpret_cast<const uint32_t*>(z)[j + k];
      } else {
        const uint32_t e = reinterpret_cast<const uint16_t*>(z)[j + k];
        v[k / 2] = k & 1 ? (v[k / 2] & 0xffffu) | e << 16 : (v[k / 2] & 0xffff0000u) | e;
      }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void write(int q, const uint32_t v[4]) const {
    if (same && whole(q)) {
      reinterpret_cast<uint4*>(g - mis)[beg + q] = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      write_elements(g, (beg + q) * N - mis, cols, make_uint4(v[0], v[1], v[2], v[3]));
    }
  }
  // Columns j .. j + N - 1, those that the row has.
  static __device__ __noinline__ void write_elements(T* g, int j, int cols, uint4 x) {
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t w = v[k * (int)sizeof(T) / 4];
      if (j + k < 0 || j + k >= cols) continue;
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(g)[j + k] = w;
      } else {
        reinterpret_cast<uint16_t*>(g)[j + k] = (uint16_t)(k & 1 ? w >> 16 : w);
      }
    }
  }
  __device__ __forceinline__ bool holds(int j) const {   // column j
    const int q = (j + mis) / N - beg;
    return j >= 0 && q >= 0 && q < cnt;
  }
};

// ---- long rows: a block, or a cluster of blocks, per row -----------------------------
constexpr int kMaxCluster = 8;
constexpr uint64_t kDrainNs = 1000000000ull;   // 1 s: for what is on its way when a block gives up

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory address of another block of the cluster.
template <typename P> __device__ __forceinline__ P* of_block(P* p, int rank) {
  uint64_t out;
  asm("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"((uint64_t)p), "r"(rank));
  return reinterpret_cast<P*>(out);
}
// (m, s) into block `rank` of the cluster, counted on its barrier.
__device__ __forceinline__ void send_pair(const float2* at, const uint64_t* bar, int rank, float m, float s) {
  uint32_t ra, rb;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
               :: "r"(ra), "r"(__float_as_uint(m)), "r"(__float_as_uint(s)), "r"(rb) : "memory");
}

// A row's list as one warp keeps it in shared memory.  Per slot: the class
// (none if it does not count), its weight 2^((t - max) log2e / T), its logit
// z, and, for the first slot of a class of this block's slice, the class's
// place in a hash table (at most half full) that sums the weights of repeats.
struct List {
  int32_t *id, *place, *key;
  float *e, *z, *sum;
  int top, log_size;
  // Of the whole list: 1 / sum of e, its logarithm, sum of p (t - max); whether any slot counts.
  float inv, log_e, p_d;
  bool any;
  __device__ __forceinline__ List(int32_t* words, int top_);
};
__host__ __device__ inline int table_log_size(int top) {
  int n = 5;
  while (1 << n < 2 * top) ++n;
  return n;
}
__host__ __device__ inline int list_words(int top) { return 4 * top + 2 * (1 << table_log_size(top)); }
__device__ __forceinline__ List::List(int32_t* words, int top_) : top(top_), log_size(table_log_size(top_)), any(false) {
  id = words;
  place = id + top;
  e = reinterpret_cast<float*>(place + top);
  z = e + top;
  key = reinterpret_cast<int32_t*>(z + top);
  sum = reinterpret_cast<float*>(key + (1 << log_size));
}

// Slots are taken 128 at a time, four of a lane's side by side: the list is
// a chain of short steps, and its warp has latency to lose, not work.
#define LOPT_LIST_SLOTS(k0, top)                 \
  for (int k0 = 0; k0 < (top); k0 += 128)

// The first 128 slots as loaded, a row ahead of their use.
struct ListAhead {
  int64_t id[4];
  uint32_t t[4];
};
template <typename T>
__device__ __forceinline__ void load_list(const Distill& a, int64_t row, int k0, ListAhead& x) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = k0 + u * 32 + lane;
    x.id[u] = -1;
    x.t[u] = 0;
    if (k >= a.top) continue;
    if (a.itype == LOPT_I32) x.id[u] = static_cast<const int32_t*>(a.top_index)[row * a.is + k];
    else x.id[u] = static_cast<const int64_t*>(a.top_index)[row * a.is + k];
    if (a.ttype == LOPT_F32) x.t[u] = static_cast<const uint32_t*>(a.top_logits)[row * a.ts + k];
    else x.t[u] = static_cast<const uint16_t*>(a.top_logits)[row * a.ts + k];
  }
}
template <typename T>
__device__ __forceinline__ float top_logit(const Distill& a, uint32_t raw) {
  if (a.ttype == LOPT_F32) return __uint_as_float(raw);
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(raw);
  } else {
    const uint16_t h = (uint16_t)raw;
    return to_f(*reinterpret_cast<const T*>(&h));
  }
}

// Where a list's slots come from: slot k, the u-th of four, as loaded.
// From registers (the first 128 slots), the rest from memory ...
template <typename T> struct FromRegs {
  const Distill& a;
  int64_t row;
  ListAhead x;
  __device__ __forceinline__ void block(int k0) {
    if (k0 > 0) load_list<T>(a, row, k0, x);
  }
  __device__ __forceinline__ int64_t id(int k, int u) const { return x.id[u]; }
  __device__ __forceinline__ float t(int k, int u) const { return top_logit<T>(a, x.t[u]); }
};
// ... or from shared memory, where asynchronous copies put them a row ahead
// (a lane's slots by the lane itself: no other thread waits for them).  16-bit
// logits are too narrow for such copies and wait in registers, the first 128.
template <typename T> struct FromShared {
  const Distill& a;
  char* ids;       // [top] of the index type
  float* logits;   // [top] if float32
  uint32_t raw[4];
  int64_t row;
  __device__ __forceinline__ FromShared(const Distill& a_, void* at) : a(a_), ids(static_cast<char*>(at)), row(0) {
    logits = reinterpret_cast<float*>(ids + (size_t)a.top * (a.itype == LOPT_I32 ? 4 : 8));
  }
  static __device__ __forceinline__ uint32_t addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
  __device__ __forceinline__ void fetch(int64_t row_) {
    row = row_;
    const int lane = threadIdx.x % 32;
    asm volatile("cp.async.wait_group 0;" ::: "memory");   // a list that no one wanted may still be landing here
    for (int k = lane; k < a.top; k += 32) {
      if (a.itype == LOPT_I32)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                     :: "r"(addr(ids + k * 4)), "l"(static_cast<const int32_t*>(a.top_index) + row * a.is + k) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                     :: "r"(addr(ids + k * 8)), "l"(static_cast<const int64_t*>(a.top_index) + row * a.is + k) : "memory");
      if (a.ttype == LOPT_F32)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                     :: "r"(addr(logits + k)), "l"(static_cast<const float*>(a.top_logits) + row * a.ts + k) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (a.ttype != LOPT_F32) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        raw[u] = u * 32 + lane < a.top ? static_cast<const uint16_t*>(a.top_logits)[row * a.ts + u * 32 + lane] : 0;
    }
  }
  __device__ __forceinline__ void block(int k0) {
    if (k0 == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ int64_t id(int k, int u) const {
    if (k >= a.top) return -1;
    return a.itype == LOPT_I32 ? (int64_t)reinterpret_cast<const int32_t*>(ids)[k] : reinterpret_cast<const int64_t*>(ids)[k];
  }
  __device__ __forceinline__ float t(int k, int u) const {
    if (k >= a.top) return 0.f;
    if (a.ttype == LOPT_F32) return logits[k];
    return k < 128 ? top_logit<T>(a, raw[u]) : load_as_f(a.top_logits, row * a.ts + k, a.ttype);
  }
};
inline int64_t shared_list_bytes(const Distill& a) {   // a multiple of 8
  return ((int64_t)a.top * ((a.itype == LOPT_I32 ? 4 : 8) + (a.ttype == LOPT_F32 ? 4 : 0)) + 7) / 8 * 8;
}

template <typename T, bool GRAD, typename From>
__device__ __forceinline__ void make_list(const Distill& a, const Slice<T>& r, bool report, From& from, List& l) {
  const int lane = threadIdx.x % 32, size = 1 << l.log_size;
  if (GRAD) {
    for (int h = lane; h < size; h += 32) {
      l.key[h] = -1;
      l.sum[h] = 0.f;
    }
  }
  float tmax = -INFINITY;
  bool any = false, bad = false;
  LOPT_LIST_SLOTS(k0, l.top) {
    from.block(k0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 32 + lane;
      const float t = from.t(k, u);
      const int64_t i = from.id(k, u);
      bad |= i >= a.cols;
      const bool counts = i >= 0 && i < a.cols && t != -INFINITY;
      if (k < l.top) {
        l.id[k] = counts ? (int32_t)i : -1;
        l.e[k] = t;
      }
      if (counts) tmax = fmaxf(tmax, t);
      any |= counts;
    }
  }
  if (bad && report && a.status) atomicOr(a.status, kStatusIndex);
  l.any = __any_sync(0xffffffffu, any);
  if (l.any) {   // the same for all lanes
    tmax = warp_max(tmax);
    float es = 0.f, ed = 0.f;
    LOPT_LIST_SLOTS(k0, l.top) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * 32 + lane;
        if (k >= l.top) continue;
        const float d = l.e[k] - tmax, e = l.id[k] < 0 ? 0.f : ex2(d * a.log2e_t);
        es += e;
        if (e != 0.f) ed = fmaf(e, d, ed);   // 0 log 0 = 0
        l.e[k] = e;
      }
    }
    es = warp_sum(es);
    ed = warp_sum(ed);
    l.inv = 1.f / es;
    l.log_e = logf(es);
    l.p_d = __fmul_rn(ed, l.inv);   // rounded here in every form of the kernels: the loss has the same bits
    __syncwarp();
    if (GRAD) {
      for (int k0 = 0; k0 < l.top; k0 += 32) {
        const int k = k0 + lane;
        int32_t i = k < l.top ? l.id[k] : -1;
        if (!r.holds(i)) i = -1;   // another block's
        int place = -1;
        const unsigned alike = __match_any_sync(0xffffffffu, i);
        if (i >= 0 && lane == __ffs(alike) - 1) {   // its first slot here: sums in slot order
          float e = 0.f;
          for (unsigned rest = alike; rest; rest &= rest - 1) e += l.e[k0 + __ffs(rest) - 1];
          unsigned h = (unsigned)i * 2654435761u >> (32 - l.log_size);
          int32_t old;
          while ((old = atomicCAS(l.key + h, -1, i)) != -1 && old != i) h = (h + 1) & (size - 1);
          l.sum[h] += e;
          if (old == -1) place = (int)h;
        }
        if (k < l.top) l.place[k] = place;
        __syncwarp();
      }
    }
  }
}

// The logits of the slots of this slice, from where it landed: those in whole
// 16-byte slots, or those in the others.
template <typename T, bool WHOLE>
__device__ __forceinline__ void read_listed(const Slice<T>& r, const uint4* buf, const List& l) {
  const T* z = reinterpret_cast<const T*>(buf) + (r.mis - r.beg * Slice<T>::N);   // column j at z[j]
  LOPT_LIST_SLOTS(k0, l.top) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 32 + (int)(threadIdx.x % 32);
      if (k >= l.top) continue;
      const int j = l.id[k];
      if (r.holds(j) && r.whole((j + r.mis) / Slice<T>::N - r.beg) == WHOLE) l.z[k] = to_f(z[j]);
    }
  }
}

// This lane's part of half the sum of p (z - m) over the slots of the slice.
template <typename T>
__device__ __forceinline__ float sum_listed(const Slice<T>& r, const List& l, float m) {
  float pz = 0.f;
  LOPT_LIST_SLOTS(k0, l.top) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 32 + (int)(threadIdx.x % 32);
      if (k >= l.top || !r.holds(l.id[k])) continue;
      const float p = l.e[k] * l.inv;
      if (p != 0.f) pz = fmaf(p, half_distance(l.z[k], m), pz);   // 0 log 0 = 0
    }
  }
  return pz;
}

// A list of at most 128 slots whose gradient is not wanted (or at most 32, in
// a lane each): registers hold it.
template <int U> struct SlotRegs {
  int32_t id[U];
  float e[U], z[U];
  float inv, log_e, p_d;
  bool any;
};
template <int U, typename From>
__device__ __forceinline__ void make_slots(const Distill& a, From& from, bool report, SlotRegs<U>& l) {
  from.block(0);
  float tmax = -INFINITY;
  bool any = false, bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = u * 32 + (int)(threadIdx.x % 32);
    l.e[u] = from.t(k, u);
    const int64_t i = from.id(k, u);
    bad |= i >= a.cols;
    const bool counts = i >= 0 && i < a.cols && l.e[u] != -INFINITY;
    l.id[u] = counts ? (int32_t)i : -1;
    if (counts) tmax = fmaxf(tmax, l.e[u]);
    any |= counts;
  }
  if (bad && report && a.status) atomicOr(a.status, kStatusIndex);
  l.any = __any_sync(0xffffffffu, any);
  tmax = warp_max(tmax);
  float2 sums = make_float2(0.f, 0.f);   // of e, of e (t - max)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float d = l.e[u] - tmax, e = l.id[u] < 0 ? 0.f : ex2(d * a.log2e_t);
    l.e[u] = e;
    sums.x += e;
    if (e != 0.f) sums.y = fmaf(e, d, sums.y);   // 0 log 0 = 0
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sums = __fadd2_rn(sums, make_float2(__shfl_xor_sync(0xffffffffu, sums.x, o), __shfl_xor_sync(0xffffffffu, sums.y, o)));
  l.inv = 1.f / sums.x;
  l.log_e = logf(sums.x);
  l.p_d = __fmul_rn(sums.y, l.inv);
}
template <typename T, bool WHOLE, int U>
__device__ __forceinline__ void read_slots(const Slice<T>& r, const uint4* buf, SlotRegs<U>& l) {
  const T* z = reinterpret_cast<const T*>(buf) + (r.mis - r.beg * Slice<T>::N);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (r.holds(l.id[u]) && r.whole((l.id[u] + r.mis) / Slice<T>::N - r.beg) == WHOLE) l.z[u] = to_f(z[l.id[u]]);
}
template <typename T, int U>
__device__ __forceinline__ float sum_slots(const Slice<T>& r, const SlotRegs<U>& l, float m) {
  float pz = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float p = l.e[u] * l.inv;
    if (p != 0.f && r.holds(l.id[u])) pz = fmaf(p, half_distance(l.z[u], m), pz);
  }
  return pz;
}

// The gradient of the listed classes, over what the dense part wrote.
template <typename T>
__device__ __forceinline__ void write_listed(const Slice<T>& r, const List& l, float c, float m, float f, float wt) {
  const float wp = wt * l.inv;
  LOPT_LIST_SLOTS(k0, l.top) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * 32 + (int)(threadIdx.x % 32);
      const int h = k < l.top ? l.place[k] : -1;
      if (h >= 0) r.g[l.id[k]] = from_f<T>(fmaf(ex2((l.z[k] - m) * c), f, -wp * l.sum[h]));
    }
  }
}

// The same for a list of a slot in each lane.
template <typename T>
__device__ __forceinline__ void write_slots(const Slice<T>& r, const SlotRegs<1>& l, float c, float m, float f, float wt) {
  const int lane = threadIdx.x % 32;
  // By the first slot of a class, the repeats added in slot order.
  const unsigned alike = __match_any_sync(0xffffffffu, l.id[0]);
  float e = l.e[0];
  if (__any_sync(0xffffffffu, l.id[0] >= 0 && alike != 1u << lane)) {
    e = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float ek = __shfl_sync(0xffffffffu, l.e[0], k);
      if (alike >> k & 1) e += ek;
    }
  }
  if (l.id[0] >= 0 && lane == __ffs(alike) - 1)
    r.g[l.id[0]] = from_f<T>(fmaf(ex2((l.z[0] - m) * c), f, -wt * l.inv * e));
}

// ---- short rows: a warp per row ----------------------------------------------------
// The row stays in registers, NV slots per lane.  Its loads go out before
// its weight is known: a short row is a chain of latencies.  Float32 rows of
// 1000 with 20 slots and gradient: 10.2 us for 4,096 (3.3 TB/s, one wave), 100
// us for 67,108 (5.3 TB/s).
constexpr int kWarpRows = 4;   // rows of a block: small blocks even out the last wave

template <typename T, int NV, bool GRAD>
__global__ void __launch_bounds__(32 * kWarpRows, 8) k_distill_warp(const Distill a) {
  using S = Slots<T>;
  extern __shared__ int32_t words[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * kWarpRows + warp;
  if (row >= a.rows) return;
  FromRegs<T> from{a, row, {}};
  load_list<T>(a, row, 0, from.x);
  const ListAhead& x = from.x;
  const Slice<T> r(a, row, 0, 0);
  uint32_t v[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = i * 32 + lane;
    uint4 y = make_uint4(S::kNegInf, S::kNegInf, S::kNegInf, S::kNegInf);
    if (q < r.cnt) y = r.whole(q) ? r.z16()[q] : r.read_edge(q);
    v[i][0] = y.x; v[i][1] = y.y; v[i][2] = y.z; v[i][3] = y.w;
  }
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  float z[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (x.id[u] >= 0 && x.id[u] < a.cols) z[u] = to_f(r.z[x.id[u]]);
  const float c = a.log2e_t;
  Partial<T> part;
  part.template add<NV>(v, c);
  float m = part.m, s = part.s;
  join_warp(m, s, c);
  const float wt = w * a.temperature, f = wt / s;
  // The loss, or a row of zeros; whether there is a gradient to write.
  auto finish = [&](bool any, float p_d, float log_e, float pz) {
    if (lane == 0) a.loss[row] = any ? loss_of(a, wt, p_d, log_e, pz, s) : 0.f;
    if (!GRAD) return false;
    if (!any) {   // nothing to learn from this row
      const uint32_t o[4] = {0, 0, 0, 0};
      for (int q = lane; q < r.cnt; q += 32) r.write(q, o);
      return false;
    }
    const Dense<T> dense(m, c, f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = i * 32 + lane;
      if (q >= r.cnt) continue;
      uint32_t o[4];
      dense.of(v[i], o);
      r.write(q, o);
    }
    __syncwarp();
    return true;
  };
  if (a.top <= 32) {   // a slot in each lane
    SlotRegs<1> l;
    make_slots(a, from, w != 0.f, l);
    l.z[0] = z[0];
    const bool any = w != 0.f && l.any;
    if (!finish(any, l.p_d, l.log_e, warp_sum(sum_slots(r, l, m)))) return;
    write_slots(r, l, c, m, f, wt);
    return;
  }
  List l(words + warp * list_words(a.top), a.top);
  if (w != 0.f) {
    make_list<T, GRAD>(a, r, true, from, l);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u * 32 + lane < l.top) l.z[u * 32 + lane] = z[u];
    for (int k = 128 + lane; k < l.top; k += 32)
      if (l.id[k] >= 0) l.z[k] = to_f(r.z[l.id[k]]);
    __syncwarp();
  }
  if (finish(l.any, l.p_d, l.log_e, warp_sum(l.any ? sum_listed(r, l, m) : 0.f))) write_listed(r, l, c, m, f, wt);
}

// ---- rows of up to 16 KB: a block per row ---------------------------------------------
// The row stays in registers, kBlockSlots slots per thread; the first warp has
// the list.  A block takes one row and ends: the SM's other blocks run through
// its waits.
constexpr int kBlockSlots = 4, kBlockThreads = 256;

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kBlockThreads, 4) k_distill_block(const Distill a) {
  using S = Slots<T>;
  constexpr int NV = kBlockSlots;
  const int TH = blockDim.x, W = TH / 32;
  extern __shared__ int32_t words[];
  __shared__ float2 pairs[kBlockThreads / 32];   // (m, s) of the warps
  __shared__ int any_slot;
  const int t = threadIdx.x, lane = t % 32, warp = t / 32;
  const int64_t row = blockIdx.x;
  FromRegs<T> from{a, row, {}};
  if (warp == 0) load_list<T>(a, row, 0, from.x);
  const Slice<T> r(a, row, 0, 0);
  uint32_t v[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = i * TH + t;
    uint4 y = make_uint4(S::kNegInf, S::kNegInf, S::kNegInf, S::kNegInf);
    if (q < r.cnt) y = r.whole(q) ? r.z16()[q] : r.read_edge(q);
    v[i][0] = y.x; v[i][1] = y.y; v[i][2] = y.z; v[i][3] = y.w;
  }
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  const float c = a.log2e_t;
  const bool slots = a.top <= 32;   // a slot in each lane
  SlotRegs<1> lr;
  List l(words, a.top);
  if (warp == 0 && w != 0.f) {
    if (slots) {
      make_slots(a, from, true, lr);
      if (lr.id[0] >= 0) lr.z[0] = to_f(r.z[lr.id[0]]);
    } else {
      make_list<T, GRAD>(a, r, true, from, l);
      for (int k = lane; k < l.top; k += 32)
        if (l.id[k] >= 0) l.z[k] = to_f(r.z[l.id[k]]);
    }
    if (lane == 0) any_slot = slots ? lr.any : l.any;
  }
  Partial<T> part;
  part.template add<NV>(v, c);
  float m = part.m, s = part.s;
  join_warp(m, s, c);
  if (lane == 0) pairs[warp] = make_float2(m, s);
  __syncthreads();
  if (w == 0.f || !any_slot) {   // nothing to learn from this row
    if (t == 0) a.loss[row] = 0.f;
    const uint32_t o[4] = {0, 0, 0, 0};
    if (GRAD)
      for (int q = t; q < r.cnt; q += TH) r.write(q, o);
    return;
  }
  const float2 x = lane < W ? pairs[lane] : make_float2(-INFINITY, 0.f);
  m = x.x;
  s = x.y;
  join_warp(m, s, c);
  const float wt = w * a.temperature, f = wt / s;
  if (warp == 0) {
    const float pz = warp_sum(slots ? sum_slots(r, lr, m) : sum_listed(r, l, m));
    if (lane == 0) a.loss[row] = slots ? loss_of(a, wt, lr.p_d, lr.log_e, pz, s) : loss_of(a, wt, l.p_d, l.log_e, pz, s);
  }
  if (!GRAD) return;
  const Dense<T> dense(m, c, f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = i * TH + t;
    if (q >= r.cnt) break;
    uint32_t o[4];
    dense.of(v[i], o);
    r.write(q, o);
  }
  __syncthreads();
  if (warp != 0) return;
  if (slots) write_slots(r, lr, c, m, f, wt);
  else write_listed(r, l, c, m, f, wt);
}

// The row's (m, s) from all its warps' pairs, by one warp, in a fixed order.
template <int N>
__device__ __forceinline__ void join_pairs(const float2* got, int n, float c, float& m, float& s) {
  const int lane = threadIdx.x % 32;
  m = -INFINITY;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 32) {
    if (k >= n) break;
    float mk = -INFINITY, sk = 0.f;
    if (k + lane < n) {
      const float2 x = got[k + lane];
      mk = x.x;
      sk = x.y;
    }
    join_warp(mk, sk, c);
    const float top = fmaxf(m, mk);
    s = (m == -INFINITY ? s : s * ex2((m - top) * c)) + (mk == -INFINITY ? sk : sk * ex2((mk - top) * c));
    m = top;
  }
}

// Persistent: cluster i takes rows i, i + clusters, ...  TH threads compute
// and one more warp works ahead of them: it has each block's slice of the next
// row copied into shared memory as soon as the last read of the current one
// is done, so that loads run while the block still stores and the SM's other
// blocks compute; it prepares the next row's list, whose loads went out a row
// before; it reads the listed classes' logits where they landed; and it
// writes their gradient again once the dense part is stored.  A
// computing thread reads its slots twice: for its part of (m, s), and for the
// dense gradient.
//
// Hand-offs of a row of weight other than 0 (the others use none), all by
// mbarriers whose phase is the row's number among those:
//   full    the copy's bytes are there
//   summed  the computing warps have their (m, s), and are done with the
//           buffer if no gradient is wanted
//   listed  the row's list is ready
//   empty   the computing warps' dense stores are out: the buffer is free and
//           the listed classes may be written
// Blocks of a cluster send their warps' pairs to each other, and their parts
// of the loss to the first one, by stores that count on the receiver's `xch`
// and `parts`.  The ahead warp of a block fetches row e + 1 only after it
// waited for summed (and empty) of row e, so no barrier is ever two phases
// ahead of a waiter; a block sends for row e + 4 only after its ahead warp
// finished row e + 2 with all pairs of that row, whose senders' ahead warps
// had then finished row e: with four sets in rotation no set is overwritten
// while it is read.
//
// Every wait is bounded.  A warp whose wait runs out sets gave_up in all
// blocks of the cluster, which ends their other waits too, and leaves at the
// row it is in.  No block goes before all are here; if one gave up, they then
// agree on how far the stores to each other have come, send what is missing
// (nobody reads it), wait until all of it and the copies have landed, and mark
// the rows that are not whole: their loss is NaN, and the caller's status says
// so.  A warp's answer in common and the last barrier cost 0.6 % of the first
// case below and 2 % of the second (247.6 and 36.0 us when waits that ran out
// went unnoticed), and of 7 rows of 50,257 in a graph 4 % (6.4 us, 6.15).
//
// Bound by HBM bytes: 8,192 rows of 50,257 bfloat16 (two blocks to a row) with
// gradient 249 us, 6.21 TB/s; the loss alone of 2,048 rows of 50,304 float16
// 37 us, 5.0 TB/s, since a block has six rows and nothing covers the first
// one's load.  Copying the next row chunk by chunk, as the current one's are
// done with, was slower (264 and 64 us), and so was a row in the registers of a
// cluster (469).
template <typename T, int TH, bool GRAD>
__global__ void __launch_bounds__(TH + 32, 1024 / TH) k_distill_ring(const Distill a, const int log_c, const int slice_slots,
                                                                     const int ahead_bytes, const uint64_t wait_ns) {
  constexpr int GW = TH / 32, U = 4, SETS = 4;
  extern __shared__ __align__(128) unsigned char sm[];
  uint4* buf = reinterpret_cast<uint4*>(sm);
  __shared__ float2 pairs[SETS][GW * kMaxCluster];    // (m, s) of the row's warps
  __shared__ float2 loss_parts[SETS][kMaxCluster];    // (half the sum of p (z - m), 0) of the blocks
  __shared__ uint64_t full, summed, listed, empty, xch[SETS], parts[SETS];
  __shared__ int gave_up;                             // here or in another block of the cluster
  __shared__ int32_t any[2];   // whether a slot of the row counts
  const int t = threadIdx.x, lane = t % 32, gw = t / 32;
  const int C = 1 << log_c;
  const int rank = C == 1 ? 0 : (int)cluster_rank();
  const int clusters = gridDim.x >> log_c;
  int64_t row = blockIdx.x >> log_c;
  if (t == 0) {
    mbar_init(&full, 1);
    mbar_init(&summed, GW);
    mbar_init(&listed, 1);
    mbar_init(&empty, GW);
    for (int k = 0; k < SETS; ++k) {
      mbar_init(&xch[k], 1);
      mbar_init(&parts[k], 1);
    }
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  auto weight = [&](int64_t r) { return r >= a.rows ? 0.f : a.row_weight ? a.row_weight[r] : 1.f; };
  // By a whole warp, with one answer.
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
    return __all_sync(0xffffffffu, mbar_wait_slow(bar, phase & 1, wait_ns, &gave_up)) != 0;
  };
  // The pairs of a computing warp for the n-th row, and the ahead warp's part.
  auto send_pairs = [&](uint32_t n, float m, float s) {
    const int b = n & (SETS - 1);
    if (t == 0) mbar_arrive_expect_tx(&xch[b], (uint32_t)(GW * C * sizeof(float2)));
    if (lane < C) send_pair(&pairs[b][rank * GW + gw], &xch[b], lane, m, s);
  };
  auto send_part = [&](uint32_t n, float pz) {
    const int b = n & (SETS - 1);
    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&parts[b], (uint32_t)(C * sizeof(float2)));
    __syncwarp();
    if (lane == 0) send_pair(&loss_parts[b][rank], &parts[b], 0, pz, 0.f);
  };
  float w = weight(row);
  uint32_t e = 0;         // rows of weight other than 0 so far; a warp that gives up counts one whose pairs or part it sent
  uint32_t fetched = 0;   // the ahead warp's copies
  const float c = a.log2e_t;
  int32_t* const words = reinterpret_cast<int32_t*>(sm + (size_t)slice_slots * 16 + ahead_bytes);

  if (gw == GW) {   // the warp that works ahead
    FromShared<T> from(a, sm + (size_t)slice_slots * 16);
    List l(words, a.top);
    // The whole slots of a row's slice, when all lanes are done with the last one's.
    auto fetch = [&](const Slice<T>& n) {
      __syncwarp();
      if (lane == 0) {
        const int lo = n.first == 0 ? 1 : 0, hi = n.last >= 0 ? n.last : n.cnt;
        const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16 : 0;
        mbar_arrive_expect_tx(&full, bytes);
        if (bytes) bulk_g2s(buf + lo, n.z16() + lo, bytes, &full);
      }
      ++fetched;
      __syncwarp();
    };
    SlotRegs<4> lr;
    const bool regs = !GRAD && a.top <= 128;
    auto list = [&](const Slice<T>& n, int par) {
      if (regs) make_slots(a, from, rank == 0, lr);
      else make_list<T, GRAD>(a, n, rank == 0, from, l);
      if (lane == 0) {
        any[par] = regs ? lr.any : l.any;
        mbar_arrive(&listed);
      }
      __syncwarp();
    };
    auto read = [&](const Slice<T>& n, auto whole) {
      if (regs) read_slots<T, decltype(whole)::value>(n, buf, lr);
      else read_listed<T, decltype(whole)::value>(n, buf, l);
    };
    from.fetch(row);
    Slice<T> r(a, row, rank, log_c);
    if (w != 0.f) {
      fetch(r);
      list(r, 0);
    }
    if (row + clusters < a.rows) from.fetch(row + clusters);
    for (int par = 0; row < a.rows; par ^= 1) {
      const int64_t next = row + clusters;
      const float w_next = weight(next);
      const Slice<T> r_next(a, next < a.rows ? next : row, rank, log_c);
      if (w != 0.f) {
        const int b = e & (SETS - 1);
        const bool learn = regs ? lr.any : l.any;
        if (!wait(&full, e)) break;
        if (learn) read(r, std::true_type());
        if (!wait(&summed, e)) break;
        if (learn && (r.first >= 0 || r.last >= 0)) read(r, std::false_type());
        if (!GRAD && w_next != 0.f) fetch(r_next);
        if (C > 1 && !wait(&xch[b], e / SETS)) break;
        float m, s;
        join_pairs<GW * kMaxCluster>(pairs[b], GW * C, c, m, s);
        float pz = learn ? warp_sum(regs ? sum_slots(r, lr, m) : sum_listed(r, l, m)) : 0.f;
        if (C > 1) {   // the first block adds the blocks' parts
          send_part(e, pz);
          if (rank == 0) {
            if (!wait(&parts[b], e / SETS)) {
              ++e;
              break;
            }
            pz = warp_sum(lane < C ? loss_parts[b][lane].x : 0.f);
          }
        }
        float loss = 0.f;
        if (learn) {
          const float wt = w * a.temperature;
          loss = regs ? loss_of(a, wt, lr.p_d, lr.log_e, pz, s) : loss_of(a, wt, l.p_d, l.log_e, pz, s);
        }
        if (rank == 0 && lane == 0) a.loss[row] = loss;
        if (GRAD) {
          if (!wait(&empty, e)) {
            ++e;
            break;
          }
          if (w_next != 0.f) fetch(r_next);
          if (learn) {   // the listed classes of this slice, again
            const float wt = w * a.temperature;
            write_listed(r, l, c, m, wt / s, wt);
          }
          __syncwarp();
        }
        ++e;
      } else {
        if (w_next != 0.f) fetch(r_next);
        if (rank == 0 && lane == 0) a.loss[row] = 0.f;
      }
      if (w_next != 0.f) list(r_next, par ^ 1);
      if (next + clusters < a.rows) from.fetch(next + clusters);
      r = r_next;
      row = next;
      w = w_next;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");   // a list that no one wanted
  } else {
    for (int par = 0; row < a.rows; par ^= 1) {
      const int64_t next = row + clusters;
      const float w_next = weight(next);
      const Slice<T> r(a, row, rank, log_c);
      bool learn = false;
      if (w != 0.f) {
        // Slots that are not whole are read by the threads that use them (a
        // slot of the buffer is the same thread's in every row), and stored
        // when the copy is there: until then the ahead warp may still read
        // the row before.
        const bool edge_first = r.first == 0 && t == 0, edge_last = r.last >= 0 && r.last != r.first && t == r.last % TH;
        uint4 edge = make_uint4(0, 0, 0, 0);
        if (edge_first) edge = r.read_edge(0);
        else if (edge_last) edge = r.read_edge(r.last);
        if (!wait(&full, e)) break;
        if (edge_first || edge_last) {
          buf[edge_first ? 0 : r.last] = edge;
          if (edge_first && edge_last) buf[r.last] = r.read_edge(r.last);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // a later row's copy may land there
        }
        Partial<T> part;
        int q = t;
        for (; q + (U - 1) * TH < r.cnt; q += U * TH) {
          uint32_t v[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint4 x = buf[q + u * TH];
            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          }
          part.template add<U>(v, c);
        }
        for (; q < r.cnt; q += TH) {
          const uint4 x = buf[q];
          const uint32_t v[1][4] = {{x.x, x.y, x.z, x.w}};
          part.template add<1>(v, c);
        }
        float m = part.m, s = part.s;
        join_warp(m, s, c);
        const int b = e & (SETS - 1);
        if (C == 1) {
          if (lane == 0) pairs[b][gw] = make_float2(m, s);
        } else {
          send_pairs(e, m, s);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&summed);
        if (GRAD) {
          if (!(C > 1 ? wait(&xch[b], e / SETS) : wait(&summed, e)) || !wait(&listed, e)) {
            ++e;
            break;
          }
          learn = any[par];
          if (learn) {
            join_pairs<GW * kMaxCluster>(pairs[b], GW * C, c, m, s);
            const Dense<T> dense(m, c, w * a.temperature / s);
#pragma unroll 4
            for (int k = t; k < r.cnt; k += TH) {
              const uint4 x = buf[k];
              const uint32_t v[4] = {x.x, x.y, x.z, x.w};
              uint32_t o[4];
              dense.of(v, o);
              r.write(k, o);
            }
          }
        }
      }
      if (GRAD && !learn) {   // nothing to learn from this row
        const uint32_t o[4] = {0, 0, 0, 0};
        for (int q = t; q < r.cnt; q += TH) r.write(q, o);
      }
      if (w != 0.f) {
        if (GRAD) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty);
        }
        ++e;
      }
      row = next;
      w = w_next;
    }
  }

  // Leaving; `row` is the first row that this warp has not finished.
  if (row < a.rows) {
    if (C == 1) gave_up = 1;
    else if (lane < C) *of_block(&gave_up, lane) = 1;
  }
  __syncwarp();
  if (C == 1) __syncthreads();
  else cluster_sync();
  if (*(volatile int*)&gave_up == 0) return;
  // Some warp gave up.
  if (C > 1) {
    // How far the cluster's computing warps (its ahead warps) came: no one is
    // more than two rows behind.  The lists are not wanted any more.
    uint32_t* sent_n = reinterpret_cast<uint32_t*>(words);   // [GW + 1]
    if (lane == 0) sent_n[gw] = e;
    __syncwarp();
    cluster_sync();
    const int n = gw == GW ? 1 : GW;
    uint32_t most = 0;
    for (int k = lane; k < n * C; k += 32) most = max(most, of_block(sent_n, k / n)[gw == GW ? GW : k % n]);
    most = __reduce_max_sync(0xffffffffu, most);
    for (; e < most; ++e) {
      if (gw == GW) send_part(e, 0.f);
      else send_pairs(e, 0.f, 0.f);
    }
    __syncwarp();
    cluster_sync();   // all is sent, and no one reads another block's memory any more
    if (gw == 0 || (gw == GW && rank == 0)) {
      uint64_t* bars = gw == GW ? parts : xch;
      for (uint32_t k = most > SETS ? most - SETS : 0; k < most; ++k)
        mbar_wait_bounded(bars + (k & (SETS - 1)), k / SETS & 1, kDrainNs);
    }
  }
  if (gw != GW) return;
  if (fetched) mbar_wait_bounded(&full, (fetched - 1) & 1, kDrainNs);
  // The ahead warp finishes a row last of its block's.
  if (row < a.rows && lane == 0 && a.status) atomicOr(a.status, kStatusGaveUp);
  for (int64_t k = row + (int64_t)lane * clusters; k < a.rows; k += (int64_t)32 * clusters) a.loss[k] = NAN;
}

// Rows beyond a cluster's shared memory: one block per row, which is read for
// each of the three passes.  304 rows of 500,009 float32 with gradient: 722 us,
// 3.4 TB/s of the four passes' bytes; each pass waits for the one before, and
// rows this long come few at a time.
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
  const float inv_ps = 1.f / ps;
  const float log_q = 0.5f * a.temperature * (logf(s) - logf(ps));
  float kl = 0.f;
  for (int k = tid; k < a.top; k += L) {
    if (id[k] < 0) continue;
    const float d = p[k] - tmax;
    const float pk = ex2(d * a.log2e_t) * inv_ps;
    if (pk != 0.f) kl += pk * ((0.5f * d - half_distance(zi[k], m)) + log_q);   // 0 log 0 = 0
    p[k] = pk;
  }
  kl = block_sum<W>(kl, red);
  const float wt = w * a.temperature, f = wt / s;
  if (tid == 0) a.loss[row] = 2.f * (wt * kl);
  if (!g) return;
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

#undef LOPT_LIST_SLOTS

// ---- choice of the kernel -------------------------------------------------------
template <typename T, int NV>
cudaError_t warp_as(const Distill& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.rows + kWarpRows - 1) / kWarpRows)), block(32 * kWarpRows);
  const size_t smem = a.top <= 32 ? 0 : (size_t)kWarpRows * list_words(a.top) * 4;
  if (a.grad) return launch(k_distill_warp<T, NV, true>, grid, block, smem, s, false, 1, a);
  return launch(k_distill_warp<T, NV, false>, grid, block, smem, s, false, 1, a);
}

template <typename T>
cudaError_t block_as(const Distill& a, int threads, cudaStream_t s) {
  const size_t smem = a.top <= 32 ? 0 : (size_t)list_words(a.top) * 4;
  return launch(a.grad ? k_distill_block<T, true> : k_distill_block<T, false>, dim3((unsigned)a.rows), dim3(threads), smem, s,
                false, 1, a);
}

template <typename T, int TH, bool GRAD>
cudaError_t ring_as(const Distill& a, int log_c, int slice_slots, size_t smem, int blocks, uint64_t wait_ns,
                    cudaStream_t s) {
  auto* k = &k_distill_ring<T, TH, GRAD>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  const int64_t clusters = std::min<int64_t>(a.rows, blocks >> log_c);
  return launch(k, dim3((unsigned)(clusters << log_c)), dim3(TH + 32), smem, s, false, 1 << log_c, a, log_c, slice_slots,
                (int)shared_list_bytes(a), wait_ns);
}

template <typename T>
cudaError_t distill_rows(const Distill& a, uint64_t wait_ns, int sms, cudaStream_t s) {
  constexpr int N = Slots<T>::N;
  // Most slots that cover a row, wherever it starts.
  const bool aligned = (uintptr_t)a.logits % 16 == 0 && (a.rows == 1 || (a.ls * (int64_t)sizeof(T)) % 16 == 0);
  const int64_t slots = (a.cols + (aligned ? 0 : N - 1) + N - 1) / N;
  auto ceil = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  // Up to 4 KB, with lists of four warps that stay within 48 KB (rows of 1000
  // float32 by warps and by blocks: 20,000 with 33 slots 56 and 66 us, with 256
  // 150 and 171; only a few rows with long lists are the other way round, 4,096
  // with 256 52 and 46).
  if (slots <= 32 * 8 && a.top <= 256) {
    if (slots <= 32 * 1) return warp_as<T, 1>(a, s);
    if (slots <= 32 * 2) return warp_as<T, 2>(a, s);
    if (slots <= 32 * 3) return warp_as<T, 3>(a, s);
    if (slots <= 32 * 4) return warp_as<T, 4>(a, s);
    if (slots <= 32 * 6) return warp_as<T, 6>(a, s);
    return warp_as<T, 8>(a, s);
  }
  // Up to 16 KB.  (64M elements with gradient: rows of 4000 bfloat16 64 us,
  // 132 by the persistent blocks; rows of 2000 float32 105, 244.  A little
  // above it is the other way round, rows of 5003 float32 178 us with 512
  // threads to a block, 119.)
  if (slots <= kBlockSlots * kBlockThreads)
    return block_as<T>(a, (int)std::max<int64_t>(ceil(slots, kBlockSlots * 32) * 32, 64), s);
  // Shared memory of a block: its slice of the row and the lists.  The fewest
  // blocks to a row of which three still fit an SM (64M float32 elements in
  // rows of 131,072 with gradient: 131 us with slices of 64 KB so, 163 with two
  // larger blocks per SM; rows of 32,000: 97 in two slices, 136 in four), or
  // four where they do; else two blocks of 512 threads, else one.
  constexpr int64_t kFour = 54912, kThree = 74368, kTwo = 107 * 1024, kOne = 216 * 1024;
  const int64_t list_bytes = (int64_t)list_words(a.top) * 4 + shared_list_bytes(a);
  auto bytes = [&](int lc) { return ceil(slots, 1 << lc) * 16 + list_bytes; };
  int lc = 0;   // log2 of the blocks per row
  while (1 << lc < kMaxCluster && bytes(lc) > kThree) ++lc;
  if (bytes(lc) <= kOne) {
    // Few rows: more blocks for each, while a slice is 8 KB (bfloat16 with
    // gradient, in a graph: 30 rows of 20,000 6.4 us, 9 without, 6.4 down to 4 KB,
    // 6.9 down to 16 KB; 7 rows of 50,257 6.4, 6.9, 6.4 and 6.3).
    while (1 << lc < kMaxCluster && (a.rows << lc) * 2 <= sms && ceil(slots, 2 << lc) >= 512) ++lc;
    const bool small = bytes(lc) <= kThree;
    const int per_sm = bytes(lc) <= kFour ? 4 : small ? 3 : bytes(lc) <= kTwo ? 2 : 1;
    const int slice = (int)ceil(slots, 1 << lc), blocks = sms * per_sm;
    const size_t smem = (size_t)bytes(lc);
    if (a.grad)
      return small ? ring_as<T, 256, true>(a, lc, slice, smem, blocks, wait_ns, s)
                   : ring_as<T, 512, true>(a, lc, slice, smem, blocks, wait_ns, s);
    return small ? ring_as<T, 256, false>(a, lc, slice, smem, blocks, wait_ns, s)
                 : ring_as<T, 512, false>(a, lc, slice, smem, blocks, wait_ns, s);
  }
  return launch(k_distill_rows<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
}

}  // namespace
#endif
}  // namespace train
}  // namespace lopt
