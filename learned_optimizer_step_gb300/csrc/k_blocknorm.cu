// Block norm, forward and backward (see lopt_lm.h for the formulas).
//
// Forward: a row of h, residual and gate is read once into registers; two sums
// of squares over the row, one after the other, give rms(h) and rms(summed).
// Backward: sum(q hhat) needs grad_residual, which needs sum(g xhat).  But it is
// linear in it: with c1 = -rstd_pre sum(g xhat) / cols, grad_residual = A + c1 xhat,
// and sum(q hhat) = scale (sum(u A) + c1 sum(u xhat)) with u = open w_post hhat.  So
// three sums over the row, taken together, do: a row waits once, not twice.  They are taken
// of summed and h themselves, as the products of two rows of the same size as the sums of
// squares are, and the roots come in afterwards.  Each thread keeps the sums over rows of its
// own columns (the gradients of both weights) in registers, the blocks' sums go to
// the workspace and a second kernel adds them in block order.  Both directions
// are bound by HBM bytes: 4 arrays forward, 6 backward, one and two more with a
// gate.  65,536 x 768 bfloat16 with a gate forward 78 us (6.5 TB/s), 16,421 rows 25 us
// (launch and first loads are a quarter of it); backward 32,768 x 2048 144 us (5.6 TB/s;
// a row's chain of sum, barrier and stores at 16 warps), with a gate 194 us (5.5 TB/s).
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "lopt_lm.h"
#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

struct Fwd {
  const void *h, *residual, *gate, *w_post, *w_pre;
  void *y, *summed;
  float *rstd_post, *rstd_pre;
  int64_t rows, cols, hs, rs, gs, ys, ss;
  int wtype;
  float scale, eps;
};

struct Bwd {
  const void *dy, *h, *summed, *gate, *dsum, *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *dh, *dres, *dgate;
  float* part;      // [2][gridDim.x][cols]: sums of dz * hhat, then of dy * xhat
  float* coef;      // rows too long for registers: sum(g xhat) / cols of each
  int64_t rows, cols, dys, hs, xs, gs, dss, dhs, drs, dgs;
  int wtype;
  float scale;
};

// Sum over the L threads of group `group` of a block.  red: an area of this one
// of a row's two sums; the other sum's barrier stands between two uses of it.
template <int L>
__device__ __forceinline__ float group_sum(float v, float* red, int group) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (L <= 32) return v;
  constexpr int W = L <= 32 ? 1 : L / 32;
  red += group * W;
  if (threadIdx.x % 32 == 0) red[threadIdx.x % L / 32] = v;
  asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "n"(L) : "memory");
  float t = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) t += red[k];
  return t;
}

// Three sums; red alternates between two areas from row to row.
struct Sums {
  float a, b, c;
};
template <int L>
__device__ __forceinline__ Sums group_sum3(Sums v, Sums* red, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.a += __shfl_xor_sync(0xffffffffu, v.a, o);
    v.b += __shfl_xor_sync(0xffffffffu, v.b, o);
    v.c += __shfl_xor_sync(0xffffffffu, v.c, o);
  }
  if (L == 32) return v;
  constexpr int W = L / 32;
  red += group * W;
  if (threadIdx.x % 32 == 0) red[threadIdx.x % L / 32] = v;
  asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "n"(L) : "memory");
  v = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) {
    const Sums t = red[k];
    v.a += t.a, v.b += t.b, v.c += t.c;
  }
  return v;
}

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

// sigmoid(x) and 1 - sigmoid(x), neither by a difference that cancels.
__device__ __forceinline__ void sigmoid(float x, float& open, float& shut) {
  const float e = __expf(-fabsf(x)), s = __fdividef(1.f, 1.f + e);
  open = x < 0.f ? e * s : s;
  shut = x < 0.f ? s : e * s;
  if (x != x) open = shut = x;
}

__device__ __forceinline__ void fetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---- forward -------------------------------------------------------------------
__host__ __device__ constexpr int fwd_threads(int L) { return L <= 32 ? 128 : L; }

template <typename T, int VEC, int SLOTS, int L, bool GATE>
__global__ void __launch_bounds__(fwd_threads(L)) k_block_norm_fwd(const Fwd a) {
  constexpr int TH = fwd_threads(L), R = TH / L;
  using P = Pack<T, VEC>;
  __shared__ float red[2][L <= 32 ? 1 : L / 32];
  const int lane = threadIdx.x % L;
  const int cols = (int)a.cols;
  const float inv = 1.f / (float)cols;
  int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / L;
  const bool live = row < a.rows;
  if (L >= 32 && !live) return;         // whole warps when L == 32, else never
  if (!live) row = a.rows - 1;          // half a warp: reads, and writes nothing
  const T* hp = static_cast<const T*>(a.h) + row * a.hs + lane * VEC;
  const T* rp = static_cast<const T*>(a.residual) + row * a.rs + lane * VEC;
  const T* gp = GATE ? static_cast<const T*>(a.gate) + row * a.gs + lane * VEC : nullptr;
  auto in = [&](int s) { return (s * L + lane) * VEC < cols; };
  P ph[SLOTS], pr[SLOTS], pg[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
    ph[s] = *reinterpret_cast<const P*>(hp + s * L * VEC);
    pr[s] = *reinterpret_cast<const P*>(rp + s * L * VEC);
    if (GATE) pg[s] = *reinterpret_cast<const P*>(gp + s * L * VEC);
  }
  // The weights are wanted after a sum: a small call fetches them meanwhile.
  if (gridDim.x <= 256) {
    const size_t size = a.wtype == LOPT_F32 ? 4 : sizeof(T);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (!in(s)) continue;
      fetch_line(static_cast<const char*>(a.w_post) + (s * L + lane) * VEC * size);
      fetch_line(static_cast<const char*>(a.w_pre) + (s * L + lane) * VEC * size);
    }
  }
  float v[SLOTS][VEC];
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
    to_floats(ph[s], v[s]);
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum = fmaf(v[s][k], v[s][k], sum);
  }
  const float r1 = rsqrtf(group_sum<L>(sum, red[0], 0) * inv + a.eps);
  sum = 0.f;
  T* sp = static_cast<T*>(a.summed) + row * a.ss + lane * VEC;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
    float w[VEC], r[VEC];
    load_weights<T, VEC>(a.w_post, a.wtype, (s * L + lane) * VEC, w);
    to_floats(pr[s], r);
    if (GATE) {
      float g[VEC];
      to_floats(pg[s], g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float open, shut;
        sigmoid(g[k], open, shut);
        w[k] *= open;
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      v[s][k] = fmaf(v[s][k] * r1 * w[k], a.scale, r[k]);
      sum = fmaf(v[s][k], v[s][k], sum);
    }
    if (live) *reinterpret_cast<P*>(sp + s * L * VEC) = from_floats<T, VEC>(v[s]);
  }
  const float r2 = rsqrtf(group_sum<L>(sum, red[1], 0) * inv + a.eps);
  if (!live) return;
  if (lane == 0) {
    a.rstd_post[row] = r1;
    a.rstd_pre[row] = r2;
  }
  T* yp = static_cast<T*>(a.y) + row * a.ys + lane * VEC;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
    float w[VEC];
    load_weights<T, VEC>(a.w_pre, a.wtype, (s * L + lane) * VEC, w);
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[k] *= v[s][k] * r2;
    *reinterpret_cast<P*>(yp + s * L * VEC) = from_floats<T, VEC>(w);
  }
}

// Rows too long for registers: read three times, from L2 after the first.
template <typename T>
__global__ void __launch_bounds__(512) k_block_norm_fwd_long(const Fwd a) {
  constexpr int L = 512;
  __shared__ float red[2][L / 32];
  const int64_t row = blockIdx.x;
  const T* h = static_cast<const T*>(a.h) + row * a.hs;
  const T* r = static_cast<const T*>(a.residual) + row * a.rs;
  const T* g = a.gate ? static_cast<const T*>(a.gate) + row * a.gs : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ys;
  T* sm = static_cast<T*>(a.summed) + row * a.ss;
  const float inv = 1.f / (float)a.cols;
  float sum = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) sum = fmaf(to_f(h[j]), to_f(h[j]), sum);
  const float r1 = rsqrtf(group_sum<L>(sum, red[0], 0) * inv + a.eps);
  auto make = [&](int64_t j) {
    float w[1], open = 1.f, shut;
    load_weights<T, 1>(a.w_post, a.wtype, j, w);
    if (g) sigmoid(to_f(g[j]), open, shut);
    return fmaf(to_f(h[j]) * r1 * (w[0] * open), a.scale, to_f(r[j]));
  };
  sum = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    const float v = make(j);
    sum = fmaf(v, v, sum);
  }
  const float r2 = rsqrtf(group_sum<L>(sum, red[1], 0) * inv + a.eps);
  if (threadIdx.x == 0) {
    a.rstd_post[row] = r1;
    a.rstd_pre[row] = r2;
  }
  for (int64_t j = threadIdx.x; j < a.cols; j += L) {
    const float v = make(j);      // before either store: both may be in place
    float w[1];
    load_weights<T, 1>(a.w_pre, a.wtype, j, w);
    sm[j] = from_f<T>(v);
    y[j] = from_f<T>(v * r2 * w[0]);
  }
}

// ---- backward ------------------------------------------------------------------
// Threads of a block, of which an SM takes one: 16 warps with 128 registers, 12 with 168
// where a lane has 24 elements.  24 warps spilled and were slower (32,768 x 2048 bfloat16 with
// 8 elements a lane 341 us against 185).  The forms of 16-byte accesses do not spill, but for
// float32 rows above 8,192; of those of single elements the widest do, by up to 230 bytes.
__host__ __device__ constexpr int bwd_threads(int E, int L) { return E == 24 ? 384 : L % 96 == 0 ? 480 : 512; }

// Rows of whole vectors come ahead into shared memory: every thread copies its own 16
// bytes of each array asynchronously and reads them back itself, so that no barrier is
// needed; slots of rows of at most 5 arrays.
__host__ __device__ constexpr bool bwd_ring(int vec, int slots, int L, int es) {
  return vec * es == 16 && bwd_threads(vec * slots, L) * slots * 16 * 5 * 2 <= 200 * 1024;
}
__host__ __device__ constexpr int bwd_depth(int vec, int slots, int L) {
  return bwd_threads(vec * slots, L) * slots * 16 * 5 * 3 <= 200 * 1024 ? 3 : 2;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}

// Persistent: a block's groups of L threads take rows blockIdx.x * R + group,
// striding by gridDim.x * R.
template <typename T, int VEC, int SLOTS, int L, bool GATE>
__global__ void __launch_bounds__(bwd_threads(VEC * SLOTS, L), 1) k_block_norm_bwd(const Bwd a) {
  constexpr int TH = bwd_threads(VEC * SLOTS, L), R = TH / L, W = L * VEC * SLOTS;
  using P = Pack<T, VEC>;
  __shared__ Sums red[2][TH / 32];
  // The rows ahead, and at the end the groups' sums: [2][R][W]
  extern __shared__ __align__(16) float comb[];
  constexpr bool RING = bwd_ring(VEC, SLOTS, L, sizeof(T));
  constexpr int DEPTH = bwd_depth(VEC, SLOTS, L);
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int cols = (int)a.cols;
  const float inv = 1.f / (float)cols;
  const int64_t stride = (int64_t)gridDim.x * R;
  const bool sums = a.dsum != nullptr;
  let_next_start();
  auto in = [&](int s) { return (s * L + lane) * VEC < cols; };
  float dw1[SLOTS][VEC], dw2[SLOTS][VEC];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw1[s][k] = dw2[s][k] = 0.f;
  enum { kDy, kX, kH, kSum, kGate, kArrays };
  const void* const base[kArrays] = {a.dy, a.summed, a.h, a.dsum, a.gate};
  const int64_t strides[kArrays] = {a.dys, a.xs, a.hs, a.dss, a.gs};
  auto slot = [&](int d, int k, int s) { return (((d * kArrays + k) * SLOTS + s) * TH + threadIdx.x) * 16; };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(comb);
  auto fetch = [&](int64_t r, int d) {
    if (r < a.rows) {
#pragma unroll
      for (int k = 0; k < kArrays; ++k) {
        if ((k == kSum && !sums) || (k == kGate && !GATE)) continue;
        const T* p = static_cast<const T*>(base[k]) + r * strides[k] + lane * VEC;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
          if (in(s)) copy16(ring + slot(d, k, s), p + s * L * VEC);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = (int64_t)blockIdx.x * R + group;
  if (RING) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(row + d * stride, d);
  }
  float r1 = 0.f, r2 = 0.f;
  if (row < a.rows) r1 = a.rstd_post[row], r2 = a.rstd_pre[row];
  for (int par = 0, d = 0; row < a.rows; row += stride, par ^= 1) {
    P own[kArrays][SLOTS];
    float r1_next = 0.f, r2_next = 0.f;
    if (row + stride < a.rows) r1_next = a.rstd_post[row + stride], r2_next = a.rstd_pre[row + stride];
    if (RING) {
      asm volatile("cp.async.wait_group %0;" :: "n"(DEPTH - 1) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < kArrays; ++k) {
        if ((k == kSum && !sums) || (k == kGate && !GATE)) continue;
        const T* p = static_cast<const T*>(base[k]) + row * strides[k] + lane * VEC;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
          if (in(s)) own[k][s] = *reinterpret_cast<const P*>(p + s * L * VEC);
      }
    }
    auto get = [&](int k, int s, float (&v)[VEC]) {
      if constexpr (RING) to_floats(*reinterpret_cast<const P*>(reinterpret_cast<const char*>(comb) + slot(d, k, s)), v);
      else to_floats(own[k][s], v);
    };
    float A[SLOTS][VEC];
    Sums t{0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (!in(s)) continue;
      float dy[VEC], x[VEC], w[VEC], h[VEC];
      get(kDy, s, dy);
      get(kX, s, x);
      load_weights<T, VEC>(a.w_pre, a.wtype, (s * L + lane) * VEC, w);
      if (sums) get(kSum, s, A[s]);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float dx = dy[k] * x[k];
        dw2[s][k] = fmaf(dx, r2, dw2[s][k]);
        t.a = fmaf(dx, w[k], t.a);
        A[s][k] = fmaf(dy[k] * w[k], r2, sums ? A[s][k] : 0.f);
      }
      load_weights<T, VEC>(a.w_post, a.wtype, (s * L + lane) * VEC, w);
      get(kH, s, h);
      if (GATE) get(kGate, s, dy);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float u = h[k] * w[k];
        if (GATE) {
          float open, shut;
          sigmoid(dy[k], open, shut);
          u *= open;
        }
        t.b = fmaf(u, A[s][k], t.b);
        t.c = fmaf(u, x[k], t.c);
      }
    }
    t = group_sum3<L>(t, red[par], group);
    T* to_r = static_cast<T*>(a.dres) + row * a.drs + lane * VEC;
    T* to_g = static_cast<T*>(a.dgate) + row * a.dgs + lane * VEC;
    T* to_h = static_cast<T*>(a.dh) + row * a.dhs + lane * VEC;
    // From xhat = f2(summed) and hhat = f1(h), or from the rows themselves with the roots in
    // the coefficients, which spares three products an element (32,768 x 2048 bfloat16 144
    // us, 166 with them).  Their cubes are then in these, so that only rows of ordinary size may.
    auto gradients = [&](float c1, float c2, auto f2, auto f1, float scale, auto last) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (!in(s)) continue;
        float x[VEC], w[VEC], h[VEC];
        get(kX, s, x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) A[s][k] = fmaf(f2(x[k]), c1, A[s][k]);
        *reinterpret_cast<P*>(to_r + s * L * VEC) = from_floats<T, VEC>(A[s]);
        load_weights<T, VEC>(a.w_post, a.wtype, (s * L + lane) * VEC, w);
        get(kH, s, h);
        if (GATE) get(kGate, s, x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          float dz = A[s][k] * scale, shut = 0.f;
          if (GATE) {
            float open;
            sigmoid(x[k], open, shut);
            dz *= open;
          }
          h[k] = f1(h[k]);
          dw1[s][k] = fmaf(dz, h[k], dw1[s][k]);
          const float q = dz * w[k];
          if (GATE) x[k] = q * h[k] * shut;
          h[k] = last(fmaf(h[k], c2, q));
        }
        if (GATE) *reinterpret_cast<P*>(to_g + s * L * VEC) = from_floats<T, VEC>(x);
        *reinterpret_cast<P*>(to_h + s * L * VEC) = from_floats<T, VEC>(h);
      }
    };
    auto same = [](float v) { return v; };
    if (fminf(r1, r2) > 0x1p-24f && fmaxf(r1, r2) < 0x1p24f) {
      const float c1 = -r2 * r2 * r2 * (t.a * inv);
      gradients(c1, -r1 * r1 * r1 * a.scale * (fmaf(c1, t.c, t.b) * inv), same, same, a.scale * r1, same);
    } else {
      auto times1 = [&](float v) { return v * r1; };
      auto times2 = [&](float v) { return v * r2; };
      const float c1 = -r2 * (r2 * (t.a * inv));
      gradients(c1, -a.scale * (fmaf(c1, r1 * (r2 * t.c), r1 * t.b) * inv), times2, times1, a.scale, times1);
    }
    r1 = r1_next, r2 = r2_next;
    if (RING) {
      fetch(row + DEPTH * stride, d);
      if (++d == DEPTH) d = 0;
    }
  }
  if (RING) {      // the ring's place is wanted for the sums
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
  }
  // The block's sums: over its groups in order.
  float* p1 = a.part + (int64_t)blockIdx.x * cols;
  const int64_t second = (int64_t)gridDim.x * cols;
  float* to1 = R == 1 ? p1 : comb + group * W;
  float* to2 = R == 1 ? p1 + second : comb + (R + group) * W;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    if (!in(s)) continue;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      to1[(s * L + lane) * VEC + k] = dw1[s][k];
      to2[(s * L + lane) * VEC + k] = dw2[s][k];
    }
  }
  if (R > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * W; c += TH) {
      const int half = c / W, j = c % W;
      if (j >= cols) continue;
      float t = 0.f;
#pragma unroll
      for (int g = 0; g < R; ++g) t += comb[(half * R + g) * W + j];
      p1[half * second + j] = t;
    }
  }
}

// Rows too long for registers, in three kernels: sum(g xhat) of each row; the
// column sums, before anything may be overwritten in place; the gradients.
template <typename T> struct LongRow {
  const T *dy, *x, *h, *g, *ds;
  float r1, r2;
  const Bwd& a;
  __device__ LongRow(const Bwd& b, int64_t row)
      : dy(static_cast<const T*>(b.dy) + row * b.dys), x(static_cast<const T*>(b.summed) + row * b.xs),
        h(static_cast<const T*>(b.h) + row * b.hs), g(b.gate ? static_cast<const T*>(b.gate) + row * b.gs : nullptr),
        ds(b.dsum ? static_cast<const T*>(b.dsum) + row * b.dss : nullptr), r1(b.rstd_post[row]), r2(b.rstd_pre[row]), a(b) {}
  __device__ float weight(const void* p, int64_t j) const {
    float w[1];
    load_weights<T, 1>(p, a.wtype, j, w);
    return w[0];
  }
  __device__ float grad_sum(int64_t j, float coef) const {
    const float o = r2 * (to_f(dy[j]) * weight(a.w_pre, j) - to_f(x[j]) * r2 * coef);
    return ds ? o + to_f(ds[j]) : o;
  }
  // dz, and 1 - open
  __device__ float dz(int64_t j, float o, float& shut) const {
    float open = 1.f;
    shut = 0.f;
    if (g) sigmoid(to_f(g[j]), open, shut);
    return o * a.scale * open;
  }
};

template <typename T>
__global__ void __launch_bounds__(512) k_block_norm_coef_long(const Bwd a) {
  __shared__ float red[16];
  const LongRow<T> q(a, blockIdx.x);
  float sg = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += 512)
    sg = fmaf(to_f(q.dy[j]) * q.weight(a.w_pre, j), to_f(q.x[j]) * q.r2, sg);
  sg = group_sum<512>(sg, red, 0);
  if (threadIdx.x == 0) a.coef[blockIdx.x] = sg / (float)a.cols;
}

template <typename T>
__global__ void __launch_bounds__(256) k_block_norm_cols_long(const Bwd a) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= a.cols) return;
  const int64_t per = (a.rows + gridDim.y - 1) / gridDim.y;
  const int64_t end = min(a.rows, per * (blockIdx.y + 1));
  float d1 = 0.f, d2 = 0.f;
  for (int64_t row = per * blockIdx.y; row < end; ++row) {
    const LongRow<T> q(a, row);
    float shut;
    const float dz = q.dz(j, q.grad_sum(j, a.coef[row]), shut);
    d1 = fmaf(dz, to_f(q.h[j]) * q.r1, d1);
    d2 = fmaf(to_f(q.dy[j]), to_f(q.x[j]) * q.r2, d2);
  }
  a.part[(int64_t)blockIdx.y * a.cols + j] = d1;
  a.part[((int64_t)gridDim.y + blockIdx.y) * a.cols + j] = d2;
}

template <typename T>
__global__ void __launch_bounds__(512) k_block_norm_bwd_long(const Bwd a) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const LongRow<T> q(a, row);
  T* dh = static_cast<T*>(a.dh) + row * a.dhs;
  T* dr = static_cast<T*>(a.dres) + row * a.drs;
  T* dg = a.dgate ? static_cast<T*>(a.dgate) + row * a.dgs : nullptr;
  const float coef = a.coef[row];
  float sq = 0.f;
  for (int64_t j = threadIdx.x; j < a.cols; j += 512) {
    float shut;
    const float dz = q.dz(j, q.grad_sum(j, coef), shut);
    sq = fmaf(dz * q.weight(a.w_post, j), to_f(q.h[j]) * q.r1, sq);
  }
  const float c2 = group_sum<512>(sq, red, 0) / (float)a.cols;
  for (int64_t j = threadIdx.x; j < a.cols; j += 512) {
    const float o = q.grad_sum(j, coef);
    float shut;
    const float qw = q.dz(j, o, shut) * q.weight(a.w_post, j), hh = to_f(q.h[j]) * q.r1;
    // All of the column is read: the stores may be in place.
    dr[j] = from_f<T>(o);
    dh[j] = from_f<T>(q.r1 * (qw - hh * c2));
    if (dg) dg[j] = from_f<T>(qw * hh * shut);
  }
}

// The blocks' sums of 32 columns: warp w adds blocks w, w + 8, ..., then one
// warp the eight sums in order.  blockIdx.y: which weight.
__global__ void __launch_bounds__(256) k_block_norm_finish(const float* part, int blocks, int64_t cols, float* d1,
                                                           float* d2, int accumulate) {
  __shared__ float red[8][32];
  float* out = blockIdx.y ? d2 : d1;
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

template <typename T> struct FwdRun {
  const Fwd& a;
  cudaStream_t s;
  template <int V, int S, int L> cudaError_t run() {
    constexpr int R = fwd_threads(L) / L;
    return launch(a.gate ? k_block_norm_fwd<T, V, S, L, true> : k_block_norm_fwd<T, V, S, L, false>,
                  dim3((unsigned)((a.rows + R - 1) / R)), dim3(fwd_threads(L)), 0, s, false, 1, a);
  }
  cudaError_t long_rows() { return launch(k_block_norm_fwd_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a); }
};

template <typename T> struct BwdRun {
  const Bwd& a;
  int sms;
  cudaStream_t s;
  int* blocks;
  template <int V, int S, int L, bool G> cudaError_t run_as() {
    constexpr int TH = bwd_threads(V * S, L), R = TH / L;
    const size_t ring = bwd_ring(V, S, L, sizeof(T)) ? (size_t)bwd_depth(V, S, L) * 5 * S * TH * 16 : 0;
    const size_t smem = std::max(ring, R > 1 ? (size_t)TH * V * S * 8 : (size_t)0);
    auto* k = &k_block_norm_bwd<T, V, S, L, G>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
    if (e != cudaSuccess) return e;
    *blocks = (int)std::min<int64_t>({(a.rows + R - 1) / R, (int64_t)sms, kMaxBlocks});
    return launch(k, dim3((unsigned)*blocks), dim3(TH), smem, s, false, 1, a);
  }
  template <int V, int S, int L> cudaError_t run() { return a.gate ? run_as<V, S, L, true>() : run_as<V, S, L, false>(); }
  cudaError_t long_rows() {
    *blocks = (int)std::min<int64_t>(a.rows, 32);
    cudaError_t e = launch(k_block_norm_coef_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.cols + 255) / 256), (unsigned)*blocks);
    e = launch(k_block_norm_cols_long<T>, grid, dim3(256), 0, s, false, 1, a);
    if (e != cudaSuccess) return e;
    return launch(k_block_norm_bwd_long<T>, dim3((unsigned)a.rows), dim3(512), 0, s, false, 1, a);
  }
};

// Slots and threads by the row's accesses of V elements.  Forward: half a warp for the
// shortest; a warp, with up to 24 elements a lane, while that holds a row; then 16 (us,
// bfloat16 with a gate: 65,536 x 768 77.8 by warps, 86.8 by 96 threads; 32,768 x 1024
// 53.2 by 64 threads, 60.1 by 128; 16,384 x 2048 54.1 by 128, 62.4 by 256; 8,192 x 4096
// 58.3 by 256, 68.3 by 512).  Without a gate: 16,384 x 2048 float32 82; single elements
// 32,768 x 2001 bfloat16 113 (82 at 2000), 16,384 x 2001 float32 109; 4,096 x 16,384 bfloat16
// 127, floor 79; read three times, 2,048 x 20,000 150, floor 48.
#define LOPT_ROWS(V, S, L_) if (n <= (int64_t)(S) * (L_)) return f.template run<V, S, L_>()
template <int FULL, typename F> cudaError_t pick_fwd(int64_t cols, bool vec, F f) {
  if (vec) {
    constexpr int B = 8 / FULL;   // slots of 8 elements
    const int64_t n = cols / FULL;
    LOPT_ROWS(FULL, 1, 16);
    LOPT_ROWS(FULL, 1, 32);
    LOPT_ROWS(FULL, 2 * B, 32);
    LOPT_ROWS(FULL, 3 * B, 32);
    LOPT_ROWS(FULL, 2 * B, 64);
    LOPT_ROWS(FULL, 2 * B, 128);
    LOPT_ROWS(FULL, 2 * B, 256);
    LOPT_ROWS(FULL, 2 * B, 512);
    LOPT_ROWS(FULL, 4 * B, 512);
  } else {
    const int64_t n = cols;
    LOPT_ROWS(1, 4, 32);
    LOPT_ROWS(1, 16, 32);
    LOPT_ROWS(1, 8, 128);
    LOPT_ROWS(1, 8, 256);
    LOPT_ROWS(1, 16, 512);
  }
  return f.long_rows();
}
// Backward in 16 bits: a lane takes 16 elements (a row's sum costs the same whatever
// it has), a warp alone up to 24; in 32 bits 8 (us, 2048 wide, 33.5M elements float32 138
// with 8, 203 with 16; 67M bfloat16 183 with 8, 144 with 16, 166 with 24, 342 with 32; with a
// gate 256, 195, 220, 493; 50M 768 wide with a gate 204 with 8 by 96 threads, 154 with 24 by
// a warp).  Single elements: 32,768 x 2001 bfloat16 273 us (152 at 2000), 16,384 x 2001
// float32 177 (145 at 2048).  Longer rows: 4,096 x 12,288 bfloat16 472 us, floor 89.
template <int FULL, typename F> cudaError_t pick_bwd(int64_t cols, bool vec, F f) {
  if (vec) {
    const int64_t n = cols / FULL;
    if constexpr (FULL == 8) {
      LOPT_ROWS(8, 1, 32);
      LOPT_ROWS(8, 2, 32);
      LOPT_ROWS(8, 3, 32);
      LOPT_ROWS(8, 2, 64);
      LOPT_ROWS(8, 2, 128);
      LOPT_ROWS(8, 2, 256);
      LOPT_ROWS(8, 2, 512);
    } else {
      LOPT_ROWS(4, 2, 32);
      LOPT_ROWS(4, 2, 64);
      LOPT_ROWS(4, 2, 96);
      LOPT_ROWS(4, 2, 128);
      LOPT_ROWS(4, 2, 256);
      LOPT_ROWS(4, 2, 512);
      LOPT_ROWS(4, 4, 512);
    }
  } else {
    const int64_t n = cols;
    LOPT_ROWS(1, 4, 32);
    LOPT_ROWS(1, 8, 64);
    LOPT_ROWS(1, 8, 128);
    LOPT_ROWS(1, 8, 256);
    LOPT_ROWS(1, 8, 512);
    LOPT_ROWS(1, 16, 512);
  }
  return f.long_rows();
}

bool vec_ok(int64_t cols, int es, std::initializer_list<Span> ms, const void* w1, const void* w2) {
  if ((cols * es) % 16) return false;
  for (const Span& m : ms)
    if (!rows_aligned(m, 16)) return false;
  return (uintptr_t)w1 % 16 == 0 && (uintptr_t)w2 % 16 == 0;
}

int check_weight(const void* w, int wtype, int type) {
  if (!w) return LOPT_E_ARG;
  if (wtype != LOPT_F32 && wtype != type) return LOPT_E_ARG;
  return (uintptr_t)w % type_size(wtype) ? LOPT_E_ALIGN : LOPT_OK;
}

// Outputs against each other and against inputs; the first `in_place` outputs
// may stand in the place of the first `replaceable` inputs.
int check_alias(std::initializer_list<Span> outs, int in_place, std::initializer_list<Span> ins, int replaceable) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return LOPT_E_ALIAS;
    for (auto i = ins.begin(); i != ins.end(); ++i)
      if (overlap(*o, *i) && !(o - outs.begin() < in_place && i - ins.begin() < replaceable && o->same_place(*i)))
        return LOPT_E_ALIAS;
  }
  return LOPT_OK;
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_block_norm_forward(const void* h, int type, int64_t rows, int64_t cols, int64_t h_stride, const void* residual,
                            int64_t residual_stride, const void* gate, int64_t gate_stride, const void* w_post,
                            const void* w_pre, int weight_type, float scale, float eps, void* y, int64_t y_stride,
                            void* summed, int64_t summed_stride, float* rstd_post, float* rstd_pre, void* stream) {
  const int es = type_size(type);
  if (!es || !(eps >= 0.f) || !std::isfinite(scale)) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols) return LOPT_E_SHAPE;
  if (rows == 0) return LOPT_OK;
  const Span mh{h, rows, cols, h_stride, es}, mr{residual, rows, cols, residual_stride, es};
  const Span mg{gate, rows, cols, gate_stride, es}, my{y, rows, cols, y_stride, es};
  const Span ms{summed, rows, cols, summed_stride, es};
  const Span s1{rstd_post, 1, rows, rows, 4}, s2{rstd_pre, 1, rows, rows, 4};
  int rc;
  if ((rc = check_matrix(mh, false)) || (rc = check_matrix(mr, false)) || (gate && (rc = check_matrix(mg, false))) ||
      (rc = check_matrix(my, true)) || (rc = check_matrix(ms, true)) || (rc = check_matrix(s1, true)) ||
      (rc = check_matrix(s2, true)) || (rc = check_weight(w_post, weight_type, type)) ||
      (rc = check_weight(w_pre, weight_type, type)))
    return rc;
  const int wes = type_size(weight_type);
  if ((rc = check_alias({my, ms, s1, s2}, 2, {mh, mr, mg, Span{w_post, 1, cols, cols, wes}, Span{w_pre, 1, cols, cols, wes}}, 3)))
    return rc;
  const Fwd a{h, residual, gate, w_post, w_pre, y, summed, rstd_post, rstd_pre, rows, cols,
              h_stride, residual_stride, gate_stride, y_stride, summed_stride, weight_type, scale, eps};
  const bool vec = vec_ok(cols, es, {mh, mr, mg, my, ms}, w_post, w_pre);
  cudaStream_t s = (cudaStream_t)stream;
  switch (type) {
    case LOPT_F32: return done(pick_fwd<4>(cols, vec, FwdRun<float>{a, s}));
    case LOPT_F16: return done(pick_fwd<8>(cols, vec, FwdRun<__half>{a, s}));
    default: return done(pick_fwd<8>(cols, vec, FwdRun<__nv_bfloat16>{a, s}));
  }
}

int lopt_block_norm_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes) return LOPT_E_ARG;
  if (rows < 0 || cols < 1 || rows >= kMaxRows || cols > kMaxCols) return LOPT_E_SHAPE;
  // the blocks' sums, then a coefficient per row
  *bytes = 2 * std::min<int64_t>(std::max<int64_t>(rows, 1), kMaxBlocks) * cols * 4 + rows * 4;
  return LOPT_OK;
}

int lopt_block_norm_backward(const void* grad_y, int type, int64_t rows, int64_t cols, int64_t grad_y_stride,
                             const void* h, int64_t h_stride, const void* summed, int64_t summed_stride,
                             const void* gate, int64_t gate_stride, const float* rstd_post, const float* rstd_pre,
                             const void* w_post, const void* w_pre, int weight_type, float scale,
                             const void* grad_summed, int64_t grad_summed_stride, void* grad_h, int64_t grad_h_stride,
                             void* grad_residual, int64_t grad_residual_stride, void* grad_gate,
                             int64_t grad_gate_stride, float* grad_w_post, float* grad_w_pre, int accumulate,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const int es = type_size(type);
  if (!es || !std::isfinite(scale) || (accumulate != 0 && accumulate != 1) || !gate != !grad_gate) return LOPT_E_ARG;
  int64_t need = 0;
  int rc = lopt_block_norm_workspace(rows, cols, &need);
  if (rc) return rc;
  const Span g1{grad_w_post, 1, cols, cols, 4}, g2{grad_w_pre, 1, cols, cols, 4};
  if ((rc = check_matrix(g1, true)) || (rc = check_matrix(g2, true))) return rc;
  if (overlap(g1, g2)) return LOPT_E_ALIAS;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    if (accumulate) return LOPT_OK;
    cudaError_t e = cudaMemsetAsync(grad_w_post, 0, cols * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(grad_w_pre, 0, cols * 4, s);
    return done(e);
  }
  const Span md{grad_y, rows, cols, grad_y_stride, es}, mh{h, rows, cols, h_stride, es};
  const Span mx{summed, rows, cols, summed_stride, es}, mg{gate, rows, cols, gate_stride, es};
  const Span ms{grad_summed, rows, cols, grad_summed_stride, es};
  const Span oh{grad_h, rows, cols, grad_h_stride, es}, og{grad_gate, rows, cols, grad_gate_stride, es};
  const Span od{grad_residual, rows, cols, grad_residual_stride, es};
  const Span s1{rstd_post, 1, rows, rows, 4}, s2{rstd_pre, 1, rows, rows, 4};
  const int wes = type_size(weight_type);
  if ((rc = check_matrix(md, false)) || (rc = check_matrix(mh, false)) || (rc = check_matrix(mx, false)) ||
      (gate && ((rc = check_matrix(mg, false)) || (rc = check_matrix(og, true)))) ||
      (grad_summed && (rc = check_matrix(ms, false))) || (rc = check_matrix(oh, true)) || (rc = check_matrix(od, true)) ||
      (rc = check_matrix(s1, false)) || (rc = check_matrix(s2, false)) ||
      (rc = check_weight(w_post, weight_type, type)) || (rc = check_weight(w_pre, weight_type, type)))
    return rc;
  if (!workspace || workspace_bytes < need) return LOPT_E_ARG;
  if ((uintptr_t)workspace % 256) return LOPT_E_ALIGN;
  if ((rc = check_alias({oh, od, og, g1, g2, Span{workspace, 1, need, need, 1}}, 3,
                        {md, mh, mx, mg, ms, s1, s2, Span{w_post, 1, cols, cols, wes}, Span{w_pre, 1, cols, cols, wes}}, 5)))
    return rc;
  float* part = (float*)workspace;
  const Bwd a{grad_y, h, summed, gate, grad_summed, w_post, w_pre, rstd_post, rstd_pre, grad_h, grad_residual, grad_gate,
              part, part + (need / 4 - rows), rows, cols, grad_y_stride, h_stride, summed_stride, gate_stride,
              grad_summed_stride, grad_h_stride, grad_residual_stride, grad_gate_stride, weight_type, scale};
  const bool vec = vec_ok(cols, es, {md, mh, mx, mg, ms, oh, od, og}, w_post, w_pre);
  const int sms = sm_count();
  int blocks = 0;
  cudaError_t e;
  switch (type) {
    case LOPT_F32: e = pick_bwd<4>(cols, vec, BwdRun<float>{a, sms, s, &blocks}); break;
    case LOPT_F16: e = pick_bwd<8>(cols, vec, BwdRun<__half>{a, sms, s, &blocks}); break;
    default: e = pick_bwd<8>(cols, vec, BwdRun<__nv_bfloat16>{a, sms, s, &blocks}); break;
  }
  if (e != cudaSuccess) return done(e);
  return done(launch(k_block_norm_finish, dim3((unsigned)((cols + 31) / 32), 2u), dim3(256), 0, s, true, 1,
                     (const float*)part, blocks, cols, grad_w_post, grad_w_pre, accumulate));
}

}  // extern "C"
