// AdamW over a list of tensors (see lopt_lm.h for the formulas).
//
// One pass over param, grad and the moments; bound by HBM bytes (28 a float32
// element, 30 with a 16-bit copy, 16 with 8-bit moments and 16-bit gradients).  Tensors that
// are not on 16-byte boundaries go element by element: 100M with bfloat16 gradients and copy
// 516 us (432 on them), with 8-bit moments 501 (367).
// The list travels in the kernel's parameters, so a step copies nothing to the
// device and may be captured.  1.31G float32 elements with a bfloat16 copy take 5.64 ms
// (7.0 TB/s), the norm of their gradients before it 0.79 ms (6.6 TB/s); 304M elements with
// 8-bit moments, bfloat16 gradients and copy 1.06 ms (4.6 TB/s: some 100 instructions an
// element, 81 % of the issue slots).  A warp takes 256 consecutive elements, eight a
// lane: they are one block of 8-bit moments, whose largest value is a few
// shuffles away.
//
// Every operation is rounded on its own (the __f*_rn intrinsics are not fused),
// so that the codes of 8-bit moments are those of the formulas bit for bit.
#include <algorithm>
#include <cmath>
#include <vector>

#include "lopt_lm.h"
#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

constexpr int kUnit = LOPT_ADAMW_BLOCK;   // elements of a warp
constexpr int kWarps = 8;

struct Desc {
  float* param;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  void* copy;
  int64_t n;
  uint32_t key;
  int32_t first;      // its first chunk in the launch
  uint8_t grad_type, copy_type, decay, vec;
  int32_t pad;
};
static_assert(sizeof(Desc) == 80, "");

// Kernel parameters hold up to 32,764 bytes; small lists take the small form,
// whose parameters are quicker to send.
template <int N> struct List {
  Desc d[N];
};
constexpr int kSmall = 24, kLarge = 400;

struct Hyper {
  float b1, nb1, b2, nb2, c1, c2, eps, keep;   // nb = 1 - b; c1 = lr / (1 - b1^t); c2 = 1 / sqrt(1 - b2^t); keep = 1 - lr * decay
  const double* part;                          // sums of squares of the gradients; NULL: no clipping
  int parts;
  double max_norm;
  float* norm;
  int count, units;                            // tensors; warp units of a chunk
  float minus_zero;                            // see Mul
};

// Two fp32 operations as one instruction, each rounded on its own.  A product is a
// fused multiply-add of -0, which has to come from the launch's parameters: the
// compiler joins mul.f32x2 (or one with a -0 that it knows) and add.f32x2, though
// both say .rn.
__device__ __forceinline__ uint64_t packed(float2 v) { return (uint64_t)__float_as_uint(v.y) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ float2 unpacked(uint64_t v) { return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(packed(a)), "l"(packed(b)));
  return unpacked(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(packed(a)), "l"(packed(b)), "l"(packed(c)));
  return unpacked(r);
}

struct Mul {
  float2 zero;
  __device__ __forceinline__ explicit Mul(float minus_zero) : zero(make_float2(minus_zero, minus_zero)) {}
  __device__ __forceinline__ float2 operator()(float2 a, float2 b) const { return fma2(a, b, zero); }
};

__host__ __device__ inline uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85ebca6bu;
  h ^= h >> 13;
  h *= 0xc2b2ae35u;
  return h ^ (h >> 16);
}

// The tensor of a chunk: the last whose first chunk is not behind it.
template <int N>
__device__ __forceinline__ int find(const List<N>& list, int count, int chunk) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.d[mid].first <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A lane's eight elements of a unit.  In vectors: four from lane * 4 on and
// four more 128 behind; one by one: every 32nd.
__device__ __forceinline__ int place(bool vec, int lane, int k) {
  return vec ? (k / 4) * 128 + lane * 4 + k % 4 : k * 32 + lane;
}

template <typename T, typename F>
__device__ __forceinline__ void load8(const T* p, bool vec, int lane, int left, F put) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Pack<T, 4> q = *reinterpret_cast<const Pack<T, 4>*>(p + j * 128 + lane * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) put(j * 4 + e, q.v[e]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) put(k, k * 32 + lane < left ? p[k * 32 + lane] : T(0));
  }
}
template <typename T, typename F>
__device__ __forceinline__ void store8(T* p, bool vec, int lane, int left, F get) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      Pack<T, 4> q;
#pragma unroll
      for (int e = 0; e < 4; ++e) q.v[e] = get(j * 4 + e);
      *reinterpret_cast<Pack<T, 4>*>(p + j * 128 + lane * 4) = q;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 32 + lane < left) p[k * 32 + lane] = get(k);
  }
}

__device__ __forceinline__ void load_grad(const Desc& d, int64_t at, bool vec, int lane, int left, float (&g)[8]) {
  if (d.grad_type == LOPT_F32)
    load8(static_cast<const float*>(d.grad) + at, vec, lane, left, [&](int k, float x) { g[k] = x; });
  else if (d.grad_type == LOPT_F16)
    load8(static_cast<const __half*>(d.grad) + at, vec, lane, left, [&](int k, __half x) { g[k] = __half2float(x); });
  else
    load8(static_cast<const __nv_bfloat16*>(d.grad) + at, vec, lane, left,
          [&](int k, __nv_bfloat16 x) { g[k] = __bfloat162float(x); });
}

__device__ __forceinline__ float decode(int q, float scale) { return __fmul_rn((float)(q * abs(q)), scale); }

// Largest |x| of a warp; NaN if any is.
__device__ __forceinline__ float largest(const float (&x)[8]) {
  float most = fabsf(x[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(x[k])));
  // Above 0 the bits are in the values' order, and NaN's are above infinity's.
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu));
}

__device__ __forceinline__ void fetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 8-bit moments, two elements at a time.  Conversions between small integers and
// floats go through the bits of 2^23 + integer: the conversion instructions run at an
// eighth of the rate.
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
constexpr float k2p23 = 8388608.f;
constexpr float kCode = 12582912.f;   // 1.5 * 2^23: kCode + q has the low byte of q, below 0 too

// Bytes 2 * PAIR and 2 * PAIR + 1 of w, minus `bias`.
template <int PAIR> __device__ __forceinline__ float2 bytes(uint32_t w, float bias) {
  const float2 f = make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 | (2 * PAIR))),
                               __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 | (2 * PAIR + 1))));
  return add2(f, two(-k2p23 - bias));
}

__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
  const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// A lane's eight codes, four in a word.
__device__ __forceinline__ void load_codes(const uint8_t* p, bool vec, int lane, int left, uint32_t (&w)[2]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = *reinterpret_cast<const uint32_t*>(p + j * 128 + lane * 4);
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 32 + lane < left) w[k / 4] |= (uint32_t)p[k * 32 + lane] << (8 * (k % 4));
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, bool vec, int lane, int left, const uint32_t (&w)[2]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<uint32_t*>(p + j * 128 + lane * 4) = w[j];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k * 32 + lane < left) p[k * 32 + lane] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
  }
}

// The codes of |x| = y / inv units, 0 to TOP: floor(sqrt(y)), or one more where the
// random number u = bits / 2^16 is below y's place between the two squares.  Gives
// kCode + code.
template <int TOP>
__device__ __forceinline__ float2 encode(const Mul& mul, float2 x, float2 inv, uint32_t h0, uint32_t h1) {
  constexpr float kMost = (float)(TOP * TOP);
  float2 y = mul(x, inv);
  y = make_float2(fminf(fabsf(y.x), kMost), fminf(fabsf(y.y), kMost));
  // A root that is never above the true one; its floor is then at most one too low.
  float2 r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(y.x));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(y.y));
  constexpr float kLess = 1.f - 0x1p-21f;
  float2 low = add2(make_float2(__fmaf_rd(r.x, kLess, k2p23), __fmaf_rd(r.y, kLess, k2p23)), two(-k2p23));
  const float2 next = add2(low, two(1.f)), square = mul(next, next);
  low = make_float2(square.x <= y.x ? next.x : low.x, square.y <= y.y ? next.y : low.y);
  const float2 share = make_float2(__fmaf_rn(-low.x, low.x, y.x), __fmaf_rn(-low.y, low.y, y.y));
  // u * (2 low + 1), rounded once: the step is scaled by 2^-16.
  const float2 step = fma2(low, two(0x1p-15f), two(0x1p-16f));
  // bits: the lower (255) or upper half of the hash, as a float.
  constexpr uint32_t kSel = TOP == 127 ? 0x7632 : 0x7610;
  const float2 u = add2(make_float2(__uint_as_float(__byte_perm(h0, 0x4b000000u, kSel)),
                                          __uint_as_float(__byte_perm(h1, 0x4b000000u, kSel))), two(-k2p23));
  const float2 edge = mul(u, step);
  const float2 code = add2(low, make_float2(share.x > edge.x ? kCode + 1.f : kCode, share.y > edge.y ? kCode + 1.f : kCode));
  return code;
}

// A root and a quotient in some 46 bits: Newton's step on fp32's, whose residual alone
// is taken in fp64.  (The fp64 functions take microseconds here.)
__device__ __forceinline__ double root(double t) {
  if (!(t > 1e-30 && t < 1e30)) return sqrt(t);
  const float n = __fsqrt_rn((float)t);
  return (double)n + (double)__fdiv_rn((float)fma(-(double)n, (double)n, t), 2.f * n);
}
// min(1, a / b) for a, b > 0
__device__ __forceinline__ float clip_of(double a, double b) {
  if (a >= b) return 1.f;
  if (!(a > 1e-30 && b < 1e30)) return (float)(a / b);
  const float d = (float)b, q = __fdiv_rn((float)a, d);
  return (float)((double)q + (double)__fdiv_rn((float)fma(-(double)q, b, a), d));
}

// The clip factor from the blocks' sums, in a fixed order; false: the norm is not
// finite.  Every block adds them again, by one warp: some 600 numbers from L2, beside a
// launch that would do it once (4.7 us).  fp64 is slow here: all warps' sums cost a
// small step 11 us.
__device__ __forceinline__ bool clip_factor(const Hyper& h, float& clip) {
  __shared__ float s_clip;
  if (threadIdx.x < 32) {
    double t = 0.0;
    constexpr int U = 20;
    for (int k = threadIdx.x; k < h.parts; k += U * 32) {
      double v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = k + u * 32 < h.parts ? h.part[k + u * 32] : 0.0;
#pragma unroll
      for (int n = U; n > 1; n = (n + 1) / 2)      // as a tree: few additions one after the other
#pragma unroll
        for (int u = 0; u < n / 2; ++u) v[u] += v[u + (n + 1) / 2];
      t += v[0];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0) {
      t = root(t);
      const float n = (float)t;
      if (h.norm && blockIdx.x == 0) *h.norm = n;
      s_clip = n <= 3.4028235e38f ? clip_of(h.max_norm, t + 1e-6) : -1.f;
    }
  }
  __syncthreads();
  clip = s_clip;
  return clip >= 0.f;
}

template <int N, bool EIGHT>
__global__ void __launch_bounds__(kWarps * 32) k_adamw(const __grid_constant__ List<N> list, const Hyper h) {
  const int lane = threadIdx.x % 32;
  const Mul mul(h.minus_zero);
  float clip = 1.f;
  wait_for_previous();
  if (h.part && !clip_factor(h, clip)) return;
  const Desc& d = list.d[find(list, h.count, blockIdx.x)];
  const int64_t first = (int64_t)(blockIdx.x - d.first) * h.units;
  for (int u = threadIdx.x / 32; u < h.units; u += kWarps) {
    const int64_t unit = first + u, at = unit * kUnit;
    if (at >= d.n) return;
    const int left = (int)min((int64_t)kUnit, d.n - at);
    const bool vec = d.vec && left == kUnit;
    float p[8], g[8], m[8], v[8];
    if (EIGHT && vec && at + (kWarps + 1) * kUnit <= d.n) {
      const int64_t next = at + kWarps * kUnit;
      fetch_line(d.param + next + lane * 8);
      fetch_line(static_cast<const char*>(d.grad) + (next + lane * 8) * (d.grad_type == LOPT_F32 ? 4 : 2));
      if (lane < 8) fetch_line(static_cast<const uint8_t*>(d.m) + next + lane * 32);
      else if (lane < 16) fetch_line(static_cast<const uint8_t*>(d.v) + next + lane * 32 - 256);
    }
    load_grad(d, at, vec, lane, left, g);
    load8(d.param + at, vec, lane, left, [&](int k, float x) { p[k] = x; });
    if (EIGHT) {
      const float ms = d.m_scale[unit], vs = d.v_scale[unit];
      uint32_t qm[2], qv[2];
      load_codes(static_cast<const uint8_t*>(d.m) + at, vec, lane, left, qm);
      load_codes(static_cast<const uint8_t*>(d.v) + at, vec, lane, left, qv);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        // int8 + 128 is a byte's value with the sign bit turned over.
        const uint32_t wm = qm[k / 4] ^ 0x80808080u, wv = qv[k / 4];
        const float2 a = k % 4 == 0 ? bytes<0>(wm, 128.f) : bytes<1>(wm, 128.f);
        const float2 b = k % 4 == 0 ? bytes<0>(wv, 0.f) : bytes<1>(wv, 0.f);
        const float2 x = mul(mul(a, make_float2(fabsf(a.x), fabsf(a.y))), two(ms));
        const float2 r = mul(mul(b, b), two(vs)), r2 = mul(r, r);
        m[k] = x.x, m[k + 1] = x.y, v[k] = r2.x, v[k + 1] = r2.y;
      }
    } else {
      load8(static_cast<const float*>(d.m) + at, vec, lane, left, [&](int k, float x) { m[k] = x; });
      load8(static_cast<const float*>(d.v) + at, vec, lane, left, [&](int k, float x) { v[k] = x; });
    }
    const float keep = d.decay ? h.keep : 1.f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 x = mul(make_float2(g[k], g[k + 1]), two(clip));
      const float2 mk = add2(mul(make_float2(m[k], m[k + 1]), two(h.b1)), mul(x, two(h.nb1)));
      const float2 vk = add2(mul(make_float2(v[k], v[k + 1]), two(h.b2)), mul(mul(x, two(h.nb2)), x));
      const float2 root = make_float2(__fsqrt_rn(vk.x), __fsqrt_rn(vk.y));
      const float2 under = add2(mul(root, two(h.c2)), two(h.eps));
      const float2 step = make_float2(__fdiv_rn(mk.x, under.x), __fdiv_rn(mk.y, under.y));
      // p * keep - c1 * step; the difference of two rounded products
      const float2 pk = add2(mul(make_float2(p[k], p[k + 1]), two(keep)), mul(step, two(-h.c1)));
      p[k] = pk.x, p[k + 1] = pk.y;
      m[k] = mk.x, m[k + 1] = mk.y;
      v[k] = EIGHT ? root.x : vk.x, v[k + 1] = EIGHT ? root.y : vk.y;
    }
    store8(d.param + at, vec, lane, left, [&](int k) { return p[k]; });
    if (d.copy) {
      if (d.copy_type == LOPT_F16)
        store8(static_cast<__half*>(d.copy) + at, vec, lane, left, [&](int k) { return __float2half_rn(p[k]); });
      else
        store8(static_cast<__nv_bfloat16*>(d.copy) + at, vec, lane, left, [&](int k) { return __float2bfloat16_rn(p[k]); });
    }
    if (EIGHT) {
      constexpr float kM = 127.f * 127.f, kV = 255.f * 255.f;
      const float am = largest(m), av = largest(v);
      // NaN passes both tests and makes the block's scale NaN.
      const float im = am <= 1e-30f ? 0.f : __fdiv_rn(kM, am), iv = av <= 1e-30f ? 0.f : __fdiv_rn(kV, av);
      const uint32_t key = d.key ^ ((uint32_t)(at >> 32) * 0x85ebca6bu);
      uint32_t qm[2], qv[2];
      float2 fm[4], fv[4];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint32_t h0 = mix((uint32_t)(at + place(vec, lane, k)) ^ key), h1 = mix((uint32_t)(at + place(vec, lane, k + 1)) ^ key);
        const float2 q = encode<127>(mul, make_float2(m[k], m[k + 1]), two(im), h0, h1);
        fm[k / 2] = make_float2(m[k] < 0.f ? 2.f * kCode - q.x : q.x, m[k + 1] < 0.f ? 2.f * kCode - q.y : q.y);
        fv[k / 2] = encode<255>(mul, make_float2(v[k], v[k + 1]), two(iv), h0, h1);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        qm[j] = low_bytes(fm[2 * j], fm[2 * j + 1]);
        qv[j] = low_bytes(fv[2 * j], fv[2 * j + 1]);
      }
      store_codes(static_cast<uint8_t*>(d.m) + at, vec, lane, left, qm);
      store_codes(static_cast<uint8_t*>(d.v) + at, vec, lane, left, qv);
      if (lane == 0) {
        d.m_scale[unit] = __fmul_rn(am, (float)(1.0 / (127 * 127)));
        d.v_scale[unit] = __fmul_rn(av, (float)(1.0 / (255 * 255)));
      }
    } else {
      store8(static_cast<float*>(d.m) + at, vec, lane, left, [&](int k) { return m[k]; });
      store8(static_cast<float*>(d.v) + at, vec, lane, left, [&](int k) { return v[k]; });
    }
  }
}

// ---- the gradients' norm ----------------------------------------------------------
constexpr int kNormBlocks = 608;       // most blocks of a launch
constexpr int kNormLaunches = 16;      // that have partial sums of their own; more add to theirs in turn
constexpr int kMaxPartials = kNormLaunches * kNormBlocks;

// The sum of squares in about 48 bits: s the running sum, c the roundings of
// the squares and of the sums (two-sum and fused multiply-add residuals), two sums
// side by side.
struct Sum {
  float2 s = {0.f, 0.f}, c = {0.f, 0.f};
  uint32_t any = 0;
  __device__ __forceinline__ void add(const Mul& mul, float x, float y) {
    const float2 v = make_float2(x, y), minus = make_float2(-1.f, -1.f);
    const float2 p = mul(v, v), e = fma2(v, v, mul(p, minus));
    const float2 t = add2(s, p), b = fma2(s, minus, t);
    const float2 lost = add2(fma2(fma2(b, minus, t), minus, s), fma2(b, minus, p));
    c = add2(c, add2(lost, e));
    s = t;
    any |= __float_as_uint(x) | __float_as_uint(y);
  }
  __device__ __forceinline__ double total() const { return ((double)s.x + (double)s.y) + ((double)c.x + (double)c.y); }
  // Squares that overflow or vanish in fp32: the caller adds again in fp64.
  __device__ __forceinline__ bool lost() const {
    return !(s.x + s.y < 1e38f) || (s.x + s.y < 1e-20f && (any << 1));
  }
};

// Four blocks an SM: 64 registers (1.31G float32 gradients 0.79 ms; 0.95 with 80, three blocks).
template <int N>
__global__ void __launch_bounds__(kWarps * 32, 4)
    k_adamw_norm(const __grid_constant__ List<N> list, int count, int units, int chunks, float minus_zero, double* part, bool add) {
  const Mul mul(minus_zero);
  __shared__ double red[kWarps];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  double total = 0.0;
  for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const Desc& d = list.d[find(list, count, chunk)];
    const int64_t first = (int64_t)(chunk - d.first) * units;
    Sum sum;
    // Four units' loads side by side: 80 KB of an SM on their way.
    for (int u = w; u < units; u += 4 * kWarps) {
      float g[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t at = (first + u + q * kWarps) * kUnit;
        const int left = u + q * kWarps < units && at < d.n ? (int)min((int64_t)kUnit, d.n - at) : 0;
        if (left > 0) {
          load_grad(d, at, d.vec && left == kUnit, lane, left, g[q]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[q][k] = 0.f;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 8; k += 2) sum.add(mul, g[q][k], g[q][k + 1]);
    }
    if (!sum.lost()) {
      total += sum.total();
      continue;
    }
    for (int u = w; u < units; u += kWarps) {
      const int64_t at = (first + u) * kUnit;
      if (at >= d.n) break;
      const int left = (int)min((int64_t)kUnit, d.n - at);
      float g[8];
      load_grad(d, at, d.vec && left == kUnit, lane, left, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) total += (double)g[k] * (double)g[k];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) red[w] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kWarps; ++k) total += red[k];
    part[blockIdx.x] = add ? part[blockIdx.x] + total : total;
  }
}

// For a list without elements.
__global__ void k_adamw_no_norm(float* norm) {
  wait_for_previous();
  *norm = 0.f;
}

// ---- the moments as values ----------------------------------------------------------
struct Out {
  const void *m, *v;
  const float *m_scale, *v_scale;
  float *to_m, *to_v;
  int64_t n;
  int32_t first;
  uint8_t eight, vec;
};
template <int N> struct Outs {
  Out d[N];
};
constexpr int kOuts = 400;

__global__ void __launch_bounds__(kWarps * 32) k_adamw_moments(const __grid_constant__ Outs<kOuts> list, int count, int units) {
  const int lane = threadIdx.x % 32;
  const int chunk = blockIdx.x;
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.d[mid].first <= chunk) lo = mid; else hi = mid - 1;
  }
  const Out& d = list.d[lo];
  const int64_t first = (int64_t)(chunk - d.first) * units;
  for (int u = threadIdx.x / 32; u < units; u += kWarps) {
    const int64_t unit = first + u, at = unit * kUnit;
    if (at >= d.n) return;
    const int left = (int)min((int64_t)kUnit, d.n - at);
    const bool vec = d.vec && left == kUnit;
    float m[8], v[8];
    if (d.eight) {
      const float ms = d.m_scale[unit], vs = d.v_scale[unit];
      load8(static_cast<const int8_t*>(d.m) + at, vec, lane, left, [&](int k, int8_t x) { m[k] = decode(x, ms); });
      load8(static_cast<const uint8_t*>(d.v) + at, vec, lane, left, [&](int k, uint8_t x) {
        const float r = decode(x, vs);
        v[k] = __fmul_rn(r, r);
      });
    } else {
      load8(static_cast<const float*>(d.m) + at, vec, lane, left, [&](int k, float x) { m[k] = x; });
      load8(static_cast<const float*>(d.v) + at, vec, lane, left, [&](int k, float x) { v[k] = x; });
    }
    store8(d.to_m + at, vec, lane, left, [&](int k) { return m[k]; });
    store8(d.to_v + at, vec, lane, left, [&](int k) { return v[k]; });
  }
}

// ---- host ------------------------------------------------------------------------
constexpr int64_t kMaxElements = (int64_t)1 << 40;

struct Range {
  uintptr_t lo, hi;
  bool in;      // read only
};

// A tensor's arrays.
int ranges(const lopt_adamw_tensor& t, Range (&r)[7], int* count) {
  const int gs = type_size(t.grad_type), cs = t.copy_type == LOPT_F32 ? 0 : type_size(t.copy_type);
  if (!gs || (t.moments != 32 && t.moments != 8) || (t.decay != 0 && t.decay != 1)) return LOPT_E_ARG;
  if (t.copy && !cs) return LOPT_E_ARG;
  if (t.n < 0 || t.n > kMaxElements) return LOPT_E_SHAPE;
  *count = 0;
  if (t.n == 0) return LOPT_OK;
  const bool eight = t.moments == 8;
  if (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale))) return LOPT_E_ARG;
  const int64_t blocks = (t.n + kUnit - 1) / kUnit;
  const struct { const void* p; int64_t n; int size; } a[7] = {
      {t.param, t.n, 4}, {t.grad, t.n, gs}, {t.m, t.n, eight ? 1 : 4}, {t.v, t.n, eight ? 1 : 4},
      {t.copy, t.n, cs}, {eight ? t.m_scale : nullptr, blocks, 4}, {eight ? t.v_scale : nullptr, blocks, 4}};
  for (int k = 0; k < 7; ++k) {
    if (!a[k].p) continue;
    if ((uintptr_t)a[k].p % a[k].size) return LOPT_E_ALIGN;
    r[(*count)++] = Range{(uintptr_t)a[k].p, (uintptr_t)a[k].p + (uintptr_t)(a[k].n * a[k].size), k == 1};
  }
  return LOPT_OK;
}

bool all_aligned(const lopt_adamw_tensor& t) {
  const uintptr_t es = t.moments == 8 ? 4 : 16;
  return (uintptr_t)t.param % 16 == 0 && (uintptr_t)t.grad % (t.grad_type == LOPT_F32 ? 16 : 8) == 0 &&
         (uintptr_t)t.m % es == 0 && (uintptr_t)t.v % es == 0 && (uintptr_t)t.copy % 8 == 0;
}

// Warp units of a chunk: lists that would not fill the GPU otherwise get
// small chunks.
int chunk_units(int64_t units, int sms) { return units > (int64_t)sms * 8 * 16 * kWarps ? 16 * kWarps : kWarps; }

template <int N, bool EIGHT>
cudaError_t launch_step(const List<N>& list, const Hyper& h, int chunks, cudaStream_t s) {
  return launch(k_adamw<N, EIGHT>, dim3((unsigned)chunks), dim3(kWarps * 32), 0, s, true, 1, list, h);
}

struct Part {     // tensors of one launch
  std::vector<int> index;
  int chunks = 0;
};

// The list in launches of at most kLarge tensors and 2^30 chunks.
std::vector<Part> parts(const lopt_adamw_tensor* t, int n, int bits, int units) {
  std::vector<Part> out;
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0 || (bits && t[i].moments != bits)) continue;
    const int64_t chunk = (int64_t)units * kUnit;
    const int chunks = (int)((t[i].n + chunk - 1) / chunk);
    if (out.empty() || out.back().index.size() == (size_t)kLarge || (int64_t)out.back().chunks + chunks > (1 << 30))
      out.emplace_back();
    out.back().index.push_back(i);
    out.back().chunks += chunks;
  }
  return out;
}

template <int N>
void fill(List<N>& list, const lopt_adamw_tensor* t, const Part& part, int units, uint32_t seed) {
  int at = 0;
  for (size_t k = 0; k < part.index.size(); ++k) {
    const lopt_adamw_tensor& x = t[part.index[k]];
    Desc& d = list.d[k];
    d = Desc{x.param, x.grad, x.m, x.v, x.m_scale, x.v_scale, x.copy, x.n,
             mix(seed ^ ((uint32_t)(part.index[k] + 1) * 0x9e3779b9u)), at, (uint8_t)x.grad_type, (uint8_t)x.copy_type,
             (uint8_t)x.decay, (uint8_t)all_aligned(x), 0};
    const int64_t chunk = (int64_t)units * kUnit;
    at += (int)((x.n + chunk - 1) / chunk);
  }
}

// The list, as large as it has to be, to `f`.
template <typename F>
cudaError_t with_list(const lopt_adamw_tensor* t, const Part& part, int units, uint32_t seed, F f) {
  if (part.index.size() <= (size_t)kSmall) {
    List<kSmall> list{};
    fill(list, t, part, units, seed);
    return f(list);
  }
  List<kLarge> list{};
  fill(list, t, part, units, seed);
  return f(list);
}

int check_each(const lopt_adamw_tensor* t, int32_t n, std::vector<Range>* all) {
  if (n < 0 || (n && !t)) return LOPT_E_ARG;
  for (int32_t i = 0; i < n; ++i) {
    Range r[7];
    int count = 0;
    const int rc = ranges(t[i], r, &count);
    if (rc) return rc;
    for (int a = 0; a < count; ++a)
      for (int b = a + 1; b < count; ++b)
        if (r[a].lo < r[b].hi && r[b].lo < r[a].hi) return LOPT_E_ALIAS;
    if (all) all->insert(all->end(), r, r + count);
  }
  return LOPT_OK;
}

int step(const lopt_adamw_tensor* tensors, int32_t n, int64_t t, double lr, double beta1, double beta2, double eps,
         double weight_decay, double max_norm, uint32_t seed, float* norm, void* workspace, int64_t workspace_bytes,
         cudaStream_t s) {
  if (t < 1 || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || !std::isfinite(eps) ||
      !std::isfinite(lr) || !std::isfinite(weight_decay) || !(max_norm >= 0))
    return LOPT_E_ARG;
  int rc = check_each(tensors, n, nullptr);
  if (rc) return rc;
  const bool clipped = max_norm > 0;
  double* part = static_cast<double*>(workspace);
  if (clipped) {
    int64_t need = 0;
    lopt_adamw_workspace(&need);
    if (!norm || !workspace || workspace_bytes < need) return LOPT_E_ARG;
    if ((uintptr_t)workspace % 256 || (uintptr_t)norm % 4) return LOPT_E_ALIGN;
    const uintptr_t lo = (uintptr_t)workspace, hi = lo + (uintptr_t)need, nl = (uintptr_t)norm, nh = nl + 4;
    if (nl < hi && lo < nh) return LOPT_E_ALIAS;
    for (int32_t i = 0; i < n; ++i) {
      Range r[7];
      int count = 0;
      ranges(tensors[i], r, &count);
      for (int k = 0; k < count; ++k)
        if ((r[k].lo < hi && lo < r[k].hi) || (r[k].lo < nh && nl < r[k].hi)) return LOPT_E_ALIAS;
    }
  }
  const int sms = sm_count();
  int64_t units = 0;
  for (int32_t i = 0; i < n; ++i) units += (tensors[i].n + kUnit - 1) / kUnit;
  const int per = chunk_units(units, sms);
  Hyper h;
  h.b1 = (float)beta1, h.nb1 = (float)(1.0 - beta1), h.b2 = (float)beta2, h.nb2 = (float)(1.0 - beta2);
  h.c1 = (float)(lr / (1.0 - std::pow(beta1, (double)t)));
  h.c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)t)));
  h.eps = (float)eps, h.keep = (float)(1.0 - lr * weight_decay), h.part = nullptr, h.parts = 0, h.max_norm = max_norm, h.norm = nullptr, h.units = per, h.minus_zero = -0.f;
  cudaError_t e = cudaSuccess;
  if (clipped) {
    int count = 0;
    const std::vector<Part> ps = parts(tensors, n, 0, per);
    int first[kNormLaunches], size[kNormLaunches];
    for (size_t i = 0; i < ps.size(); ++i) {
      const Part& p = ps[i];
      const int slot = (int)(i % kNormLaunches);
      const bool add = i >= kNormLaunches;
      const int blocks = std::min(p.chunks, add ? size[slot] : kNormBlocks);
      if (!add) first[slot] = count, size[slot] = blocks, count += blocks;
      e = with_list(tensors, p, per, seed, [&](const auto& list) {
        constexpr int N = sizeof(list.d) / sizeof(list.d[0]);
        return launch(k_adamw_norm<N>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, true, 1, list,
                      (int)p.index.size(), per, p.chunks, -0.f, part + first[slot], add);
      });
      if (e != cudaSuccess) return done(e);
    }
    if (count == 0) return done(launch(k_adamw_no_norm, dim3(1), dim3(1), 0, s, true, 1, norm));
    h.part = part, h.parts = count, h.norm = norm;
  }
  for (int bits : {32, 8}) {
    for (const Part& p : parts(tensors, n, bits, per)) {
      h.count = (int)p.index.size();
      e = with_list(tensors, p, per, seed, [&](const auto& list) {
        return bits == 8 ? launch_step<sizeof(list.d) / sizeof(list.d[0]), true>(list, h, p.chunks, s)
                         : launch_step<sizeof(list.d) / sizeof(list.d[0]), false>(list, h, p.chunks, s);
      });
      if (e != cudaSuccess) return done(e);
      h.norm = nullptr;      // one launch writes it
    }
  }
  return LOPT_OK;
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_adamw_check(const lopt_adamw_tensor* tensors, int32_t n) try {
  std::vector<Range> all;
  const int rc = check_each(tensors, n, &all);
  if (rc) return rc;
  // Arrays in order of their address: one that is written may not reach into
  // the next.  Gradients may share memory among themselves.
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end = 0, end_written = 0;
  for (const Range& r : all) {
    if (r.lo < (r.in ? end_written : end)) return LOPT_E_ALIAS;
    end = std::max(end, r.hi);
    if (!r.in) end_written = std::max(end_written, r.hi);
  }
  return LOPT_OK;
} catch (...) {
  return LOPT_E_OOM;
}

int lopt_adamw_workspace(int64_t* bytes) {
  if (!bytes) return LOPT_E_ARG;
  *bytes = kMaxPartials * 8;   // partial sums
  return LOPT_OK;
}

int lopt_adamw_step(const lopt_adamw_tensor* tensors, int32_t n, int64_t t, double lr, double beta1, double beta2,
                    double eps, double weight_decay, double max_norm, uint32_t seed, float* norm, void* workspace,
                    int64_t workspace_bytes, void* stream) try {
  return step(tensors, n, t, lr, beta1, beta2, eps, weight_decay, max_norm, seed, norm, workspace, workspace_bytes,
              (cudaStream_t)stream);
} catch (...) {
  return LOPT_E_OOM;
}

int lopt_adamw_moments(const lopt_adamw_tensor* tensors, int32_t n, float* const* m, float* const* v, void* stream) try {
  std::vector<Range> all;
  int rc = check_each(tensors, n, &all);
  if (rc) return rc;
  if (n && (!m || !v)) return LOPT_E_ARG;
  for (Range& r : all) r.in = true;
  int64_t units = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].n == 0) continue;
    for (float* p : {m[i], v[i]}) {
      if (!p) return LOPT_E_ARG;
      if ((uintptr_t)p % 4) return LOPT_E_ALIGN;
      all.push_back(Range{(uintptr_t)p, (uintptr_t)(p + tensors[i].n), false});
    }
    units += (tensors[i].n + kUnit - 1) / kUnit;
  }
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end = 0, end_written = 0;
  for (const Range& r : all) {
    if (r.lo < (r.in ? end_written : end)) return LOPT_E_ALIAS;
    end = std::max(end, r.hi);
    if (!r.in) end_written = std::max(end_written, r.hi);
  }
  const int per = chunk_units(units, sm_count());
  for (const Part& p : parts(tensors, n, 0, per)) {
    Outs<kOuts> list{};
    int at = 0;
    for (size_t k = 0; k < p.index.size(); ++k) {
      const int i = p.index[k];
      const lopt_adamw_tensor& x = tensors[i];
      const uintptr_t es = x.moments == 8 ? 4 : 16;
      const bool vec = (uintptr_t)x.m % es == 0 && (uintptr_t)x.v % es == 0 && (uintptr_t)m[i] % 16 == 0 && (uintptr_t)v[i] % 16 == 0;
      list.d[k] = Out{x.m, x.v, x.m_scale, x.v_scale, m[i], v[i], x.n, at, (uint8_t)(x.moments == 8), (uint8_t)vec};
      const int64_t chunk = (int64_t)per * kUnit;
      at += (int)((x.n + chunk - 1) / chunk);
    }
    const cudaError_t e = launch(k_adamw_moments, dim3((unsigned)p.chunks), dim3(kWarps * 32), 0, (cudaStream_t)stream,
                                 false, 1, list, (int)p.index.size(), per);
    if (e != cudaSuccess) return done(e);
  }
  return LOPT_OK;
} catch (...) {
  return LOPT_E_OOM;
}

}  // extern "C"
