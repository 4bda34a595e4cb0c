// Shared pieces of the training operators (embedding, layer norm,
// distillation): element types, vector loads and stores, block reductions,
// argument checks and launches.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "lopt_train.h"

namespace lopt {

int record_cuda_error(cudaError_t e);   // lopt_host.cu

namespace train {

// ---- element types -----------------------------------------------------------
inline int type_size(int type) { return type == LOPT_F32 ? 4 : (type == LOPT_F16 || type == LOPT_BF16) ? 2 : 0; }
inline int index_size(int type) { return type == LOPT_I32 ? 4 : type == LOPT_I64 ? 8 : 0; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC elements of T as one memory access of VEC * sizeof(T) bytes.
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

// All its elements to and from float, two at a time where they are 16-bit.
template <typename T, int VEC> __device__ __forceinline__ void to_floats(const Pack<T, VEC>& p, float (&f)[VEC]) {
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      float2 v;
      if constexpr (__is_same(T, __nv_bfloat16)) {
        v = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      } else {
        v = __half22float2(*reinterpret_cast<const __half2*>(w + k));
      }
      f[2 * k] = v.x;
      f[2 * k + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = to_f(p.v[e]);
  }
}
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> from_floats(const float (&f)[VEC]) {
  Pack<T, VEC> p;
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      if constexpr (__is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 h = __float22bfloat162_rn(make_float2(f[2 * k], f[2 * k + 1]));
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __float22half2_rn(make_float2(f[2 * k], f[2 * k + 1]));
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.v[e] = from_f<T>(f[e]);
  }
  return p;
}

// An element of a float-like array whose type is known at run time.
__device__ __forceinline__ float load_as_f(const void* p, int64_t i, int type) {
  if (type == LOPT_F32) return static_cast<const float*>(p)[i];
  if (type == LOPT_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int type) {
  return type == LOPT_I32 ? (int64_t) static_cast<const int32_t*>(p)[i] : static_cast<const int64_t*>(p)[i];
}

// Bits of the caller's status word.
constexpr int32_t kStatusIndex = 1;    // an index at or above its limit
constexpr int32_t kStatusGaveUp = 2;   // a bounded wait ran out: results are not valid

// ---- reductions ----------------------------------------------------------------
// Butterflies: every lane ends with the same bits, since a + b == b + a.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---- launches ------------------------------------------------------------------
// A kernel launched with `dependent` may be set up while the kernel before it
// on the stream still runs; it calls wait_for_previous() before it touches
// what that kernel writes.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool dependent,
                   int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Lets `kernel` have all the dynamic shared memory of a block on the current
// device.  The runtime calls cost more than a small launch can spare, so which
// (kernel, device) have it is remembered in a table without locks; two threads
// that both find it missing set the same value.
inline cudaError_t allow_smem(const void* kernel, size_t smem) {
  if (smem <= 40 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int kSlots = 1024;
  static std::atomic<uintptr_t> done[kSlots];
  const uintptr_t key = (uintptr_t)kernel * 64 + (uintptr_t)(dev & 63) + 1;
  size_t h = (key * 0x9e3779b97f4a7c15ull) >> 54;
  for (int n = 0; n < kSlots; ++n, h = (h + 1) & (kSlots - 1)) {
    const uintptr_t k = done[h].load(std::memory_order_acquire);
    if (k == key) return cudaSuccess;
    if (k == 0) break;
  }
  cudaFuncAttributes at;
  int most = 0;
  if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)at.sharedSizeBytes);
  if (e != cudaSuccess) return e;
  for (int n = 0; n < kSlots; ++n, h = (h + 1) & (kSlots - 1)) {
    uintptr_t k = 0;
    if (done[h].compare_exchange_strong(k, key) || k == key) break;
  }
  return cudaSuccess;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? LOPT_OK : record_cuda_error(e); }

// SMs of the current device.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
  return n;
}

// ---- argument checks -------------------------------------------------------------
// A matrix argument: rows x cols elements of `es` bytes, rows `stride` apart.
struct Span {
  const void* p;
  int64_t rows, cols, stride;
  int es;
  uintptr_t lo() const { return (uintptr_t)p; }
  uintptr_t hi() const { return lo() + (uintptr_t)(((rows - 1) * stride + cols) * es); }
  bool same_place(const Span& o) const { return p == o.p && stride == o.stride && es == o.es; }
};

// Rows and tokens are counted in int32 with room for a block's stride past the
// end; columns / 256 has to be a grid dimension (65,535).
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 65536;
constexpr int64_t kMaxCols = (int64_t)1 << 23;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

// A present (non-null) matrix with sound stride and alignment.
inline int check_matrix(const Span& s, bool output) {
  if (!s.p) return LOPT_E_ARG;
  if (s.lo() % s.es) return LOPT_E_ALIGN;
  if (s.stride < 0 || s.stride > kMaxStride) return LOPT_E_SHAPE;
  if (output && s.rows > 1 && s.stride < s.cols) return LOPT_E_SHAPE;
  return LOPT_OK;
}

// Whether two matrices share a byte.  Interleaved column blocks of one
// buffer (equal row strides) are told apart by their offset within a row;
// otherwise the address ranges decide.
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  const int64_t sa = a.stride * a.es, sb = b.stride * b.es;
  if (sa == sb && sa > 0) {
    const int64_t wa = a.cols * a.es, wb = b.cols * b.es;
    if (wa <= sa && wb <= sa) {
      int64_t d = (int64_t)(b.lo() - a.lo()) % sa;
      if (d < 0) d += sa;
      if (d >= wa && d + wb <= sa) return false;
    }
  }
  return true;
}

// lopt_embed_backward() into rows `grad_stride` apart (k_embedding.cu).
int embed_backward_to(const void* grad_out, int type, int64_t grad_out_stride, const void* index, int index_type, int64_t n,
                      int64_t rows, int64_t cols, float scale, int accumulate, float* grad, int64_t grad_stride, void* workspace,
                      int64_t workspace_bytes, int32_t* status, void* stream);

// Rows that start on `bytes` boundaries.
inline bool rows_aligned(const Span& s, int bytes) {
  return !s.p || (s.lo() % bytes == 0 && (s.rows <= 1 || (s.stride * s.es) % bytes == 0));
}

}  // namespace train
}  // namespace lopt
