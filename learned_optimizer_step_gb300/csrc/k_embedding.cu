// Embedding lookup with a scale, and the gradient of its table by sorted
// tokens (see lopt_train.h).
//
// Forward: out[i] = scale * table[index[i]], a gather bound by HBM bytes.
//
// Backward: grad[v] = scale * sum of grad_out[i] over the i with index v.
// Token ids of text repeat: a handful take a large share of all positions and
// most occur once or never.  So the positions are first sorted by id and the
// sorted list is cut into chunks of equal length, whatever the ids: no row of
// the table is a block's fate, and every sum runs in position order, so the
// result does not depend on timing.
//   1. k_embed_sort: each block owns some ids and reads the whole index list
//      (it stays in L2) to count and place its own: a stable counting sort
//      with no exchange between blocks.  It also writes the zero rows.
//   2. k_embed_sum: each block adds the rows of one chunk of the sorted list.
//      A run of equal ids inside the chunk goes straight to its row; a run
//      that crosses chunks leaves partial sums, which the last of its blocks
//      to arrive (a ticket, no spinning) adds in chunk order.
#include <algorithm>

#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

// ---- forward ---------------------------------------------------------------
struct EmbedFwd {
  const void *table, *index;
  void* out;
  int32_t* status;
  int64_t rows, cols, ts, n, os;
  int itype;
  float scale;
};

// blockDim.x threads across the columns, blockIdx.y column blocks; a thread
// takes U tokens, blockDim.y apart, with their loads side by side.
template <typename TI, typename TO, int VEC, int U>
__global__ void __launch_bounds__(256) k_embed_fwd(const EmbedFwd a) {
  const int64_t i0 = (int64_t)blockIdx.x * (blockDim.y * U) + threadIdx.y;
  const int64_t j = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (j >= a.cols) return;
  int64_t id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * (int)blockDim.y;
    id[u] = i < a.n ? load_index(a.index, i, a.itype) : -1;
  }
  Pack<TI, VEC> p[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (id[u] >= a.rows) {
      if (a.status && j == 0) atomicOr(a.status, kStatusIndex);
      id[u] = -1;
    }
    if (id[u] >= 0) p[u] = *reinterpret_cast<const Pack<TI, VEC>*>(static_cast<const TI*>(a.table) + id[u] * a.ts + j);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * (int)blockDim.y;
    if (i >= a.n) break;
    float v[VEC];
    to_floats(p[u], v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = id[u] >= 0 ? v[e] * a.scale : 0.f;
    *reinterpret_cast<Pack<TO, VEC>*>(static_cast<TO*>(a.out) + i * a.os + j) = from_floats<TO, VEC>(v);
  }
}

// ---- backward: sort ------------------------------------------------------------
// Block b of 2^log_blocks owns the ids v with v mod 2^log_blocks == b, at most
// 1024 of them: ids are given out by frequency in most vocabularies, and so
// the common ones (each of which keeps its block busy) fall to different
// blocks.  In the sorted list the blocks follow each other, in a block its
// ids ascend, and an id's positions ascend.
constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kMinLogBlocks = 7;        // 128 blocks
constexpr int kLogIds = 10;             // ids per block: at most 1024, 128 KB of counters
constexpr int kFound = 192;             // entries a warp keeps of its part of the list
constexpr int kZeroBytes = 8192;        // what one bulk store writes of a row of zeros

struct EmbedSort {
  const void* index;
  int n, rows, log_blocks, ids_per_block;
  int64_t n_counters;
  int32_t *order, *key, *offsets, *counters, *status;
  float* grad;
  int64_t cols;
  int zero_rows, zero_bulk;
};

template <typename IT>
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const EmbedSort a) {
  extern __shared__ __align__(16) int32_t sh[];
  const int K = a.ids_per_block;
  int32_t* zeros = sh;                                      // kZeroBytes
  uint32_t* found = reinterpret_cast<uint32_t*>(sh) + kZeroBytes / 4;   // [32 warps][kFound]: id's number | place << kLogIds
  int32_t* cnt = reinterpret_cast<int32_t*>(found) + kSortWarps * kFound;   // [32 warps][K]
  int32_t* tot = cnt + kSortWarps * K;                      // [K]
  __shared__ int32_t wsum[kSortWarps];
  __shared__ int32_t below_sum;
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const unsigned lt = (1u << lane) - 1;
  const int blk = blockIdx.x, mask = (1 << a.log_blocks) - 1;
  const IT* index = static_cast<const IT*>(a.index);
  let_next_start();
  for (int i = tid; i < kSortWarps * K; i += kSortThreads) cnt[i] = 0;
  for (int i = tid; i < kZeroBytes / 4; i += kSortThreads) zeros[i] = 0;
  if (tid == 0) below_sum = 0;
  for (int64_t i = (int64_t)blk * kSortThreads + tid; i < a.n_counters; i += (int64_t)gridDim.x * kSortThreads)
    a.counters[i] = 0;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the zeros, before bulk stores read them
  __syncthreads();
  // Warp w reads its contiguous part of the list and keeps what the block owns.
  const int per = ((a.n + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int beg = min(w * per, a.n), end = min(beg + per, a.n);
  int below = 0, mine_n = 0;
  bool bad = false;
  constexpr int U = 8;
  for (int i0 = beg; i0 < end; i0 += 32 * U) {
    IT id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 32 + lane;
      id[u] = i < end ? index[i] : (IT)-1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool real = id[u] >= 0 && id[u] < a.rows;
      bad |= id[u] >= a.rows;
      const int b = (int)id[u] & mask;
      below += real && b < blk;
      const bool mine = real && b == blk;
      const unsigned who = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int at = mine_n + __popc(who & lt);
        if (at < kFound) found[w * kFound + at] = (uint32_t)((int)id[u] >> a.log_blocks) | (uint32_t)(i0 - beg + u * 32 + lane) << kLogIds;
      }
      mine_n += __popc(who);
    }
  }
  __syncwarp();
  // In list order, 32 at a time: f(number of the id in the block or -1, its
  // place in the warp's part).  From what the warp kept, or, where that was
  // not all, from the list again.
  const bool kept = mine_n <= kFound && per <= 1 << (32 - kLogIds);
  auto each = [&](auto f) {
    if (kept) {
      for (int c = 0; c < mine_n; c += 32) {
        const uint32_t x = c + lane < mine_n ? found[w * kFound + c + lane] : 0;
        f(c + lane < mine_n ? (int)(x & ((1 << kLogIds) - 1)) : -1, (int)(x >> kLogIds));
      }
    } else {
      for (int i0 = beg; i0 < end; i0 += 32 * U) {
        IT id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * 32 + lane;
          id[u] = i < end ? index[i] : (IT)-1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool mine = id[u] >= 0 && id[u] < a.rows && ((int)id[u] & mask) == blk;
          if (__any_sync(0xffffffffu, mine)) f(mine ? (int)id[u] >> a.log_blocks : -1, i0 - beg + u * 32 + lane);
        }
      }
    }
  };
  each([&](int k, int) {
    const unsigned peers = __match_any_sync(0xffffffffu, k);
    if (k >= 0 && lane == __ffs(peers) - 1) cnt[w * K + k] += __popc(peers);
    __syncwarp();
  });
  if (bad && blk == 0 && a.status) atomicOr(a.status, kStatusIndex);
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0 && below) atomicAdd(&below_sum, below);   // integers: any order gives the same
  __syncthreads();
  // Per id: the warps' counts become starts, then the ids' totals a scan.
  int mine = 0;
  if (tid < K) {
    for (int k = 0; k < kSortWarps; ++k) {
      const int c = cnt[k * K + tid];
      cnt[k * K + tid] = mine;
      mine += c;
    }
    tot[tid] = mine;
  }
  int incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) wsum[w] = incl;
  __syncthreads();
  if (w == 0) {
    int t = wsum[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    wsum[lane] = t;
  }
  // Rows no token has, while the positions are placed: bulk stores of zeros
  // where rows are 16-byte aligned.
  if (a.zero_rows) {
    if (a.zero_bulk) {
      const int64_t bytes = a.cols * 4;
      for (int k = tid; k < K; k += kSortThreads) {
        const int v = k << a.log_blocks | blk;
        if (v >= a.rows || tot[k]) continue;
        char* g = reinterpret_cast<char*>(a.grad + (int64_t)v * a.cols);
        for (int64_t o = 0; o < bytes; o += kZeroBytes) {
          const uint32_t size = (uint32_t)min((int64_t)kZeroBytes, bytes - o);
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                       :: "l"(g + o), "r"((uint32_t)__cvta_generic_to_shared(zeros)), "r"(size) : "memory");
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    } else {
      for (int k = w; k < K; k += kSortWarps) {
        const int v = k << a.log_blocks | blk;
        if (v >= a.rows || tot[k]) continue;
        float* g = a.grad + (int64_t)v * a.cols;
        for (int64_t j = lane; j < a.cols; j += 32) g[j] = 0.f;
      }
    }
  }
  __syncthreads();
  const int start = below_sum + (w ? wsum[w - 1] : 0) + incl - mine;
  if (tid < K) {
    a.offsets[blk * K + tid] = start;
    if (blk == mask && tid == K - 1) a.offsets[blk * K + K] = start + mine;
    for (int k = 0; k < kSortWarps; ++k) cnt[k * K + tid] += start;
  }
  __syncthreads();
  each([&](int k, int place) {
    const unsigned peers = __match_any_sync(0xffffffffu, k);
    if (k >= 0) {
      const int at = cnt[w * K + k] + __popc(peers & lt);
      a.order[at] = beg + place;
      a.key[at] = k << a.log_blocks | blk;
    }
    __syncwarp();
    if (k >= 0 && lane == __ffs(peers) - 1) cnt[w * K + k] += __popc(peers);
    __syncwarp();
  });
  if (a.zero_rows && a.zero_bulk) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the zeros stay until read
}

// ---- backward: sums ----------------------------------------------------------------
constexpr int kMaxChunk = 16;

struct EmbedSum {
  const void* grad_out;
  const int32_t *order, *key, *offsets;
  int32_t* counters;       // [chunks][gridDim.y]: arrivals of the run that starts in the chunk
  float* part;             // [chunks][2][cols]: sums of a run entering / leaving the chunk
  float* grad;
  int64_t gs, cols;
  int log_blocks, ids_per_block, last_offset, chunk, accumulate;
  float scale;
};

template <int VEC>
__device__ __forceinline__ void store_sums(float* p, const float v[VEC]) {
  constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
  for (int k = 0; k < VEC; k += V4) {
    Pack<float, V4> q;
#pragma unroll
    for (int e = 0; e < V4; ++e) q.v[e] = v[k + e];
    *reinterpret_cast<Pack<float, V4>*>(p + k) = q;
  }
}
template <int VEC>
__device__ __forceinline__ void add_sums(const float* p, float v[VEC]) {   // written by other blocks: from L2
  if (VEC == 1) {
    v[0] += __ldcg(p);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(p + k));
      v[k] += q.x;
      v[k + 1] += q.y;
      v[k + 2] += q.z;
      v[k + 3] += q.w;
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256, 4) k_embed_sum(const EmbedSum a) {
  __shared__ int32_t ord[kMaxChunk], key[kMaxChunk + 2];   // key[0]: before the chunk, key[len + 1]: after it
  __shared__ int32_t last_flag;
  const int64_t j = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  const bool live = j < a.cols;
  wait_for_previous();
  const int total = a.offsets[a.last_offset];
  const int base = blockIdx.x * a.chunk;
  if (base >= total) return;
  const int len = min(a.chunk, total - base);
  for (int i = threadIdx.x; i < len + 2; i += blockDim.x) {
    const int at = base + i - 1;
    key[i] = at >= 0 && at < total ? a.key[at] : -1;
    if (i >= 1 && i <= len) ord[i - 1] = a.order[at];
  }
  __syncthreads();
  const bool head_open = key[0] == key[1], tail_open = key[len + 1] == key[len];
  const T* src = static_cast<const T*>(a.grad_out) + j;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  int run_start = 0;   // first entry of the current run in this chunk
  constexpr int U = 8;
  for (int i0 = 0; i0 < len; i0 += U) {
    Pack<T, VEC> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < len && live) p[u] = *reinterpret_cast<const Pack<T, VEC>*>(src + (int64_t)ord[i0 + u] * a.gs);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= len) break;
      float v[VEC];
      to_floats(p[u], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      if (i + 1 < len && key[i + 2] == key[i + 1]) continue;   // the run goes on
      if (live) {
        const bool from_before = run_start == 0 && head_open, goes_on = i + 1 == len && tail_open;
        if (from_before || goes_on) {
          store_sums<VEC>(a.part + ((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * a.cols + j, acc);
        } else {
          float* g = a.grad + (int64_t)key[i + 1] * a.cols + j;
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] *= a.scale;
          if (a.accumulate) add_sums<VEC>(g, acc);
          store_sums<VEC>(g, acc);
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      run_start = i + 1;
    }
  }
  // Runs that cross the chunk's ends: the one from before, then the one that
  // goes on (which may be the same).
  for (int side = 0; side < 2; ++side) {
    if (side == 0 ? !head_open : !tail_open) continue;
    const int v = side == 0 ? key[1] : key[len];
    const int at = (v & ((1 << a.log_blocks) - 1)) * a.ids_per_block + (v >> a.log_blocks);
    const int s0 = a.offsets[at], s1 = a.offsets[at + 1];
    const int first = s0 / a.chunk, last = (s1 - 1) / a.chunk;
    if (side == 1 && head_open && first < (int)blockIdx.x) continue;   // one run through the whole chunk: counted
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
      last_flag = atomicAdd(a.counters + (int64_t)first * gridDim.y + blockIdx.y, 1) == last - first;
    __syncthreads();
    if (!last_flag) continue;
    __threadfence();
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    add_sums<VEC>(a.part + ((int64_t)first * 2 + 1) * a.cols + j, acc);
#pragma unroll 8
    for (int c = first + 1; c <= last; ++c) add_sums<VEC>(a.part + (int64_t)c * 2 * a.cols + j, acc);
    float* g = a.grad + (int64_t)v * a.cols + j;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] *= a.scale;
    if (a.accumulate) add_sums<VEC>(g, acc);
    store_sums<VEC>(g, acc);
  }
}

// ---- host --------------------------------------------------------------------------
struct Plan {
  int chunk, chunks, log_blocks, ids_per_block;
  int col_blocks;   // upper bound, for the counters
  int64_t o_order, o_key, o_offsets, o_counters, o_part, bytes;
};

int64_t up(int64_t x) { return (x + 255) / 256 * 256; }

// The layout of the workspace; a function of the sizes alone.
Plan plan(int64_t n, int64_t rows, int64_t cols) {
  Plan p;
  p.chunk = n >= 16384 ? 16 : 8;
  p.chunks = (int)std::max<int64_t>((n + p.chunk - 1) / p.chunk, 1);
  p.log_blocks = kMinLogBlocks;
  while (rows > (int64_t)1 << (p.log_blocks + kLogIds)) ++p.log_blocks;
  p.ids_per_block = (int)((rows + ((int64_t)1 << p.log_blocks) - 1) >> p.log_blocks);
  p.col_blocks = (int)((cols + 255) / 256);
  p.o_order = 0;
  p.o_key = p.o_order + up(n * 4);
  p.o_offsets = p.o_key + up(n * 4);
  p.o_counters = p.o_offsets + up((((int64_t)p.ids_per_block << p.log_blocks) + 1) * 4);
  p.o_part = p.o_counters + up((int64_t)p.chunks * p.col_blocks * 4);
  p.bytes = p.o_part + up((int64_t)p.chunks * 2 * cols * 4);
  return p;
}

template <typename TI, typename TO>
cudaError_t fwd_as(const EmbedFwd& a, int vec, int sms, cudaStream_t s) {
  const int64_t nv = (a.cols + vec - 1) / vec;
  const int tx = (int)std::min<int64_t>((nv + 31) / 32 * 32, 256);
  const int ty = std::max(1, 256 / tx);
  const unsigned gy = (unsigned)((nv + tx - 1) / tx);
  // Four tokens per thread once that still fills every SM's eight blocks.
  const bool many = a.n * gy >= (int64_t)sms * 8 * 4 * ty;
  const int64_t per = many ? 4 * ty : ty;
  const dim3 grid((unsigned)((a.n + per - 1) / per), gy), block(tx, ty);
  if (vec == 8)
    return many ? launch(k_embed_fwd<TI, TO, 8, 4>, grid, block, 0, s, false, 1, a) : launch(k_embed_fwd<TI, TO, 8, 1>, grid, block, 0, s, false, 1, a);
  if (vec == 4)
    return many ? launch(k_embed_fwd<TI, TO, 4, 4>, grid, block, 0, s, false, 1, a) : launch(k_embed_fwd<TI, TO, 4, 1>, grid, block, 0, s, false, 1, a);
  return many ? launch(k_embed_fwd<TI, TO, 1, 4>, grid, block, 0, s, false, 1, a) : launch(k_embed_fwd<TI, TO, 1, 1>, grid, block, 0, s, false, 1, a);
}

template <typename TI>
cudaError_t fwd_from(const EmbedFwd& a, int out_type, int vec, int sms, cudaStream_t s) {
  switch (out_type) {
    case LOPT_F32: return fwd_as<TI, float>(a, vec, sms, s);
    case LOPT_F16: return fwd_as<TI, __half>(a, vec, sms, s);
    default: return fwd_as<TI, __nv_bfloat16>(a, vec, sms, s);
  }
}

template <typename T, int VEC>
cudaError_t sum_as(const EmbedSum& a, int chunks, cudaStream_t s) {
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  const int tx = (int)std::min<int64_t>((nv + 31) / 32 * 32, 256);
  const dim3 grid((unsigned)chunks, (unsigned)((nv + tx - 1) / tx));
  return launch(k_embed_sum<T, VEC>, grid, dim3(tx), 0, s, true, 1, a);
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_embed_forward(const void* table, int table_type, int64_t rows, int64_t cols, int64_t table_stride,
                       const void* index, int index_type, int64_t n, float scale, void* out, int out_type,
                       int64_t out_stride, int32_t* status, void* stream) {
  const int ti = type_size(table_type), to = type_size(out_type), is = index_size(index_type);
  if (!ti || !to || !is) return LOPT_E_ARG;
  if (rows < 1 || cols < 1 || n < 0 || rows >= kMaxRows || cols > kMaxCols || n >= kMaxRows) return LOPT_E_SHAPE;
  if (n == 0) return LOPT_OK;
  const Span mt{table, rows, cols, table_stride, ti}, mo{out, n, cols, out_stride, to}, mi{index, 1, n, n, is};
  int rc;
  if ((rc = check_matrix(mt, false)) || (rc = check_matrix(mo, true)) || (rc = check_matrix(mi, false))) return rc;
  if (overlap(mo, mt) || overlap(mo, mi)) return LOPT_E_ALIAS;
  if (status && (uintptr_t)status % 4) return LOPT_E_ALIGN;
  // 8 elements per thread when either side is 16-bit, 4 between fp32 sides.
  int vec = ti == 4 && to == 4 ? 4 : 8;
  if (cols % vec || !rows_aligned(mt, std::min(vec * ti, 32)) || !rows_aligned(mo, std::min(vec * to, 32))) vec = 1;
  const EmbedFwd a{table, index, out, status, rows, cols, table_stride, n, out_stride, index_type, scale};
  cudaStream_t s = (cudaStream_t)stream;
  const int sms = sm_count();
  switch (table_type) {
    case LOPT_F32: return done(fwd_from<float>(a, out_type, vec, sms, s));
    case LOPT_F16: return done(fwd_from<__half>(a, out_type, vec, sms, s));
    default: return done(fwd_from<__nv_bfloat16>(a, out_type, vec, sms, s));
  }
}

int lopt_embed_workspace(int64_t n, int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes) return LOPT_E_ARG;
  if (rows < 1 || cols < 1 || n < 0 || rows >= kMaxRows || cols > kMaxCols || n >= kMaxRows)
    return LOPT_E_SHAPE;
  if (rows > (int64_t)1 << 30) return LOPT_E_SHAPE;   // the sort numbers them in int32, rounded up per block
  *bytes = plan(n, rows, cols).bytes;
  return LOPT_OK;
}

int lopt_embed_backward(const void* grad_out, int type, int64_t grad_out_stride, const void* index, int index_type,
                        int64_t n, int64_t rows, int64_t cols, float scale, int accumulate, float* grad,
                        void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  const int es = type_size(type), is = index_size(index_type);
  if (!es || !is || (accumulate != 0 && accumulate != 1)) return LOPT_E_ARG;
  int64_t need = 0;
  int rc = lopt_embed_workspace(n, rows, cols, &need);
  if (rc) return rc;
  const Span mg{grad, rows, cols, cols, 4};
  if ((rc = check_matrix(mg, true))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0) return accumulate ? LOPT_OK : done(cudaMemsetAsync(grad, 0, (size_t)rows * cols * 4, s));
  const Span md{grad_out, n, cols, grad_out_stride, es}, mi{index, 1, n, n, is}, ws{workspace, 1, need, need, 1};
  if ((rc = check_matrix(md, false)) || (rc = check_matrix(mi, false))) return rc;
  if (!workspace || workspace_bytes < need) return LOPT_E_ARG;
  if ((uintptr_t)workspace % 256 || (status && (uintptr_t)status % 4)) return LOPT_E_ALIGN;
  if (overlap(mg, md) || overlap(mg, mi) || overlap(mg, ws) || overlap(ws, md) || overlap(ws, mi)) return LOPT_E_ALIAS;
  const Plan p = plan(n, rows, cols);
  char* w = static_cast<char*>(workspace);
  const bool v4 = cols % 4 == 0 && (uintptr_t)grad % 16 == 0;
  EmbedSort a{};
  a.index = index;
  a.n = (int)n;
  a.rows = (int)rows;
  a.log_blocks = p.log_blocks;
  a.ids_per_block = p.ids_per_block;
  a.n_counters = (int64_t)p.chunks * p.col_blocks;
  a.order = (int32_t*)(w + p.o_order);
  a.key = (int32_t*)(w + p.o_key);
  a.offsets = (int32_t*)(w + p.o_offsets);
  a.counters = (int32_t*)(w + p.o_counters);
  a.status = status;
  a.grad = grad;
  a.cols = cols;
  a.zero_rows = !accumulate;
  a.zero_bulk = v4;
  const size_t smem = kZeroBytes + (size_t)kSortWarps * kFound * 4 + (size_t)(kSortWarps + 1) * p.ids_per_block * 4;
  auto* sort = index_type == LOPT_I32 ? &k_embed_sort<int32_t> : &k_embed_sort<int64_t>;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch(sort, dim3(1u << p.log_blocks), dim3(kSortThreads), smem, s, false, 1, a);
  if (e != cudaSuccess) return done(e);
  EmbedSum b{};
  b.grad_out = grad_out;
  b.order = a.order;
  b.key = a.key;
  b.offsets = a.offsets;
  b.counters = a.counters;
  b.part = (float*)(w + p.o_part);
  b.grad = grad;
  b.gs = grad_out_stride;
  b.cols = cols;
  b.log_blocks = p.log_blocks;
  b.ids_per_block = p.ids_per_block;
  b.last_offset = p.ids_per_block << p.log_blocks;
  b.chunk = p.chunk;
  b.accumulate = accumulate;
  b.scale = scale;
  const int vec = 16 / es;
  const bool wide = cols % vec == 0 && rows_aligned(md, 16) && v4;
  switch (type) {
    case LOPT_F32: return done(wide ? sum_as<float, 4>(b, p.chunks, s) : sum_as<float, 1>(b, p.chunks, s));
    case LOPT_F16: return done(wide ? sum_as<__half, 8>(b, p.chunks, s) : sum_as<__half, 1>(b, p.chunks, s));
    default:
      return done(wide ? sum_as<__nv_bfloat16, 8>(b, p.chunks, s) : sum_as<__nv_bfloat16, 1>(b, p.chunks, s));
  }
}

}  // extern "C"
