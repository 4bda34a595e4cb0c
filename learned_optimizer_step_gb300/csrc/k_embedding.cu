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
//   1. k_embed_sort: a stable counting sort.  Each block owns some ids; the
//      blocks of a cluster read the index list together, and every cluster all
//      of it (it stays in L2).
//   2. k_embed_sum: each block adds the rows of one chunk of the sorted list.
//      A run of equal ids inside the chunk goes straight to its row; a run
//      that crosses chunks leaves partial sums, which the last of its blocks
//      to arrive (a ticket, no spinning) adds in chunk order.  Blocks in
//      between write the rows without tokens, so that stores of zeros fill
//      the time in which the others wait for loads.
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
// takes U tokens, blockDim.y apart, and of each of their rows C accesses,
// blockDim.x apart, with all their loads side by side.  16,384 tokens of 2048,
// float32 to bfloat16: 22.9 us, 20 of them in the kernel (116 MB, 5.8 TB/s);
// 22.5 with two tokens per thread, 25.8 with eight.
template <typename TI, typename TO, int VEC, int U, int C>
__global__ void __launch_bounds__(256) k_embed_fwd(const EmbedFwd a) {
  const int64_t i0 = (int64_t)blockIdx.x * (blockDim.y * U) + threadIdx.y;
  const int64_t j = ((int64_t)blockIdx.y * (blockDim.x * C) + threadIdx.x) * VEC;
  const int step = blockDim.x * VEC;
  if (j >= a.cols) return;
  int64_t id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * (int)blockDim.y;
    id[u] = i < a.n ? load_index(a.index, i, a.itype) : -1;
  }
  Pack<TI, VEC> p[U][C];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (id[u] >= a.rows) {
      if (a.status && j == 0) atomicOr(a.status, kStatusIndex);
      id[u] = -1;
    }
    const TI* row = static_cast<const TI*>(a.table) + id[u] * a.ts + j;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (id[u] >= 0 && j + c * step < a.cols) p[u][c] = *reinterpret_cast<const Pack<TI, VEC>*>(row + c * step);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * (int)blockDim.y;
    if (i >= a.n) break;
    TO* to = static_cast<TO*>(a.out) + i * a.os + j;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (j + c * step >= a.cols) break;
      float v[VEC];
      to_floats(p[u][c], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = id[u] >= 0 ? v[e] * a.scale : 0.f;
      *reinterpret_cast<Pack<TO, VEC>*>(to + c * step) = from_floats<TO, VEC>(v);
    }
  }
}

// ---- backward: sort ------------------------------------------------------------
// Of 2^log_blocks blocks, the cluster v mod 2^(log_blocks - 3) and in it the
// block (v / 2^(log_blocks - 3)) mod 8 own the id v, at most 1024 ids a block:
// ids are given out by frequency in most vocabularies, and so the common ones
// (each of which keeps its block busy) fall to different clusters.  In the
// sorted list the blocks follow each other, in a block its ids ascend, and an
// id's positions ascend.
//
// The eight blocks of a cluster read the index list together, an eighth each,
// and keep what belongs to the cluster, in list order; each block then picks
// its own entries from the cluster's eight lists.  Bound by the chain of those
// steps, in cycles of the SM: 18,700 for 65,536 ids and 10,900 for 4,099 before
// the ids were loaded ahead, the counts added in one pass and the last cluster
// barrier split, which took 2 us off the whole gradient of 65,536 tokens (134
// to 132); when every block read the whole list it was 10 us longer.
constexpr int kMinLogBlocks = 7;        // 128 blocks
constexpr int kLogIds = 10;             // ids per block: at most 1024, 128 KB of counters
constexpr int kLogCluster = 3, kCluster = 1 << kLogCluster;
// Entries a warp keeps of its part of the list: all of a short list's, at most
// what shared memory has beside the counters.  What is not kept is read again
// (65,536 positions into 100,000 rows of 512, half of them one id: 192 us, 201
// with half as many); with half as many again an SM has no room for more than
// one block (131,072 text-like positions into 50,304 rows of 1024: 111 us, 113
// with half as many, 136 with half as many again).
inline int found_of(int warps, int n) {
  const int per_warp = (n + kCluster * warps - 1) / (kCluster * warps);
  return std::min((per_warp + 31) / 32 * 64, warps == 16 ? 1024 : 256);
}
constexpr int kLogPlace = 32 - kLogIds - kLogCluster;

struct EmbedSort {
  const void* index;
  int n, rows, log_blocks, ids_per_block, found;
  int64_t n_counters;
  int32_t *order, *key, *offsets, *counters, *status;
};

// The cluster an id belongs to (its low bits), or -1 where it is none.
__device__ __forceinline__ int cluster_of(int32_t id, unsigned rows, int mask) { return (unsigned)id < rows ? id & mask : -1; }
__device__ __forceinline__ int cluster_of(int64_t id, unsigned rows, int mask) {
  return (uint64_t)id >> 32 == 0 && (unsigned)id < rows ? (int)id & mask : -1;
}
// A shared-memory address of another block of the cluster.
template <typename P> __device__ __forceinline__ const P* of_block(const P* p, int rank) {
  uint64_t out;
  asm("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"((uint64_t)p), "r"(rank));
  return reinterpret_cast<const P*>(out);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename IT, int kSortWarps>
__global__ void __launch_bounds__(32 * kSortWarps) k_embed_sort(const EmbedSort a) {
  constexpr int kSortThreads = 32 * kSortWarps;
  const int keep = a.found;
  extern __shared__ int32_t sh[];
  const int K = a.ids_per_block;
  // An entry: block in the cluster | id's number in its block | place in this block's part.
  uint32_t* list = reinterpret_cast<uint32_t*>(sh);                          // [warps x keep]: the block's
  uint32_t* found = list + kSortWarps * keep;                                            // [warps][keep]
  int32_t* cnt = reinterpret_cast<int32_t*>(found) + kSortWarps * keep;    // [warps][K]
  __shared__ int32_t found_n[kSortWarps];
  __shared__ int32_t list_n;   // -1: not all kept
  __shared__ int32_t wsum[kSortWarps];
  __shared__ int32_t below_cluster, below_block;   // ids of lower clusters, in this block's part; of lower blocks in the cluster
  const int tid = threadIdx.x, lane = tid % 32, w = tid / 32;
  const unsigned lt = (1u << lane) - 1;
  const int blk = blockIdx.x, rank = blk & (kCluster - 1), cluster = blk >> kLogCluster;
  const int log_clusters = a.log_blocks - kLogCluster, mask = (1 << log_clusters) - 1;
  const unsigned rows = (unsigned)a.rows;
  const IT* index = static_cast<const IT*>(a.index);
  constexpr int U = 8;
  // The U ids of each lane from position i0 on, 32 positions side by side.
  auto load_ids = [&](int i0, int end, IT (&id)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 32 + lane;
      id[u] = i < end ? index[i] : (IT)-1;
    }
  };
  // f(cluster or -1, id, position) for the positions [beg, end), 32 at a time,
  // with the first ids loaded.
  auto scan = [&](int beg, int end, IT (&id)[U], auto f) {
    for (int i0 = beg; i0 < end; i0 += 32 * U) {
      IT next[U];
      load_ids(i0 + 32 * U, end, next);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * 32 >= end) break;
        f(cluster_of(id[u], rows, mask), id[u], i0 + u * 32 + lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = next[u];
    }
  };
  const int per_block = (a.n + kCluster - 1) / kCluster, per_warp = (per_block + kSortWarps - 1) / kSortWarps;
  const int first = min(rank * per_block, a.n), last = min(first + per_block, a.n);
  const int beg = min(first + w * per_warp, last), end = min(beg + per_warp, last);
  let_next_start();
  IT ids[U];
  load_ids(beg, end, ids);
  for (int i = tid; i < kSortWarps * K; i += kSortThreads) cnt[i] = 0;
  if (tid == 0) below_cluster = below_block = 0;
  for (int64_t i = (int64_t)blk * kSortThreads + tid; i < a.n_counters; i += (int64_t)gridDim.x * kSortThreads)
    a.counters[i] = 0;
  __syncthreads();
  int below = 0, mine_n = 0;
  bool bad = false;
  scan(beg, end, ids, [&](int b, IT id, int i) {
    below += (unsigned)b < (unsigned)cluster;
    if (cluster == 0) bad |= id >= a.rows;
    const unsigned who = __ballot_sync(0xffffffffu, b == cluster);
    if (!who) return;
    const int at = mine_n + __popc(who & lt);
    if (b == cluster && at < keep)   // the id without its cluster: block in the cluster, then number in the block
      found[w * keep + at] = (uint32_t)((int)id >> log_clusters) | (uint32_t)(i - first) << (kLogIds + kLogCluster);
    mine_n += __popc(who);
  });
  if (bad && a.status) atomicOr(a.status, kStatusIndex);
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0) {
    if (below) atomicAdd(&below_cluster, below);   // integers: any order gives the same
    found_n[w] = mine_n;
  }
  __syncthreads();
  {   // the warps' entries, one after the other
    const int n = lane < kSortWarps ? found_n[lane] : 0;
    int incl = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const bool kept = !__any_sync(0xffffffffu, n > keep) && per_block <= 1 << kLogPlace;
    const int off = __shfl_sync(0xffffffffu, incl - n, w), total = __shfl_sync(0xffffffffu, incl, 31);
    if (kept)
      for (int i = lane; i < mine_n; i += 32) list[off + i] = found[w * keep + i];
    if (tid == 0) list_n = kept ? total : -1;
  }
  cluster_arrive();
  cluster_wait();
  int start = lane < kCluster ? *of_block(&below_cluster, lane) : 0;   // all eight parts: ids of lower clusters
  for (int o = 16; o > 0; o >>= 1) start += __shfl_xor_sync(0xffffffffu, start, o);
  // f(number of the id in this block or -1, position, whether a lower block of
  // the cluster has it) over warp w's share of one of the cluster's lists, or,
  // where that was not all kept, of the positions it stands for.
  constexpr int kShares = kSortWarps / kCluster;   // warps to a list
  const int from = w / kShares, part = w % kShares;
  const int size = *of_block(&list_n, from);
  const uint32_t* theirs = of_block(list, from);
  auto each = [&](auto f) {
    const int base = min(from * per_block, a.n);
    if (size >= 0) {
      const int share = (size + 32 * kShares - 1) / (32 * kShares) * 32, end = min((part + 1) * share, size);
      constexpr int V = 8;
      for (int g0 = part * share; g0 < end; g0 += 32 * V) {
        uint32_t x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = g0 + v * 32 + lane < end ? theirs[g0 + v * 32 + lane] : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (g0 + v * 32 >= end) break;
          const int b = g0 + v * 32 + lane < end ? (int)(x[v] & (kCluster - 1)) : kCluster;
          f(b == rank ? (int)(x[v] >> kLogCluster & ((1 << kLogIds) - 1)) : -1, base + (int)(x[v] >> (kLogIds + kLogCluster)),
            b < rank);
        }
      }
    } else {
      const int stop = min(base + per_block, a.n), share = (per_block + kShares - 1) / kShares;
      const int b0 = min(base + part * share, stop), b1 = min(b0 + share, stop);
      load_ids(b0, b1, ids);
      scan(b0, b1, ids, [&](int b, IT id, int i) {
        const int in = (int)id >> log_clusters & (kCluster - 1);
        f(b == cluster && in == rank ? (int)id >> a.log_blocks : -1, i, b == cluster && in < rank);
      });
    }
  };
  // Counts, and the block's own entries of the warp's share, for the second
  // time (number in the block, position), in the place of what it found.
  int lower = 0, own_n = 0;
  const int own_keep = keep / 2;
  uint2* own = reinterpret_cast<uint2*>(found + w * keep);
  each([&](int k, int pos, bool low) {
    lower += low;
    const unsigned who = __ballot_sync(0xffffffffu, k >= 0);
    if (!who) return;
    const int at = own_n + __popc(who & lt);
    if (k >= 0) {
      atomicAdd(cnt + w * K + k, 1);
      if (at < own_keep) own[at] = make_uint2(k, pos);
    }
    own_n += __popc(who);
  });
  // No block leaves while another reads its lists: this warp says that it is
  // done with them, now if it need not read them again.
  const bool again = own_n > own_keep;
  if (!again) cluster_arrive();
  for (int o = 16; o > 0; o >>= 1) lower += __shfl_xor_sync(0xffffffffu, lower, o);
  if (lane == 0 && lower) atomicAdd(&below_block, lower);
  __syncthreads();
  // Per id: its total, then the ids' totals a scan, then the warps' starts.
  int mine = 0;
  if (tid < K) {
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) mine += cnt[k * K + tid];
  }
  int incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) wsum[w] = incl;
  __syncthreads();
  if (w == 0) {
    int t = lane < kSortWarps ? wsum[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    if (lane < kSortWarps) wsum[lane] = t;
  }
  __syncthreads();
  start += below_block + (w ? wsum[w - 1] : 0) + incl - mine;
  if (tid < K) {
    a.offsets[blk * K + tid] = start;
    if (blk == (int)gridDim.x - 1 && tid == K - 1) a.offsets[blk * K + K] = start + mine;
    int c[kSortWarps];   // all loads before the first store
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) c[k] = cnt[k * K + tid];
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) {
      cnt[k * K + tid] = start;
      start += c[k];
    }
  }
  __syncthreads();
  auto put = [&](int k, int pos) {
    const unsigned peers = __match_any_sync(0xffffffffu, k);
    if (k >= 0) {
      const int at = cnt[w * K + k] + __popc(peers & lt);
      a.order[at] = pos;
      a.key[at] = k << a.log_blocks | rank << log_clusters | cluster;
    }
    __syncwarp();
    if (k >= 0 && lane == __ffs(peers) - 1) cnt[w * K + k] += __popc(peers);
    __syncwarp();
  };
  if (!again) {
    for (int c = 0; c < own_n; c += 32) {
      const bool in = c + lane < own_n;
      const uint2 x = in ? own[c + lane] : make_uint2(0xffffffffu, 0);
      put((int)x.x, (int)x.y);
    }
  } else {
    each([&](int k, int pos, bool) {
      if (__any_sync(0xffffffffu, k >= 0)) put(k, pos);
    });
    cluster_arrive();
  }
  cluster_wait();
}

// ---- backward: sums ----------------------------------------------------------------
constexpr int kMaxChunk = 32;
constexpr int kZeroRows = 16;       // table rows a block of the other kind looks after

struct EmbedSum {
  const void* grad_out;
  const int32_t *order, *key, *offsets;
  int32_t* counters;       // [chunks][gridDim.y]: arrivals of the run that starts in the chunk
  float* part;             // [chunks][2][cols]: sums of a run entering / leaving the chunk
  float* grad;
  int64_t gs, cols, os;    // os: between rows of grad
  int rows, log_blocks, ids_per_block, last_offset, chunk, accumulate;
  int zero_blocks, zero_vec, n;
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

// Place of id v in the sorted order of ids.
__device__ __forceinline__ int place_of(const EmbedSum& a, int v) {
  const int log_clusters = a.log_blocks - kLogCluster;
  const int blk = (v & ((1 << log_clusters) - 1)) << kLogCluster | (v >> log_clusters & (kCluster - 1));
  return blk * a.ids_per_block + (v >> a.log_blocks);
}

// Zeros into the rows without tokens among the kZeroRows from b * kZeroRows
// on, a warp per row; streaming stores, since no one reads zeros soon (the
// whole gradient of 4,099 tokens, 50,257 x 768: 32.3 us, of which a plain fill
// of as many bytes takes 25; 4 us more with plain stores, 2.6 with bulk stores
// from shared memory).
__device__ __forceinline__ void zero_rows(const EmbedSum& a, int b) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  wait_for_previous();
  for (int k = threadIdx.x / 32; k < kZeroRows; k += warps) {
    const int v = b * kZeroRows + k;
    if (v >= a.rows) break;
    const int at = place_of(a, v);
    if (a.offsets[at] != a.offsets[at + 1]) continue;
    float* g = a.grad + (int64_t)v * a.os;
    if (a.zero_vec) {
      for (int64_t j = lane * 4; j < a.cols; j += 128) __stcs(reinterpret_cast<float4*>(g + j), make_float4(0.f, 0.f, 0.f, 0.f));
    } else {
      for (int64_t j = lane; j < a.cols; j += 32) __stcs(g + j, 0.f);
    }
  }
}

// 80 registers, for eight rows' loads side by side: 24 warps per SM take 114 us
// for 65,536 tokens of 2048 bfloat16 into 50,304 rows (5.7 TB/s), 32 warps with
// 64 registers 126, 16 warps 126, 40 warps 154.
template <typename T, int VEC>
__global__ void __launch_bounds__(256, 3) k_embed_sum(const EmbedSum a) {
  __shared__ int32_t ord[kMaxChunk], key[kMaxChunk + 2];   // key[0]: before the chunk, key[len + 1]: after it
  __shared__ int32_t last_flag;
  // Blocks of the two kinds alternate evenly over the grid.
  const int zeros_before = (int)((int64_t)blockIdx.x * a.zero_blocks / gridDim.x);
  if ((int64_t)(blockIdx.x + 1) * a.zero_blocks / gridDim.x > zeros_before) {
    if (blockIdx.y == 0) zero_rows(a, zeros_before);
    return;
  }
  const int chunk = (int)blockIdx.x - zeros_before;
  const int64_t j = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  const bool live = j < a.cols;
  const int base = chunk * a.chunk;
  wait_for_previous();
  const int total = a.offsets[a.last_offset];
  for (int i = threadIdx.x; i < a.chunk + 2; i += blockDim.x) {
    const int at = base + i - 1;
    const bool in = at >= 0 && at < a.n;   // what lies past the total is not sorted, but there
    const int k = in ? a.key[at] : -1;
    if (i >= 1 && i <= a.chunk) ord[i - 1] = in ? a.order[at] : 0;
    key[i] = at < total ? k : -1;
  }
  if (base >= total) return;
  const int len = min(a.chunk, total - base);
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
          store_sums<VEC>(a.part + ((int64_t)chunk * 2 + (from_before ? 0 : 1)) * a.cols + j, acc);
        } else {
          float* g = a.grad + (int64_t)key[i + 1] * a.os + j;
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
    const int at = place_of(a, v);
    const int s0 = a.offsets[at], s1 = a.offsets[at + 1];
    const int first = s0 / a.chunk, last = (s1 - 1) / a.chunk;
    if (side == 1 && head_open && first < chunk) continue;   // one run through the whole chunk: counted
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
    float* g = a.grad + (int64_t)v * a.os + j;
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
  // Short lists in short chunks, for enough blocks (text-like ids, bfloat16
  // rows of 768 into 50,257: 8,192 positions 41.6 us, 45.7 with chunks of 32;
  // 16,384 47.8 with either; 32,768 53.9, 66.2 with chunks of 8).  A hot id turns
  // that round, since its chunks are joined by one block (half of 8,192
  // positions: 79 us, 52 with chunks of 32), but is known only after the sort.
  p.chunk = n >= 16384 ? kMaxChunk : 8;
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

template <typename TI, typename TO, int VEC, int C>
cudaError_t fwd_as(const EmbedFwd& a, int sms, cudaStream_t s) {
  const int64_t nv = (a.cols + VEC * C - 1) / (VEC * C);
  const int tx = (int)std::min<int64_t>((nv + 31) / 32 * 32, 256);
  const int ty = std::max(1, 256 / tx);
  const unsigned gy = (unsigned)((nv + tx - 1) / tx);
  // Four tokens per thread once that still fills every SM's eight blocks
  // (float32 to bfloat16, in a graph: 65,536 tokens of 2048 108 us, 117 with one;
  // 4,864 of 768 5.7 with either; 256 1.65 with one, 1.97 with four).
  const bool many = a.n * gy >= (int64_t)sms * 8 * 4 * ty;
  const int64_t per = many ? 4 * ty : ty;
  return launch(many ? k_embed_fwd<TI, TO, VEC, 4, C> : k_embed_fwd<TI, TO, VEC, 1, C>, dim3((unsigned)((a.n + per - 1) / per), gy),
                dim3(tx, ty), 0, s, false, 1, a);
}
template <typename TI, typename TO>
cudaError_t fwd_as(const EmbedFwd& a, int vec, int sms, cudaStream_t s) {
  if constexpr (sizeof(TI) + sizeof(TO) < 8)
    if (vec == 8) return fwd_as<TI, TO, 8, 1>(a, sms, s);
  if (vec == 4) return fwd_as<TI, TO, 4, 1>(a, sms, s);
  // Single elements, four of a row (33.5M elements, rows of 1001: 38 us; 62 with one).
  return fwd_as<TI, TO, 1, 4>(a, sms, s);
}

template <typename TI>
cudaError_t fwd_from(const EmbedFwd& a, int out_type, int vec, int sms, cudaStream_t s) {
  switch (out_type) {
    case LOPT_F32: return fwd_as<TI, float>(a, vec, sms, s);
    case LOPT_F16: return fwd_as<TI, __half>(a, vec, sms, s);
    default: return fwd_as<TI, __nv_bfloat16>(a, vec, sms, s);
  }
}

template <typename IT, int WARPS>
cudaError_t sort_as(EmbedSort a, cudaStream_t s) {
  a.found = found_of(WARPS, a.n);
  const size_t smem = (size_t)WARPS * (2 * a.found + a.ids_per_block) * 4;
  auto* k = &k_embed_sort<IT, WARPS>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
  if (e != cudaSuccess) return e;
  return launch(k, dim3(1u << a.log_blocks), dim3(32 * WARPS), smem, s, false, kCluster, a);
}

template <typename T, int VEC>
cudaError_t sum_as(const EmbedSum& a, int chunks, cudaStream_t s) {
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  const int tx = (int)std::min<int64_t>((nv + 31) / 32 * 32, 256);
  const dim3 grid((unsigned)(chunks + a.zero_blocks), (unsigned)((nv + tx - 1) / tx));
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
  // 8 elements per thread when either side is 16-bit, else 4, as the rows allow.
  auto fits = [&](int v) { return cols % v == 0 && rows_aligned(mt, v * ti) && rows_aligned(mo, v * to); };
  const int vec = ti + to < 8 && fits(8) ? 8 : fits(4) ? 4 : 1;
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
  return embed_backward_to(grad_out, type, grad_out_stride, index, index_type, n, rows, cols, scale, accumulate, grad, cols,
                           workspace, workspace_bytes, status, stream);
}

}  // extern "C"

int lopt::train::embed_backward_to(const void* grad_out, int type, int64_t grad_out_stride, const void* index, int index_type,
                                   int64_t n, int64_t rows, int64_t cols, float scale, int accumulate, float* grad,
                                   int64_t grad_stride, void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  const int es = type_size(type), is = index_size(index_type);
  if (!es || !is || (accumulate != 0 && accumulate != 1)) return LOPT_E_ARG;
  int64_t need = 0;
  int rc = lopt_embed_workspace(n, rows, cols, &need);
  if (rc) return rc;
  const Span mg{grad, rows, cols, grad_stride, 4};
  if ((rc = check_matrix(mg, true))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  if (n == 0) return accumulate ? LOPT_OK : done(cudaMemset2DAsync(grad, (rows == 1 ? cols : grad_stride) * 4, 0, cols * 4, rows, s));
  const Span md{grad_out, n, cols, grad_out_stride, es}, mi{index, 1, n, n, is}, ws{workspace, 1, need, need, 1};
  if ((rc = check_matrix(md, false)) || (rc = check_matrix(mi, false))) return rc;
  if (!workspace || workspace_bytes < need) return LOPT_E_ARG;
  if ((uintptr_t)workspace % 256 || (status && (uintptr_t)status % 4)) return LOPT_E_ALIGN;
  if (overlap(mg, md) || overlap(mg, mi) || overlap(mg, ws) || overlap(ws, md) || overlap(ws, mi)) return LOPT_E_ALIAS;
  const Plan p = plan(n, rows, cols);
  char* w = static_cast<char*>(workspace);
  const bool v4 = cols % 4 == 0 && rows_aligned(mg, 16);
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
  // 16 warps while each thread can look after one id of its block.
  cudaError_t e;
  const bool wide = p.ids_per_block > 512;
  if (index_type == LOPT_I32) e = wide ? sort_as<int32_t, 32>(a, s) : sort_as<int32_t, 16>(a, s);
  else e = wide ? sort_as<int64_t, 32>(a, s) : sort_as<int64_t, 16>(a, s);
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
  b.os = grad_stride;
  b.rows = (int)rows;
  b.n = (int)n;
  b.zero_blocks = accumulate ? 0 : (int)((rows + kZeroRows - 1) / kZeroRows);
  b.zero_vec = v4;
  b.log_blocks = p.log_blocks;
  b.ids_per_block = p.ids_per_block;
  b.last_offset = p.ids_per_block << p.log_blocks;
  b.chunk = p.chunk;
  b.accumulate = accumulate;
  b.scale = scale;
  const int vec = 16 / es;
  const bool rows16 = cols % vec == 0 && rows_aligned(md, 16) && v4;
  switch (type) {
    case LOPT_F32: return done(rows16 ? sum_as<float, 4>(b, p.chunks, s) : sum_as<float, 1>(b, p.chunks, s));
    case LOPT_F16: return done(rows16 ? sum_as<__half, 8>(b, p.chunks, s) : sum_as<__half, 1>(b, p.chunks, s));
    default:
      return done(rows16 ? sum_as<__nv_bfloat16, 8>(b, p.chunks, s) : sum_as<__nv_bfloat16, 1>(b, p.chunks, s));
  }
}
