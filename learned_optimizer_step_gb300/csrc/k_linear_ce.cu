// Linear cross entropy: softmax cross entropy of hidden states x [N x D] against
// an output table W [V x D] (see lopt_lm.h for the formulas).
//
// Three matrix products by one persistent kernel on the tensor cores, with what
// surrounds them in its epilogues, so that logits never leave the SM:
//
//   loss     tile of x W^T  ->  each row's maximum and sum of exponentials over the
//                               tile's classes but its target
//   grad     tile of x W^T  ->  G = (exp(logit - lse) - [target]) * weight, 16-bit
//   grad_x   tile of G W        (sum over classes, in pieces of the vocabulary)
//   grad_w   tile of G^T x      (sum over tokens)
//
// The backward pass goes over the vocabulary in chunks whose G fits a bounded
// workspace; the chunk's grad_x is added to fp32 sums, its rows of grad_w are
// written.  G is held as the sum of 16-bit numbers: for a 32-bit grad_w two (16 bits
// of bfloat16, 22 of float16), or three of bfloat16 while the targets' entries are in
// it; for a 16-bit grad_w two, or one without the targets' entries.
//
// A pair of CTAs (cta_group::2) computes a 256 x 256 tile: each holds 128 rows of
// A and 128 of B per 64-wide step of K in shared memory (TMA, 128-byte swizzle) and
// 128 rows of the accumulator in its tensor memory, twice, so that a tile's
// epilogue runs beside the next tile's product.  Roles: warp 0 loads, warp 1 of the
// pair's first CTA issues, warps 4 to 11 are the epilogue.
//
// The tensor cores cut the fp32 sums they carry rather than round them: over
// thousands of steps that is more than fp32 results may be off.  What is cut goes
// by the largest terms, and those are the targets'.  So a target's logit is a dot
// product of its own, summed in two floats, which replaces the tensor cores' in the sum of
// exponentials and in G; and with many tokens the targets' entries stay out of G: their
// share is added in fp32, to grad_x by the last kernel, to a 32-bit grad_w by the
// embedding's gradient, to a 16-bit one by its tiles' epilogue, from a table whose rows are
// the classes that are targets.  Where they are in the G of a 32-bit grad_w, an accumulator
// takes a segment of a few steps only, and the epilogue's warps add the segments in
// registers, rounding to nearest (8,192 x 2048 x 50,304 with 4 steps for logits and 8 for
// grad_w throughout: float16 forward 1.32 ms, bfloat16 backward 5.09).
//
// Bound by the tensor cores and the power they draw: of 8,192 x 2048 x 50,304 bfloat16 the
// forward pass takes 1.00 ms (1,690 TFLOP/s; library products 1,914 at first, 1,705 once the
// GPU draws 1.4 kW; float16 1.09 to 1.13), the backward pass 4.5 to 4.6 ms (1,500 to 1,470
// over 6.75 TFLOP: logits again, grad_x, grad_w with both parts of G), with a 16-bit grad_w
// 3.2 to 3.3.  4,099 x 768 x 50,257 float16: 1.03 to 1.07 ms; a tile of 12 steps of K is over
// before the epilogue that makes G.  That of several segments spills 56 bytes.
// Few tokens read W at 2.5 TB/s: a tile is 256 rows of x whatever there are.
#include <algorithm>
#include <cmath>
#include <cuda.h>

#include "lopt_lm.h"
#include "tc_layout.cuh"
#include "train_common.cuh"

namespace lopt {
namespace train {
namespace {

constexpr int kTile = 256;                       // rows and columns of a pair's tile
constexpr int kHalf = 128;                       // ... of one CTA's part of an operand
constexpr int kStep = 64;                        // K elements of a stage: 128 bytes
constexpr int kStages = 5;                       // 6 were no faster (8,192 x 2048 x 50,304 backward 4.50 ms, 4.45 with 5)
constexpr int kOperand = kHalf * kStep * 2;      // bytes of one operand of a stage
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
// Registers of a thread at launch, and after the first warpgroup has handed some
// to the epilogue's two: 128 * 40 + 256 * 232 is 384 * 168.
constexpr int kRegs = 168, kRegsFew = 40, kRegsMany = 232;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads * kRegs, "");
constexpr int kPitch = 20;
constexpr int kTurn = 32 * kPitch;               // floats of a warp's place to turn 16 columns of 32 rows
constexpr size_t kSmem = (size_t)kStages * 2 * kOperand + 1024 + kEpilogueWarps * kTurn * 4;
constexpr int kRowGroup = 32;                    // tiles of rows that share the classes' operand in L2
constexpr uint64_t kLimitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

enum Mode { kLoss = 0, kGrad = 1, kGradX = 2, kGradW = 3 };

constexpr int kMaxPairs = 128;
constexpr int kMaxCtas = 256;
constexpr int kGroups = 12;

// Which pair takes which of a job's tiles.  In round r the pairs that take more than r
// tiles take the next ones, so that tiles side by side, which share an operand, are
// worked on at the same time.  The pairs that take equally many are a group.
struct Spread {
  int count[kMaxPairs];
  uint8_t place[kMaxPairs];    // among the pairs, those that take most first
  int pairs, groups, size[kGroups], takes[kGroups];
};

// Division of 0 <= t < 2^31 by d: with 2^(l - 1) < d <= 2^l and mul = ceil(2^(31 + l) / d),
// t * mul / 2^(31 + l) is above t / d by less than 1 / d.  (A division in the instruction
// stream of the thread that feeds the tensor cores takes as long as two steps of K.)
struct FastDiv {
  uint32_t mul = 1u << 31, shift = 31;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    shift = 31 + l;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int t) const { return (int)((uint64_t)(uint32_t)t * mul >> shift); }
};

// One kind of tiles of a launch.
struct Job {
  int mode, tiles;
  int m_tiles, n_tiles, splits;
  int k_steps;                 // of the whole product
  int buffer;                  // which G
  int v0, v1;                  // classes of the chunk
  int add;                     // grad_x: add to the sums
  int segment;                 // K steps that one accumulator sums
  FastDiv by_group, by_rows, by_last, by_n, by_splits;   // divisions by numbers of tiles
};
constexpr int kJobs = 3;

struct Maps {
  CUtensorMap x_k, x_m, w_k, w_m, g_k[2][2], g_m[2][3];     // by buffer, by part
};

struct Args {
  int rows, classes, cols;
  int planes, planes_x;        // parts of G, those that grad_x uses
  int is_bf16;
  const void* target;
  int index_type;
  const float* row_weight;     // NULL: 1
  const float* lse;
  const float* hit;            // [rows]: exp(target logit - lse) - 1
  int split;                   // the targets' entries stay out of G
  const int* slot;             // [classes]: a class's row of `table`, -1: none; NULL: none has
  const float* table;          // the targets' share of a 16-bit grad_w
  int64_t table_stride;
  float2* part;                // [2 * class tiles][rows]: maximum, sum
  void* g[2][3];               // [buffer][part]
  int64_t g_stride;
  const float* largest;        // the largest |row_weight|: G is scaled by 2^15 / *largest
  float* dx;
  int64_t dx_stride, dx_slice;
  void* dw;
  int dw_type, accumulate;
  int64_t dw_stride;
  int* gave_up;                // one word per CTA
  int32_t* status;
  uint64_t limit_ns;           // of a wait
  Job job[kJobs];
  Spread spread[kJobs];
  int jobs;
};

// ---- PTX -----------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A box of a matrix to this CTA's shared memory; its bytes count on the
// barrier of the pair's first CTA.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrives on the barrier at this offset of both CTAs once the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// The same without the instruction's own short wait.
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Bounded: gives up after limit_ns, or when another warp of the CTA has.
// Inline: a call would spill the sums that the epilogue holds meanwhile.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (limit_ns == 0) {      // the self-test's
    if (!*abort && test_wait(bar, parity)) return true;
    *abort = 1;
    return false;
  }
  if (try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t it = 0; it < (1u << 30); ++it) {
    if (try_wait(bar, parity)) return true;
    if ((it & 15) == 15) {
      if (*abort) return false;
      if (global_ns() - t0 > limit_ns) break;
    }
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Shared-memory descriptors, 128-byte swizzle, groups of eight 128-byte rows 1024
// bytes apart.  K along the rows: the operand is one box of 128 rows.  K across
// them: two boxes of 64 columns each, 8192 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool k_rows) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)(k_rows ? 1 : 8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// ---- tiles ---------------------------------------------------------------------
struct Tile {
  int m, n, split, k0, k1;   // K steps [k0, k1)
};

__device__ __forceinline__ Tile tile_of(const Job& j, int t) {
  Tile r;
  if (j.mode <= kGrad) {
    // Rows fastest, in groups that stay in L2 while the classes pass by.
    const int group = j.by_group(t), left = t - group * kRowGroup * j.n_tiles;
    const int in_group = min(kRowGroup, j.m_tiles - group * kRowGroup);
    r.n = in_group == kRowGroup ? j.by_rows(left) : j.by_last(left);
    r.m = group * kRowGroup + left - r.n * in_group;
    r.split = 0;
  } else {
    const int q = j.by_n(t);
    r.n = t - q * j.n_tiles;
    r.m = j.by_splits(q);
    r.split = q - r.m * j.splits;
  }
  r.k0 = j.by_splits(j.k_steps * r.split);
  r.k1 = j.by_splits(j.k_steps * (r.split + 1));
  return r;
}
// A pair's tiles of a launch, job after job.
struct Walk {
  const Args& a;
  int pair, job = 0, round = 0;
  int base = 0, active = 0, group = 0;      // the round's first tile; the pairs that take one
  __device__ __forceinline__ Walk(const Args& args, int p) : a(args), pair(p) { start(); }
  __device__ __forceinline__ void start() {
    round = base = 0;
    if (job >= a.jobs) return;
    active = a.spread[job].pairs;
    group = a.spread[job].groups;
    leave();
  }
  // The groups that have had all of theirs.
  __device__ __forceinline__ void leave() {
    const Spread& s = a.spread[job];
    while (group > 0 && s.takes[group - 1] <= round) active -= s.size[--group];
  }
  __device__ __forceinline__ bool more() {
    while (job < a.jobs && round >= a.spread[job].count[pair]) {
      ++job;
      start();
    }
    return job < a.jobs;
  }
  __device__ __forceinline__ Tile next() {
    const int t = base + a.spread[job].place[pair];
    base += active;
    ++round;
    leave();
    return tile_of(a.job[job], t);
  }
  // Its K steps alone.
  __device__ __forceinline__ void next_steps(int& k0, int& k1) {
    if (a.job[job].splits == 1) {
      k0 = 0;
      k1 = a.job[job].k_steps;
      ++round;
    } else {
      const Tile t = next();
      k0 = t.k0;
      k1 = t.k1;
    }
  }
};

// ---- epilogues: a thread has 128 columns of a row, and takes 32 at a time ----------
// From the accumulator itself, where that has summed all of K: a loop, so that few
// registers are in use.
struct FromTmem {
  static constexpr int kUnroll = 1;
  uint32_t src;
  __device__ __forceinline__ void get(int c, float (&v)[32]) const {
    uint32_t r[32];
    __syncwarp();
    tmem_ld32(src + 32 * c, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
  }
};
// From the sums of several segments.
struct FromSums {
  static constexpr int kUnroll = 4;
  const float (&acc)[kHalf];
  __device__ __forceinline__ void get(int c, float (&v)[32]) const {
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = acc[32 * c + k];
  }
};

// What an epilogue wants of its row: loaded while the tile before is worked on.
struct RowLoads {
  int64_t target = -1;
  float weight = 1.f, lse = 0.f, hit = 0.f;
};
__device__ __forceinline__ RowLoads load_row(const Args& a, const Job& j, int row) {
  RowLoads r;
  if (j.mode == kGradW) {      // its row is a class
    if (a.slot && j.v0 + row < j.v1) r.target = a.slot[j.v0 + row];
    return r;
  }
  if (j.mode > kGrad || row >= a.rows) return r;
  r.target = load_index(a.target, row, a.index_type);
  if (j.mode == kGrad) {
    if (a.row_weight) r.weight = a.row_weight[row];
    r.lse = a.lse[row];
    r.hit = a.hit[row];
  }
  return r;
}
struct RowIn {
  int target;            // -1: none; grad_w: the class's row of `table`
  float lse, scale, hit;
};
__device__ __forceinline__ RowIn row_in(const Args& a, int mode, const RowLoads& q, float largest) {
  if (mode == kGradW) return RowIn{(int)q.target, 0.f, 0.f, 0.f};
  const bool live = q.target >= 0 && q.target < a.classes && q.weight != 0.f;
  return RowIn{live ? (int)q.target : -1, q.lse, live ? q.weight / largest * 32768.f : 0.f, q.hit};
}
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

template <typename Src>
__device__ __forceinline__ void loss_tile(const Args& a, const Tile& t, const RowIn& in, int row, int col, int half, const Src& src) {
  float most = -INFINITY, sum = 0.f;
#pragma unroll Src::kUnroll
  for (int c = 0; c < 4; ++c) {
    float v[32];
    src.get(c, v);
    const int c0 = col + 32 * c;
    if (c0 + 32 > a.classes) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (c0 + k >= a.classes) v[k] = -INFINITY;
    }
    const int at = in.target - c0;      // added by the rows' kernel
    if (at >= 0 && at < 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (at == k) v[k] = -INFINITY;
    }
    float m = most;
#pragma unroll
    for (int k = 0; k < 32; ++k) m = fmaxf(m, v[k]);
    // Nothing but -inf so far: 0 keeps exponents of it at 0.
    const float base = m == -INFINITY ? 0.f : m;
    float2 s2 = two(0.f);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float2 z = __fmul2_rn(__fadd2_rn(make_float2(v[k], v[k + 1]), two(-base)), two(kLog2e));
      s2 = __fadd2_rn(s2, make_float2(exp2_fast(z.x), exp2_fast(z.y)));
    }
    sum = fmaf(sum, exp2_fast((most - base) * kLog2e), s2.x + s2.y);
    most = m;
  }
  if (row < a.rows) a.part[(int64_t)(2 * t.n + half) * a.rows + row] = make_float2(most, sum);
}

template <typename T, typename Src>
__device__ __forceinline__ void grad_tile(const Args& a, const Job& j, const RowIn& in, int row, int col, const Src& src) {
  const float lse = in.lse, scale = in.scale;
  const bool live = row < a.rows;
  const int64_t out = (int64_t)row * a.g_stride + (col - j.v0);
#pragma unroll Src::kUnroll
  for (int c = 0; c < 4; ++c) {
    float v[32];
    src.get(c, v);
    const int c0 = col + 32 * c;
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float2 z = __fmul2_rn(__fadd2_rn(make_float2(v[k], v[k + 1]), two(-lse)), two(kLog2e));
      const float2 p = __fmul2_rn(make_float2(exp2_fast(z.x), exp2_fast(z.y)), two(scale));
      v[k] = p.x, v[k + 1] = p.y;
    }
    const int at = in.target - c0;
    if (at >= 0 && at < 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        if (at == k) v[k] = a.split ? 0.f : in.hit * scale;
      }
    }
    // Rows that do not count, whatever their logits hold, and classes past the last.
    if (scale == 0.f || c0 + 32 > a.classes) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (scale == 0.f || c0 + k >= a.classes) v[k] = 0.f;
    }
    if (!live) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x[2] = {v[16 * h + 2 * k], v[16 * h + 2 * k + 1]};
        const Pack<T, 2> p = from_floats<T, 2>(x);
        float y[2];
        to_floats(p, y);
        const float2 rest = __fadd2_rn(make_float2(x[0], x[1]), make_float2(-y[0], -y[1]));
        const float z[2] = {rest.x, rest.y};
        const Pack<T, 2> q = from_floats<T, 2>(z);
        hi[k] = *reinterpret_cast<const uint32_t*>(&p);
        lo[k] = *reinterpret_cast<const uint32_t*>(&q);
      }
      store32(static_cast<T*>(a.g[j.buffer][0]) + out + 32 * c + 16 * h, hi);
      if (a.planes == 1) continue;
      store32(static_cast<T*>(a.g[j.buffer][1]) + out + 32 * c + 16 * h, lo);
      if (a.planes == 2) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float y[2], z[2], x[2] = {v[16 * h + 2 * k], v[16 * h + 2 * k + 1]};
        to_floats(*reinterpret_cast<const Pack<T, 2>*>(&hi[k]), y);
        to_floats(*reinterpret_cast<const Pack<T, 2>*>(&lo[k]), z);
        x[0] = (x[0] - y[0]) - z[0];
        x[1] = (x[1] - y[1]) - z[1];
        const Pack<T, 2> q = from_floats<T, 2>(x);
        lo[k] = *reinterpret_cast<const uint32_t*>(&q);
      }
      store32(static_cast<T*>(a.g[j.buffer][2]) + out + 32 * c + 16 * h, lo);
    }
  }
}

// A warp's 32 rows of 32 columns to memory.  They are turned in shared
// memory, 16 columns at a time, so that the lanes of a store fill whole sectors: each
// thread writing its own row leaves a sector to two stores of 32 rows each, or, element
// by element, to 16 (us, grad_w of 100 x 100,000 classes fp16: 2000 wide 448 in all, 1999
// wide 3,012).  Rows on 16-byte boundaries by vectors.
struct Block {
  int rows, cols;      // that there are, from the first on
  int64_t stride;
  bool vec, add;
};
template <typename O>
__device__ __forceinline__ void store_block(O* out, const Block& b, float* turn, const float (&x)[32]) {
  constexpr int VEC = 16 / sizeof(O), N = 16 / VEC;      // lanes of a row's 16 columns
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      *reinterpret_cast<float4*>(turn + lane * kPitch + k) =
          make_float4(x[16 * h + k], x[16 * h + k + 1], x[16 * h + k + 2], x[16 * h + k + 3]);
    __syncwarp();
    if (b.vec) {
      const int k = lane % N * VEC;
#pragma unroll
      for (int r = lane / N; r < 32; r += 32 / N) {
        if (r >= b.rows || 16 * h + k >= b.cols) continue;
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = turn[r * kPitch + k + e];
        Pack<O, VEC>* q = reinterpret_cast<Pack<O, VEC>*>(out + r * b.stride + 16 * h + k);
        if (b.add) {
          float o[VEC];
          to_floats(*q, o);
#pragma unroll
          for (int e = 0; e < VEC; ++e) y[e] += o[e];
        }
        *q = from_floats<O, VEC>(y);
      }
    } else {
      const int k = lane % 16;
#pragma unroll 4
      for (int r = lane / 16; r < 32; r += 2) {
        if (r >= b.rows || 16 * h + k >= b.cols) continue;
        O* q = out + r * b.stride + 16 * h + k;
        const float y = turn[r * kPitch + k];
        *q = from_f<O>(b.add ? y + to_f(*q) : y);
      }
    }
  }
}

template <typename Src>
__device__ __forceinline__ void grad_x_tile(const Args& a, const Job& j, const Tile& t, int row, int col, float* turn, const Src& src) {
  const int first = row - threadIdx.x % 32;
  float* out = a.dx + t.split * a.dx_slice + (int64_t)first * a.dx_stride + col;
#pragma unroll Src::kUnroll
  for (int c = 0; c < 4; ++c) {
    float v[32];
    src.get(c, v);
    store_block<float>(out + 32 * c, Block{a.rows - first, (int)a.dx_stride - col - 32 * c, a.dx_stride, true, j.add != 0}, turn, v);
  }
}

template <typename O, typename Src>
__device__ __forceinline__ void grad_w_tile(const Args& a, const Job& j, int v, int slot, int col, float* turn, const Src& src) {
  constexpr int VEC = 16 / sizeof(O);
  const bool vec = (a.cols % VEC == 0) && (a.dw_stride % VEC == 0) && (reinterpret_cast<uintptr_t>(a.dw) % 16 == 0);
  const int first = v - threadIdx.x % 32;
  O* out = static_cast<O*>(a.dw) + (int64_t)first * a.dw_stride + col;
  const float largest = *a.largest;
#pragma unroll Src::kUnroll
  for (int c = 0; c < 4; ++c) {
    float x[32];
    src.get(c, x);
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = x[k] * (1.f / 32768.f) * largest;
    if (slot >= 0) {      // the thread's class is a target: a line of its share
      const float* q = a.table + slot * a.table_stride + col + 32 * c;
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const float4 t = *reinterpret_cast<const float4*>(q + k);
        x[k] += t.x, x[k + 1] += t.y, x[k + 2] += t.z, x[k + 3] += t.w;
      }
    }
    store_block<O>(out + 32 * c, Block{j.v1 - first, a.cols - col - 32 * c, a.dw_stride, vec, a.accumulate != 0}, turn, x);
  }
}

template <typename Src>
__device__ __forceinline__ void finish_tile(const Args& a, const Job& j, const Tile& t, const RowIn& in, int row, int col, int half,
                                            float* turn, const Src& src) {
  if (j.mode == kLoss) {
    loss_tile(a, t, in, row, j.v0 + col, half, src);
  } else if (j.mode == kGrad) {
    if (a.is_bf16) grad_tile<__nv_bfloat16>(a, j, in, row, j.v0 + col, src);
    else grad_tile<__half>(a, j, in, row, j.v0 + col, src);
  } else if (j.mode == kGradX) {
    grad_x_tile(a, j, t, row, col, turn, src);
  } else if (a.dw_type == LOPT_F32) {
    grad_w_tile<float>(a, j, j.v0 + row, in.target, col, turn, src);
  } else if (a.dw_type == LOPT_F16) {
    grad_w_tile<__half>(a, j, j.v0 + row, in.target, col, turn, src);
  } else {
    grad_w_tile<__nv_bfloat16>(a, j, j.v0 + row, in.target, col, turn, src);
  }
}

// ---- the kernel ------------------------------------------------------------------
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_linear_ce(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x / 2;
  const uint32_t stages = (smem_u32(raw) + 1023) & ~1023u;
  volatile int* abort = &s_abort;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int k = 0; k < kStages; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&s_empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_acc_full[k], 1);
      mbar_init(&s_acc_empty[k], 2 * kEpilogueWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  wait_for_previous();
  let_next_start();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsFew));
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (Walk walk(a, pair); walk.more();) {
        const Job& j = a.job[walk.job];
        const Tile x = walk.next();
        const int m0 = x.m * kTile + rank * kHalf, n0 = x.n * kTile + rank * kHalf;
        for (int k = x.k0; k < x.k1; ++k) {
          if (!wait_for(smem_u32(&s_empty[stage]), phase ^ 1, abort, a.limit_ns)) break;
          const uint32_t sa = stages + stage * 2 * kOperand, sb = sa + kOperand;
          const uint32_t bar = in_cta(smem_u32(&s_full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&s_full[stage], 4 * kOperand);
          const int kk = k * kStep;
          if (j.mode <= kGrad) {
            load_box(sa, &maps.x_k, kk, m0, bar);
            load_box(sb, &maps.w_k, kk, j.v0 + n0, bar);
          } else if (j.mode == kGradX) {
            const int part = a.planes_x == 2 ? k & 1 : 0, v = (a.planes_x == 2 ? k >> 1 : k) * kStep;
            load_box(sa, &maps.g_k[j.buffer][part], v, m0, bar);
            load_box(sb, &maps.w_m, n0, j.v0 + v, bar);
            load_box(sb + kOperand / 2, &maps.w_m, n0 + 64, j.v0 + v, bar);
          } else {
            // The parts of G against the same tokens, one after the other.
            const int tokens = a.planes == 1 ? k : a.planes == 2 ? k >> 1 : k / 3, y = tokens * kStep;
            const CUtensorMap* g = &maps.g_m[j.buffer][k - tokens * a.planes];
            load_box(sa, g, m0, y, bar);
            load_box(sa + kOperand / 2, g, m0 + 64, y, bar);
            load_box(sb, &maps.x_m, n0, y, bar);
            load_box(sb + kOperand / 2, &maps.x_m, n0 + 64, y, bar);
          }
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
        if (*abort) break;
      }
      // No stage is left with the pair's barriers still to be told of it.
      for (int k = 0; k < kStages && !*abort; ++k) {
        wait_for(smem_u32(&s_empty[stage]), phase ^ 1, abort, a.limit_ns);
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (Walk walk(a, pair); walk.more();) {
        const Job& j = a.job[walk.job];
        int k0, k1;
        walk.next_steps(k0, k1);
        const bool ak = j.mode != kGradW, bk = j.mode <= kGrad;   // K along the rows of A, B
        const uint32_t idesc = (1u << 4) | ((uint32_t)a.is_bf16 << 7) | ((uint32_t)a.is_bf16 << 10) | (ak ? 0u : 1u << 15) |
                               (bk ? 0u : 1u << 16) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
        // 16 of K further: 32 bytes along the rows, two groups of eight rows across.
        const uint32_t step_a = (ak ? 32 : 2048) >> 4, step_b = (bk ? 32 : 2048) >> 4;
        for (int k = k0; k < k1;) {
          if (!wait_for(smem_u32(&s_acc_empty[buf]), acc_phase ^ 1, abort, a.limit_ns)) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * kTile;
          const int first = k, end = min(k + j.segment, k1);
          for (; k < end; ++k) {
            if (!wait_for(smem_u32(&s_full[stage]), phase, abort, a.limit_ns)) break;
            tc_fence_after();
            const uint32_t sa = stages + stage * 2 * kOperand;
            const uint64_t da = operand_desc(sa, ak), db = operand_desc(sa + kOperand, bk);
#pragma unroll
            for (int q = 0; q < kStep / 16; ++q) pair_mma(d, da + q * step_a, db + q * step_b, idesc, k > first || q > 0);
            pair_commit(smem_u32(&s_empty[stage]));
            if (++stage == kStages) stage = 0, phase ^= 1;
          }
          if (*abort) break;
          pair_commit(smem_u32(&s_acc_full[buf]));
          if (++buf == 2) buf = 0, acc_phase ^= 1;
        }
        if (*abort) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsMany));
    const int quarter = warp % 4, half = (warp - 4) / 4;
    int buf = 0;
    uint32_t phase = 0;
    float* turn = reinterpret_cast<float*>(raw + (stages - smem_u32(raw)) + (size_t)kStages * 2 * kOperand) + (warp - 4) * kTurn;
    const int own_row = rank * kHalf + quarter * 32 + lane;
    const float largest = a.lse ? *a.largest : 1.f;
    Walk walk(a, pair);
    bool more = walk.more();
    int job = walk.job;
    Tile x{};
    RowLoads ahead;
    if (more) {
      x = walk.next();
      ahead = load_row(a, a.job[job], x.m * kTile + own_row);
    }
    while (more) {
      const Job& j = a.job[job];
      const int row = x.m * kTile + own_row;
      const int col = x.n * kTile + half * kHalf;
      const RowIn in = row_in(a, j.mode, ahead, largest);
      const Tile now = x;
      auto ready = [&] {
        const bool ok = __all_sync(0xffffffffu, wait_for(smem_u32(&s_acc_full[buf]), phase, abort, a.limit_ns));
        tc_fence_after();
        return ok;
      };
      auto source = [&] { return tmem + ((uint32_t)(quarter * 32) << 16) + buf * kTile + half * kHalf; };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(in_cta(smem_u32(&s_acc_empty[buf]), 0));
        if (++buf == 2) buf = 0, phase ^= 1;
      };
      auto look_ahead = [&] {
        more = walk.more();
        job = walk.job;
        if (more) {
          x = walk.next();
          ahead = load_row(a, a.job[job], x.m * kTile + own_row);
        }
      };
      if (now.k1 - now.k0 <= j.segment && now.k1 > now.k0) {
        if (!ready()) break;
        look_ahead();
        finish_tile(a, j, now, in, row, col, half, turn, FromTmem{source()});
        release();
        continue;
      }
      float acc[kHalf];      // zeros for a slice without classes
#pragma unroll
      for (int k = 0; k < kHalf; ++k) acc[k] = 0.f;
      bool ok = true;
      for (int k = now.k0; k < now.k1; k += j.segment) {
        ok = ready();
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          FromTmem{source()}.get(c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[32 * c + e] += v[e];
        }
        release();
      }
      if (!ok) break;
      look_ahead();
      finish_tile(a, j, now, in, row, col, half, turn, FromSums{acc});
      __syncwarp();
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // A forward launch says so either way, a backward one into cleared words.
    if (s_abort || a.lse == nullptr) a.gave_up[blockIdx.x] = s_abort;
    if (s_abort) {
      if (a.status) atomicOr(a.status, kStatusGaveUp);
      // Copies and products in flight end long before this.
      const uint64_t t0 = global_ns();
      for (uint32_t it = 0; it < (1u << 28) && global_ns() - t0 < 100000000ull; ++it) __nanosleep(1000);
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

// ---- the rows' losses from the tiles' statistics -----------------------------------
// Dot product of two rows by a warp, as the sum x + y of two floats, in some 45 bits (the
// products are exact, the sums' roundings are kept): where a target is nearly certain
// its entry of G is the difference of two nearly equal numbers.  Every lane has it.
struct Sum2 {
  float x = 0.f, y = 0.f;
  __device__ __forceinline__ void add(float p) {
    const float t = __fadd_rn(x, p), b = __fsub_rn(t, x);
    y = __fadd_rn(y, __fadd_rn(__fsub_rn(x, __fsub_rn(t, b)), __fsub_rn(p, b)));
    x = t;
  }
};
template <typename T>
__device__ __forceinline__ Sum2 row_dot(const T* x, const T* w, int cols, bool vec, int lane) {
  Sum2 s;
  if (vec) {
    for (int j = lane * 8; j < cols; j += 256) {
      float a[8], b[8];
      to_floats(*reinterpret_cast<const Pack<T, 8>*>(x + j), a);
      to_floats(*reinterpret_cast<const Pack<T, 8>*>(w + j), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) s.add(__fmul_rn(a[e], b[e]));
    }
  } else {
#pragma unroll 8
    for (int j = lane; j < cols; j += 32) s.add(__fmul_rn(to_f(x[j]), to_f(w[j])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, s.y, o);
    s.add(__shfl_xor_sync(0xffffffffu, s.x, o));
    s.y = __fadd_rn(s.y, y);
  }
  // Infinities and NaN leave NaN as their rounding errors.
  if (!(fabsf(s.x) <= 3.4028235e38f)) s.y = 0.f;
  return Sum2{s.x, s.y};
}
__device__ __forceinline__ Sum2 row_dot(const uint16_t* x, const uint16_t* w, int cols, bool vec, bool bf16, int lane) {
  return bf16 ? row_dot(reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(w), cols, vec, lane)
              : row_dot(reinterpret_cast<const __half*>(x), reinterpret_cast<const __half*>(w), cols, vec, lane);
}

// Rows of x and of W, as the caller gave them.
struct Rows {
  const uint16_t *x, *w;
  int64_t x_stride, w_stride;
  int cols, classes, bf16, vec;
};

// A block has eight rows: 64 threads for the tiles' statistics of each, and a warp for
// its target's logit.
constexpr int kRowsOfBlock = 8;
__global__ void __launch_bounds__(512) k_linear_ce_rows(const float2* part, int parts, const int* gave_up, int ctas, const Rows q,
                                                        int64_t rows, const void* target, int index_type,
                                                        const float* row_weight, float* loss, float* lse, int32_t* status) {
  __shared__ float2 red[16][kRowsOfBlock];
  __shared__ float2 s_hit[kRowsOfBlock];
  __shared__ int s_bad;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int64_t first = (int64_t)blockIdx.x * kRowsOfBlock;
  if (threadIdx.x == 0) s_bad = 0;
  wait_for_previous();
  __syncthreads();
  if (threadIdx.x < ctas && gave_up[threadIdx.x]) s_bad = 1;
  float m = -INFINITY, s = 0.f;
  auto join = [&](float2 p) {
    const float top = fmaxf(m, p.x), base = top == -INFINITY ? 0.f : top;
    s = s * exp2_fast((m - base) * kLog2e) + p.y * exp2_fast((p.x - base) * kLog2e);
    m = top;
  };
  const int64_t row = first + lane % 8;
  if (row < rows) {
    constexpr int U = 8;      // 512 tiles' halves in one go
    for (int k0 = threadIdx.x / 8; k0 < parts; k0 += 64 * U) {
      float2 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = k0 + 64 * u < parts ? part[(int64_t)(k0 + 64 * u) * rows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) join(p[u]);
    }
  }
  if (w < kRowsOfBlock && first + w < rows) {
    const int64_t at = first + w, t = load_index(target, at, index_type);
    Sum2 z{-INFINITY, 0.f};
    if (t >= 0 && t < q.classes) z = row_dot(q.x + at * q.x_stride, q.w + t * q.w_stride, q.cols, q.vec, q.bf16, lane);
    if (lane == 0) s_hit[w] = make_float2(z.x, z.y);
  }
#pragma unroll
  for (int o = 8; o < 32; o *= 2)
    join(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
  if (lane < 8) red[w][lane] = make_float2(m, s);
  __syncthreads();
  if (w) return;
  m = -INFINITY, s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) join(red[lane / 8 * 4 + k][lane % 8]);
#pragma unroll
  for (int o = 8; o < 32; o *= 2)
    join(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
  if (lane >= 8 || row >= rows) return;
  const float2 hit = s_hit[lane];
  const int64_t t = load_index(target, row, index_type);
  // The loss is log(1 + sum over the others of e^(z - target)): exact also where the
  // target is nearly certain.
  float l = 0.f;
  const float weight = row_weight ? row_weight[row] : 1.f;
  if (t >= 0 && t < q.classes && weight != 0.f) {
    const float d = (m - hit.x) - hit.y;
    l = weight * (hit.x == INFINITY ? NAN : d <= 0.f ? log1pf(s * expf(d)) : d + logf(s + expf(-d)));
  }
  // A target of -inf adds nothing, one of NaN makes the sum NaN.
  if (t >= 0 && t < q.classes) join(make_float2(hit.x, 1.f));
  const float all = m == -INFINITY && s == 0.f ? -INFINITY : m + logf(s);
  if (t >= q.classes && status) atomicOr(status, kStatusIndex);
  loss[row] = s_bad ? NAN : l;
  lse[row] = s_bad ? NAN : all;
}

// ---- before and after the backward products ------------------------------------------
// What k_linear_ce_start and the atomics do, by one block, for few rows: a launch less.
__device__ __forceinline__ void start_few(int64_t rows, const void* target, int index_type, int classes, const float* row_weight,
                                          float* largest, int* gave_up) {
  __shared__ float red[8];
  gave_up[threadIdx.x] = 0;      // as many words as threads
  float most = 0.f;
  for (int64_t r = threadIdx.x; r < rows; r += 256) {
    const int64_t t = load_index(target, r, index_type);
    const float w = row_weight ? row_weight[r] : 1.f;
    if (t >= 0 && t < classes && isfinite(w)) most = fmaxf(most, fabsf(w));
  }
  most = warp_max(most);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 8; ++k) most = fmaxf(most, red[k]);
    *largest = most;
  }
}

// Rows of 16-bit elements to rows that TMA can read.  With targets, rows that
// do not count become zeros, whatever they hold, the largest weight is found and
// the targets' entries of G (without weight) are made.
__global__ void __launch_bounds__(256) k_linear_ce_copy(const uint16_t* x, int64_t stride, int64_t rows, int cols, uint16_t* out,
                                                        int64_t out_stride, const void* target, int index_type,
                                                        const Rows q, const float* row_weight, const float* lse,
                                                        float* largest, float* hit, unsigned* slot, int* gave_up, int32_t* status) {
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  wait_for_previous();
  if (gave_up && blockIdx.x == 0) start_few(rows, target, index_type, q.classes, row_weight, largest, gave_up);
  if (row >= rows) return;
  bool live = true;
  if (target) {
    const int64_t t = load_index(target, row, index_type);
    const float w = row_weight ? row_weight[row] : 1.f;
    live = t >= 0 && t < q.classes && w != 0.f;
    Sum2 z;
    if (live) z = row_dot(x + row * stride, q.w + t * q.w_stride, cols, q.vec, q.bf16, lane);
    if (lane == 0) {
      if (live) hit[row] = expm1f((z.x - lse[row]) + z.y);
      if (t >= q.classes && status) atomicOr(status, kStatusIndex);
      // Floats above 0 are in the order of their bits.
      if (!gave_up && live && isfinite(w)) atomicMax(reinterpret_cast<int*>(largest), __float_as_int(fabsf(w)));
      // A class's slot is its first row: a look at it spares a common class's many atomics.
      if (slot && live && (unsigned)row < *reinterpret_cast<volatile unsigned*>(slot + t)) atomicMin(slot + t, (unsigned)row);
    }
  }
  const uint16_t* p = x + row * stride;
  uint16_t* to = out + row * out_stride;
  if (cols % 8 == 0 && stride % 8 == 0 && (uintptr_t)x % 16 == 0) {
    for (int j = lane * 8; j < cols; j += 256)
      *reinterpret_cast<uint4*>(to + j) = live ? *reinterpret_cast<const uint4*>(p + j) : make_uint4(0, 0, 0, 0);
  } else {
    // Eight elements at a time from 4-byte words, shifted where the row starts between
    // two; words that reach past either end of the row are read in halves.
    const bool odd = reinterpret_cast<uintptr_t>(p) & 2;
#pragma unroll 2
    for (int j = lane * 8; j < cols; j += 256) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (live && (j + 8 > cols || (odd && (j == 0 || j + 9 > cols)))) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (j + e < cols) w[e / 2] |= (uint32_t)p[j + e] << (16 * (e % 2));
      } else if (live) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + j - odd);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = q[e];
        if (odd) {
          const uint32_t last = q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], e < 3 ? w[e + 1] : last, 16);
        }
      }
      *reinterpret_cast<uint4*>(to + j) = make_uint4(w[0], w[1], w[2], w[3]);      // the rows' ends are padded to 8
    }
  }
}

__global__ void __launch_bounds__(kMaxCtas) k_linear_ce_start(float* largest, int* gave_up, unsigned* slot, int classes) {
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *largest = 0.f;
    gave_up[threadIdx.x] = 0;
  }
  if (!slot) return;
  for (int v = blockIdx.x * kMaxCtas + threadIdx.x; v < classes; v += gridDim.x * kMaxCtas) slot[v] = 0xffffffffu;
}

// The targets' terms of grad_w's sum, fp32: row_weight * hit * x (x with zeros in
// the rows that do not count), and the slot that each belongs to.
template <typename T>
__global__ void __launch_bounds__(256) k_linear_ce_share(const T* x, int64_t stride, int64_t rows, int cols, const float* hit,
                                                         const void* target, int index_type, int classes,
                                                         const float* row_weight, float* out, const int* slot, int* to) {
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  wait_for_previous();
  if (row >= rows) return;
  const int64_t t = load_index(target, row, index_type);
  const float w = row_weight ? row_weight[row] : 1.f;
  const bool live = t >= 0 && t < classes && w != 0.f;
  const float c = live ? hit[row] * w : 0.f;
  if (slot && threadIdx.x % 32 == 0) to[row] = live ? slot[t] : -1;
  const T* p = x + row * stride;
  float* q = out + row * stride;
  for (int j = threadIdx.x % 32 * 8; j < cols; j += 256) {     // whole rows of 8: the stride is a multiple
    float v[8];
    to_floats(*reinterpret_cast<const Pack<T, 8>*>(p + j), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= c;
    *reinterpret_cast<float4*>(q + j) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(q + j + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void fetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// grad_x from the sums of its slices, in order.
template <typename T>
__global__ void __launch_bounds__(256) k_linear_ce_grad_x(const float* dx, int64_t dx_stride, int64_t slice, int slices,
                                                          int64_t rows, int cols, const float* largest, const void* target,
                                                          int index_type, int classes, const float* row_weight,
                                                          const float* hit, int split, const T* weight, int64_t weight_stride,
                                                          const int* gave_up, int ctas, T* out, int64_t out_stride) {
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  // What the kernel before does not write (and those before that one, for which it has
  // waited, have) is read ahead of its end.
  const int64_t row = (int64_t)blockIdx.x;
  const int64_t t = load_index(target, row, index_type);
  const float w = row_weight ? row_weight[row] : 1.f;
  const bool live = t >= 0 && t < classes && w != 0.f;
  const float f1 = 1.f / 32768.f, f2 = *largest;
  const float* p = dx + row * dx_stride;
  T* q = out + row * out_stride;
  const T* wt = hit && live ? weight + t * weight_stride : nullptr;
  // The target's entry of G, or what its rounding left out.
  float share = 0.f;
  if (wt && split) {
    share = hit[row] * w;
  } else if (wt) {
    const float entry = hit[row] * (w / f2 * 32768.f);
    share = (entry - to_f(from_f<T>(entry))) * f1 * f2;
  }
  const bool vec = cols % 4 == 0 && out_stride % 4 == 0 && (uintptr_t)out % (4 * sizeof(T)) == 0 &&
                   (!hit || (weight_stride % 4 == 0 && (uintptr_t)weight % (4 * sizeof(T)) == 0));
  if (wt && vec && (blockIdx.y * 256 + threadIdx.x) * 4 < cols) fetch_line(wt + (blockIdx.y * 256 + threadIdx.x) * 4);
  wait_for_previous();
  __syncthreads();
  if (threadIdx.x < ctas && gave_up[threadIdx.x]) s_bad = 1;
  __syncthreads();
  if (vec) {
    for (int j = (blockIdx.y * 256 + threadIdx.x) * 4; j < cols; j += 1024 * gridDim.y) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (live) {
        constexpr int U = 8;      // slices whose loads are on their way together
        for (int s = 0; s < slices; s += U) {
          float4 x[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            x[u] = s + u < slices ? *reinterpret_cast<const float4*>(p + (s + u) * slice + j) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < U; ++u) v[0] += x[u].x, v[1] += x[u].y, v[2] += x[u].z, v[3] += x[u].w;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = s_bad ? NAN : v[e] * f1 * f2;
      if (wt) {
        float w4[4];
        to_floats(*reinterpret_cast<const Pack<T, 4>*>(wt + j), w4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(share, w4[e], v[e]);
      }
      *reinterpret_cast<Pack<T, 4>*>(q + j) = from_floats<T, 4>(v);
    }
  } else {
    for (int j = blockIdx.y * 256 + threadIdx.x; j < cols; j += 256 * gridDim.y) {
      float v = 0.f;
      if (live)
        for (int s = 0; s < slices; ++s) v += p[s * slice + j];
      v = s_bad ? NAN : v * f1 * f2;
      q[j] = from_f<T>(wt ? fmaf(share, to_f(wt[j]), v) : v);
    }
  }
}

// ---- host ----------------------------------------------------------------------
constexpr int64_t kMaxTokens = (int64_t)1 << 22, kMaxClasses = (int64_t)1 << 22, kMaxWidth = (int64_t)1 << 16;
constexpr int64_t kLossRows = 32768;               // most rows of a forward launch
constexpr int64_t kPartBytes = (int64_t)256 << 20;    // of its statistics
constexpr int kPairs = 76;                         // of a GB300: what a split of the classes counts on
// Of one G (8,192 x 2048 x 50,304 backward: 4.81 ms with 128 MB, 4.65 with 256, 4.56 with 512).
constexpr int64_t kChunkBytes = (int64_t)256 << 20;
constexpr int kMaxSplits = 64;
constexpr int64_t kFewRows = 4096;                 // rows whose weights one block looks through: some 2 us, as a launch
// More tokens: the targets' entries stay out of the G of a 32-bit grad_w.  That costs some 25
// us of small kernels, and saves grad_w's short segments and in bfloat16 G's third part (768 x 20,000,
// us in G / apart: bfloat16 64 tokens 67 / 87, 200 97 / 98, 400 126 / 109, 800 181 / 147;
// float16 200 85 / 98, 400 106 / 109, 800 147 / 148; grad_w is 5e-7 / 4e-7 off).
constexpr int64_t kSplitRows = 256;
// A 16-bit grad_w is made from two parts of G, or from one without the targets' entries:
// from one with them a bfloat16 gradient would be 2.0e-3 off, 1.66e-3 of which is its own
// rounding.  Two parts cost products, the other form some 30 us of small kernels (us, two
// parts / apart, bfloat16 in all: 5,003 x 256 of 1,000 tokens 51 / 60, 2,000 70 / 68, 4,096
// 111 / 99; 20,000 x 768 of 300 78 / 93, 600 100 / 104, 1,000 134 / 120; 50,304 x 2048 of 300
// 283 / 328, 600 392 / 382, 1,000 555 / 455; with one part and the targets in it 5,003 x 256
// of 1,000 43, 20,000 x 768 of 1,000 95).
constexpr int64_t kSplitRows16 = 512, kSplitRowsAlways = 2048, kSplitProducts = (int64_t)1 << 33;
// Up to so many tokens grad_x is made from two parts of G; with more from one, and what its
// rounding leaves out of the targets' entries, the large ones, is added at the end: as exact
// where the others are small beside them (grad_x alone of 64 tokens, 20,000 x 768: 41 us,
// 43 with two parts, 39 with neither).
constexpr int64_t kExactRows = 16;
// Steps of a segment: logits whose losses are fp32, a 32-bit grad_w without and with
// the targets' entries; products that end in 16 bits.  Terms of one sign lose some 4e-7 of
// the sum a step (1.05M tokens in one segment 6e-3, more than either type's half step), in
// float16 three times what they do in bfloat16, whose logits and 32-bit sums therefore
// take segments half as long (2048 wide, logits of 20 from terms of one sign: losses
// 3.3e-5 off with 32 steps, 1.6e-5 with 16, 7e-6 with 8; bfloat16 9e-6 with 32; 8,192 x 2048 x
// 50,304 float16 forward 1.10, 1.14, 1.19 ms).
constexpr int kLossSegment = 32, kGradSegment = 32, kGradWSegment = 4, kSplitSegment = 64, kLongSegment = 128;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Rows that TMA reads in place.
bool tma_rows(const Span& s) {
  return s.lo() % 16 == 0 && (s.rows == 1 || (s.stride * 2 % 16 == 0 && s.stride >= s.cols && s.stride < (int64_t)1 << 38));
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder() {
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled fn = known.load(std::memory_order_relaxed);
  if (fn) return fn;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  fn = reinterpret_cast<EncodeTiled>(p);
  known.store(fn, std::memory_order_relaxed);
  return fn;
}

// A matrix of 16-bit elements, read in boxes of 64 columns and `box` rows.
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t stride, int box, bool bf16) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  if (rows == 1) stride = up(cols, 8);
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t boxes[2] = {kStep, (cuuint32_t)box}, steps[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), dims,
            strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs that run at once on this device.
int pair_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  int n = known[dev & 63].load(std::memory_order_relaxed);
  if (n) return n;
  allow_smem(reinterpret_cast<const void*>(&k_linear_ce), kSmem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k_linear_ce, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = sm_count() / 2;
  }
  n = std::min(std::max(n, 1), kMaxPairs);
  known[dev & 63].store(n, std::memory_order_relaxed);
  return n;
}

// Spreads a job's tiles, each of `cost`, over the pairs such that with the loads
// that they have all end together as nearly as whole tiles allow.
void spread_tiles(Spread& s, int tiles, double cost, int pairs, double* load) {
  // The level up to which the tiles fill those pairs that are below it.
  double level = 0.0;
  for (int n = pairs, before = 0; n != before;) {
    double sum = tiles * cost;
    before = n;
    for (int p = 0; p < pairs; ++p) sum += before == pairs || load[p] < level ? load[p] : 0.0;
    level = sum / n;
    n = 0;
    for (int p = 0; p < pairs; ++p) n += load[p] < level;
  }
  int left = tiles;
  for (int p = 0; p < pairs; ++p) {
    s.count[p] = load[p] < level ? std::min(left, (int)((level - load[p]) / cost)) : 0;
    left -= s.count[p];
    load[p] += s.count[p] * cost;
  }
  int order[kMaxPairs];
  for (int p = 0; p < pairs; ++p) order[p] = p;
  // What whole tiles leave over, one each to those with the least.
  std::sort(order, order + pairs, [&](int x, int y) { return load[x] != load[y] ? load[x] < load[y] : x < y; });
  for (int k = 0; left > 0; --left, k = (k + 1) % pairs) {
    ++s.count[order[k]];
    load[order[k]] += cost;
  }
  auto kinds = [&] {
    int n = 0;
    for (int k = 0; k < pairs; ++k) n += k == 0 || s.count[order[k]] != s.count[order[k - 1]];
    return n;
  };
  std::sort(order, order + pairs, [&](int x, int y) { return s.count[x] != s.count[y] ? s.count[x] > s.count[y] : x < y; });
  if (kinds() > kGroups) {     // then evenly, whatever the loads are
    for (int p = 0; p < pairs; ++p) order[p] = p, s.count[p] = tiles / pairs + (p < tiles % pairs);
  }
  s.groups = 0;
  s.pairs = pairs;
  for (int k = 0; k < pairs; ++k) {
    s.place[order[k]] = (uint8_t)k;
    const int takes = s.count[order[k]];
    if (s.groups && s.takes[s.groups - 1] == takes) {
      ++s.size[s.groups - 1];
    } else {
      s.takes[s.groups] = takes;
      s.size[s.groups++] = 1;
    }
  }
}

// Steps of K that a tile costs, with its epilogue: G's takes as long as some 20, and
// only the next tile's product runs beside it.
double tile_cost(const Job& j) {
  const double steps = (double)j.k_steps / j.splits;
  return j.mode == kGrad ? std::max(steps + 2.0, 20.0) : steps + 4.0;
}

cudaError_t launch_tiles(const Maps& maps, Args& a, int pairs, cudaStream_t s) {
  int tiles = 0;
  for (int k = 0; k < a.jobs; ++k) tiles += a.job[k].tiles;
  pairs = std::min(pairs, tiles);
  double load[kMaxPairs] = {};
  for (int k = 0; k < a.jobs; ++k) {
    Job& j = a.job[k];
    spread_tiles(a.spread[k], j.tiles, tile_cost(j), pairs, load);
    j.by_group = FastDiv(kRowGroup * j.n_tiles), j.by_rows = FastDiv(kRowGroup), j.by_n = FastDiv(j.n_tiles);
    j.by_last = FastDiv(j.m_tiles % kRowGroup ? j.m_tiles % kRowGroup : kRowGroup), j.by_splits = FastDiv(j.splits);
  }
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(&k_linear_ce), kSmem);
  if (e != cudaSuccess) return e;
  // The kernel's warps wait for registers that only a launch with kRegs has.
  static std::atomic<bool> right{false};
  if (!right.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, reinterpret_cast<const void*>(&k_linear_ce))) != cudaSuccess) return e;
    if (at.numRegs != kRegs) return cudaErrorInvalidKernelImage;
    right.store(true, std::memory_order_relaxed);
  }
  return launch(k_linear_ce, dim3(2 * (unsigned)pairs), dim3(kThreads), kSmem, s, true, 1, maps, a);
}

// Where things are in the workspace, in bytes from its start.
struct Plan {
  int64_t x = 0, w = 0, part = 0, g = 0, g_plane = 0, dx = 0, flags = 0, largest = 0, size = 0;
  int64_t hit = 0, share = 0, table = 0, slot = 0, to = 0, sort = 0, sort_bytes = 0;
  int64_t x_stride, w_stride, chunk = 0, dx_stride = 0, slice = 0;
  int splits = 1, buffers = 1;
};

int64_t take(Plan& p, int64_t bytes) {
  const int64_t at = p.size;
  p.size += up(bytes, 1024);
  return at;
}

// copy: also room for rows that TMA cannot read.
Plan plan_loss(int64_t rows, int64_t classes, int64_t cols, bool copy) {
  Plan p;
  p.x_stride = p.w_stride = up(cols, 8);
  const int64_t parts = 2 * up(classes, kTile) / kTile;
  p.chunk = std::min(rows, std::min(kLossRows, std::max<int64_t>(kPartBytes / (parts * 8) / kTile, 1) * kTile));
  p.flags = take(p, kMaxCtas * 4);
  p.part = take(p, parts * p.chunk * 8);
  if (copy) {
    p.x = take(p, rows * p.x_stride * 2);
    p.w = take(p, classes * p.w_stride * 2);
  }
  return p;
}

// How a backward call holds G, for a grad_w of so many bits (0: none is asked for).
struct Parts {
  int planes, planes_x;      // its parts for grad_w, for grad_x
  bool split;                // the targets' entries stay out of it
};
Parts parts_of(int64_t rows, int64_t classes, int64_t cols, int bits, bool bf16) {
  Parts q;
  q.split = bits == 32 ? rows > kSplitRows
                       : bits == 16 && rows > kSplitRows16 && (rows > kSplitRowsAlways || rows * classes * cols > kSplitProducts);
  q.planes_x = rows > kExactRows ? 1 : 2;
  q.planes = bits == 0 ? q.planes_x : q.split ? bits / 16 : bits == 32 && bf16 ? 3 : 2;
  return q;
}

Plan plan_grad(int64_t rows, int64_t classes, int64_t cols, const Parts& q, bool copy) {
  Plan p;
  p.x_stride = p.w_stride = up(cols, 8);
  if (q.split) {
    p.share = take(p, rows * p.x_stride * 4);
    if (q.planes == 1) {      // a 16-bit grad_w
      p.table = take(p, (rows * p.x_stride + kTile) * 4);      // the epilogue reads whole tiles of its rows
      p.slot = take(p, classes * 4);
      p.to = take(p, rows * 4);
      lopt_embed_workspace(rows, rows, p.x_stride, &p.sort_bytes);
    } else {
      lopt_embed_workspace(rows, classes, cols, &p.sort_bytes);
    }
    p.sort = take(p, p.sort_bytes);
  }
  p.flags = take(p, kMaxCtas * 4);
  p.largest = take(p, 4);
  p.hit = take(p, rows * 4);
  p.x = take(p, rows * p.x_stride * 2);
  if (copy) p.w = take(p, classes * p.w_stride * 2);
  const int64_t all = up(classes, kTile);
  p.chunk = std::min(all, std::max<int64_t>(kChunkBytes / (rows * 2 * q.planes) / kTile, 1) * kTile);
  p.buffers = p.chunk < all ? 2 : 1;
  p.g_plane = up(rows * p.chunk * 2, 1024);
  p.g = take(p, p.g_plane * q.planes * p.buffers);
  p.dx_stride = up(cols, 8);
  p.slice = up(rows * p.dx_stride, 256);
  // Few tiles of grad_x: the classes are split over slices, added in order at the end.
  const int64_t tiles = up(rows, kTile) / kTile * (up(cols, kTile) / kTile), steps = p.chunk / kStep;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({kPairs / tiles, steps / 4, kMaxSplits}));
  p.dx = take(p, p.slice * p.splits * 4);
  return p;
}

struct Call {
  const void *x, *w, *target;
  const float* row_weight;
  int type, index_type;
  int64_t rows, classes, cols;
  Span mx, mw;
};

int check_call(const Call& c) {
  if (c.type != LOPT_F16 && c.type != LOPT_BF16) return LOPT_E_ARG;
  if (!index_size(c.index_type)) return LOPT_E_ARG;
  if (c.rows < 0 || c.rows > kMaxTokens || c.classes < 1 || c.classes > kMaxClasses || c.cols < 1 || c.cols > kMaxWidth)
    return LOPT_E_SHAPE;
  int rc;
  if ((rc = check_matrix(c.mw, false))) return rc;
  if (c.rows == 0) return LOPT_OK;
  if ((rc = check_matrix(c.mx, false))) return rc;
  if (!c.target) return LOPT_E_ARG;
  if ((uintptr_t)c.target % index_size(c.index_type) || (uintptr_t)c.row_weight % 4) return LOPT_E_ALIGN;
  return LOPT_OK;
}

// Rows from r0 on.
Rows rows_of(const Call& c, int64_t r0) {
  return Rows{static_cast<const uint16_t*>(c.x) + r0 * c.mx.stride, static_cast<const uint16_t*>(c.w), c.mx.stride, c.mw.stride,
              (int)c.cols, (int)c.classes, c.type == LOPT_BF16,
              c.cols % 8 == 0 && rows_aligned(c.mx, 16) && rows_aligned(c.mw, 16)};
}

int check_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return LOPT_E_ALIAS;
    for (const Span& i : ins)
      if (overlap(*o, i)) return LOPT_E_ALIAS;
  }
  return LOPT_OK;
}

}  // namespace
}  // namespace train
}  // namespace lopt

using namespace lopt::train;

extern "C" {

int lopt_linear_ce_workspace(int64_t rows, int64_t classes, int64_t cols, int aligned, int backward,
                             int grad_weight_type, int64_t* bytes) {
  if (!bytes || (aligned != 0 && aligned != 1) || (backward != 0 && backward != 1) || (backward && !type_size(grad_weight_type))) return LOPT_E_ARG;
  if (rows < 0 || rows > kMaxTokens || classes < 1 || classes > kMaxClasses || cols < 1 || cols > kMaxWidth) return LOPT_E_SHAPE;
  const int64_t n = std::max<int64_t>(rows, 1);
  if (!backward) {
    *bytes = plan_loss(n, classes, cols, !aligned).size;
    return LOPT_OK;
  }
  // x of either type, grad_weight of 16 bits, of 32 where those are asked for, or NULL:
  // fewer parts of G may take more, since chunks are whole tiles of classes.
  *bytes = 0;
  for (bool bf16 : {false, true})
    for (int bits : {0, 16, grad_weight_type == LOPT_F32 ? 32 : 16})
      *bytes = std::max(*bytes, plan_grad(n, classes, cols, parts_of(n, classes, cols, bits, bf16), !aligned).size);
  return LOPT_OK;
}

static int forward(uint64_t limit_ns, const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                   int64_t classes, int64_t weight_stride, const void* target, int index_type, const float* row_weight,
                   float* loss, float* lse, void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  const Call c{x, weight, target, row_weight, type, index_type, rows, classes, cols,
               Span{x, rows, cols, x_stride, 2}, Span{weight, classes, cols, weight_stride, 2}};
  int rc = check_call(c);
  if (rc || rows == 0) return rc;
  const Plan p = plan_loss(rows, classes, cols, !tma_rows(c.mx) || !tma_rows(c.mw));
  if (!loss || !lse || !workspace || workspace_bytes < p.size) return LOPT_E_ARG;
  if ((uintptr_t)loss % 4 || (uintptr_t)lse % 4 || (uintptr_t)status % 4 || (uintptr_t)workspace % 256) return LOPT_E_ALIGN;
  const Span so{loss, 1, rows, rows, 4}, sl{lse, 1, rows, rows, 4}, sw{workspace, 1, p.size, p.size, 1};
  const Span st{target, 1, rows, rows, index_size(index_type)}, sr{row_weight, 1, rows, rows, 4};
  if ((rc = check_alias({so, sl, sw}, {c.mx, c.mw, st, sr}))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  char* ws = static_cast<char*>(workspace);
  const bool bf16 = type == LOPT_BF16;
  cudaError_t e;
  const void *xp = x, *wp = weight;
  int64_t xs = x_stride, wst = weight_stride;
  if (!tma_rows(c.mx)) {
    xp = ws + p.x, xs = p.x_stride;
    e = launch(k_linear_ce_copy, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, true, 1, (const uint16_t*)x, x_stride, rows,
               (int)cols, (uint16_t*)xp, xs, (const void*)nullptr, 0, Rows{}, (const float*)nullptr, (const float*)nullptr, (float*)nullptr, (float*)nullptr, (unsigned*)nullptr, (int*)nullptr, (int32_t*)nullptr);
    if (e != cudaSuccess) return done(e);
  }
  if (!tma_rows(c.mw)) {
    wp = ws + p.w, wst = p.w_stride;
    e = launch(k_linear_ce_copy, dim3((unsigned)((classes + 7) / 8)), dim3(256), 0, s, true, 1, (const uint16_t*)weight, weight_stride,
               classes, (int)cols, (uint16_t*)wp, wst, (const void*)nullptr, 0, Rows{}, (const float*)nullptr, (const float*)nullptr, (float*)nullptr,
               (float*)nullptr, (unsigned*)nullptr, (int*)nullptr, (int32_t*)nullptr);
    if (e != cudaSuccess) return done(e);
  }
  const int pairs = pair_count();
  const int n_tiles = (int)(up(classes, kTile) / kTile);
  for (int64_t r0 = 0; r0 < rows; r0 += p.chunk) {
    const int64_t n = std::min(p.chunk, rows - r0);
    Maps maps{};
    Args a{};
    if (!make_map(&maps.x_k, static_cast<const uint16_t*>(xp) + r0 * xs, n, cols, xs, kHalf, bf16) ||
        !make_map(&maps.w_k, wp, classes, cols, wst, kHalf, bf16))
      return LOPT_E_UNSUPPORTED;
    a.rows = (int)n, a.classes = (int)classes, a.cols = (int)cols, a.is_bf16 = bf16, a.planes = 1, a.limit_ns = limit_ns;
    a.target = static_cast<const char*>(target) + r0 * index_size(index_type), a.index_type = index_type;
    a.part = reinterpret_cast<float2*>(ws + p.part);
    a.gave_up = reinterpret_cast<int*>(ws + p.flags), a.status = status;
    const int m_tiles = (int)(up(n, kTile) / kTile);
    a.jobs = 1;
    a.job[0] = Job{kLoss, m_tiles * n_tiles, m_tiles, n_tiles, 1, (int)(up(cols, kStep) / kStep), 0, 0, (int)classes, 0,
                   bf16 ? kLossSegment : kLossSegment / 2};
    if ((e = launch_tiles(maps, a, pairs, s)) != cudaSuccess) return done(e);
    const float* rw = row_weight ? row_weight + r0 : nullptr;
    e = launch(k_linear_ce_rows, dim3((unsigned)((n + kRowsOfBlock - 1) / kRowsOfBlock)), dim3(512), 0, s, true, 1, (const float2*)a.part, 2 * n_tiles,
               (const int*)a.gave_up, 2 * std::min(pairs, a.job[0].tiles), rows_of(c, r0), n, a.target, index_type, rw, loss + r0, lse + r0, status);
    if (e != cudaSuccess) return done(e);
  }
  return LOPT_OK;
}

int lopt_linear_ce_forward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                           int64_t classes, int64_t weight_stride, const void* target, int index_type,
                           const float* row_weight, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                           int32_t* status, void* stream) {
  return forward(kLimitNs, x, type, rows, cols, x_stride, weight, classes, weight_stride, target, index_type, row_weight, loss, lse,
                 workspace, workspace_bytes, status, stream);
}

int lopt_selftest_linear_ce(int64_t limit_ns, const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride,
                            const void* weight, int64_t classes, int64_t weight_stride, const void* target, int index_type,
                            const float* row_weight, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                            int32_t* status, void* stream) {
  if (limit_ns < 0 || limit_ns > (int64_t)kLimitNs) return LOPT_E_ARG;
  return forward((uint64_t)limit_ns, x, type, rows, cols, x_stride, weight, classes, weight_stride, target, index_type, row_weight,
                 loss, lse, workspace, workspace_bytes, status, stream);
}

int lopt_linear_ce_backward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                            int64_t classes, int64_t weight_stride, const void* target, int index_type,
                            const float* row_weight, const float* lse, void* grad_x, int64_t grad_x_stride,
                            void* grad_weight, int grad_weight_type, int64_t grad_weight_stride, int accumulate,
                            void* workspace, int64_t workspace_bytes, int32_t* status, void* stream) {
  const Call c{x, weight, target, row_weight, type, index_type, rows, classes, cols,
               Span{x, rows, cols, x_stride, 2}, Span{weight, classes, cols, weight_stride, 2}};
  int rc = check_call(c);
  if (rc) return rc;
  if ((accumulate != 0 && accumulate != 1) || (grad_weight && grad_weight_type != LOPT_F32 && grad_weight_type != type) ||
      (accumulate && grad_weight && grad_weight_type != LOPT_F32))
    return LOPT_E_ARG;
  const int gs = grad_weight ? type_size(grad_weight_type) : 4;
  const Span mg{grad_weight, classes, cols, grad_weight_stride, gs};
  if (grad_weight && (rc = check_matrix(mg, true))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    if (!grad_weight || accumulate) return LOPT_OK;
    return done(cudaMemset2DAsync(grad_weight, (classes == 1 ? cols : grad_weight_stride) * gs, 0, cols * gs, classes, s));
  }
  const Span mo{grad_x, rows, cols, grad_x_stride, 2};
  if (grad_x && (rc = check_matrix(mo, true))) return rc;
  if (!grad_x && !grad_weight) return LOPT_OK;
  const bool fp32_weight = grad_weight && grad_weight_type == LOPT_F32;
  const bool bf16 = type == LOPT_BF16;
  const Parts parts = parts_of(rows, classes, cols, !grad_weight ? 0 : fp32_weight ? 32 : 16, bf16);
  const int planes = parts.planes, planes_x = parts.planes_x;
  const bool split = parts.split;
  const int pairs = pair_count();
  const Plan p = plan_grad(rows, classes, cols, parts, !tma_rows(c.mw));
  if (!lse || !workspace || workspace_bytes < p.size) return LOPT_E_ARG;
  if ((uintptr_t)lse % 4 || (uintptr_t)status % 4 || (uintptr_t)workspace % 256) return LOPT_E_ALIGN;
  const Span sl{lse, 1, rows, rows, 4}, sw{workspace, 1, p.size, p.size, 1};
  const Span st{target, 1, rows, rows, index_size(index_type)}, sr{row_weight, 1, rows, rows, 4};
  if ((rc = check_alias({mo, mg, sw}, {c.mx, c.mw, st, sr, sl}))) return rc;
  char* ws = static_cast<char*>(workspace);
  float *largest = reinterpret_cast<float*>(ws + p.largest), *hit = reinterpret_cast<float*>(ws + p.hit);
  cudaError_t e;
  int* flags = reinterpret_cast<int*>(ws + p.flags);
  static_assert(kMaxCtas == 256, "start_few clears a word a thread");
  // The targets' share goes into an fp32 grad_w when that is done, into a 16-bit one, which
  // is rounded once, from a table (300 tokens, 50,304 x 2048, fp32: 338 us, 380 from a table).
  int* slot = split && !fp32_weight ? reinterpret_cast<int*>(ws + p.slot) : nullptr;
  const bool start = rows > kFewRows || slot;
  if (start) {
    e = launch(k_linear_ce_start, dim3(slot ? (unsigned)std::min<int64_t>((classes + kMaxCtas - 1) / kMaxCtas, 304) : 1u), dim3(kMaxCtas), 0, s,
               false, 1, largest, flags, reinterpret_cast<unsigned*>(slot), (int)classes);
    if (e != cudaSuccess) return done(e);
  }
  uint16_t* xp = reinterpret_cast<uint16_t*>(ws + p.x);
  e = launch(k_linear_ce_copy, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, true, 1, (const uint16_t*)x, x_stride, rows,
             (int)cols, xp, p.x_stride, target, index_type, rows_of(c, 0), row_weight, lse, largest, hit, reinterpret_cast<unsigned*>(slot),
             start ? (int*)nullptr : flags, status);
  if (e != cudaSuccess) return done(e);
  const void* wp = weight;
  int64_t wst = weight_stride;
  if (!tma_rows(c.mw)) {
    wp = ws + p.w, wst = p.w_stride;
    e = launch(k_linear_ce_copy, dim3((unsigned)((classes + 7) / 8)), dim3(256), 0, s, true, 1, (const uint16_t*)weight, weight_stride,
               classes, (int)cols, (uint16_t*)wp, wst, (const void*)nullptr, 0, Rows{}, (const float*)nullptr, (const float*)nullptr, (float*)nullptr,
               (float*)nullptr, (unsigned*)nullptr, (int*)nullptr, (int32_t*)nullptr);
    if (e != cudaSuccess) return done(e);
  }
  // The targets' share, summed into the rows of `to` (a class, or its slot).
  auto add_share = [&](int64_t to_rows, int64_t to_cols, const void* to, int to_type, float* out, int64_t out_stride, int add) {
    const dim3 grid((unsigned)((rows + 7) / 8));
    float* share = reinterpret_cast<float*>(ws + p.share);
    int* slots = slot ? reinterpret_cast<int*>(ws + p.to) : nullptr;
    if (bf16)
      e = launch(k_linear_ce_share<__nv_bfloat16>, grid, dim3(256), 0, s, true, 1, (const __nv_bfloat16*)xp, p.x_stride, rows, (int)cols,
                 (const float*)hit, target, index_type, (int)classes, row_weight, share, (const int*)slot, slots);
    else
      e = launch(k_linear_ce_share<__half>, grid, dim3(256), 0, s, true, 1, (const __half*)xp, p.x_stride, rows, (int)cols,
                 (const float*)hit, target, index_type, (int)classes, row_weight, share, (const int*)slot, slots);
    if (e != cudaSuccess) return done(e);
    return embed_backward_to(share, LOPT_F32, p.x_stride, to, to_type, rows, to_rows, to_cols, 1.f, add, out, out_stride,
                             ws + p.sort, p.sort_bytes, status, stream);
  };
  if (slot && (rc = add_share(rows, p.x_stride, ws + p.to, LOPT_I32, reinterpret_cast<float*>(ws + p.table), p.x_stride, 0))) return rc;
  Maps maps{};
  Args a{};
  bool ok = make_map(&maps.x_k, xp, rows, cols, p.x_stride, kHalf, bf16) && make_map(&maps.x_m, xp, rows, cols, p.x_stride, kStep, bf16) &&
            make_map(&maps.w_k, wp, classes, cols, wst, kHalf, bf16) && make_map(&maps.w_m, wp, classes, cols, wst, kStep, bf16);
  for (int b = 0; b < p.buffers; ++b) {
    for (int k = 0; k < planes; ++k) a.g[b][k] = ws + p.g + (b * planes + k) * p.g_plane;
    for (int k = 0; k < planes_x; ++k) ok = ok && make_map(&maps.g_k[b][k], a.g[b][k], rows, p.chunk, p.chunk, kHalf, bf16);
    ok = ok && make_map(&maps.g_m[b][0], a.g[b][0], rows, p.chunk, p.chunk, kStep, bf16);
    for (int k = 1; k < planes; ++k) ok = ok && make_map(&maps.g_m[b][k], a.g[b][k], rows, p.chunk, p.chunk, kStep, bf16);
  }
  if (!ok) return LOPT_E_UNSUPPORTED;
  a.rows = (int)rows, a.classes = (int)classes, a.cols = (int)cols, a.planes = planes, a.planes_x = planes_x, a.is_bf16 = bf16, a.limit_ns = kLimitNs;
  a.target = target, a.index_type = index_type, a.row_weight = row_weight, a.lse = lse;
  a.g_stride = p.chunk, a.largest = largest;
  a.hit = hit, a.split = split;
  if (slot) a.slot = slot, a.table = reinterpret_cast<const float*>(ws + p.table), a.table_stride = p.x_stride;
  a.dx = reinterpret_cast<float*>(ws + p.dx), a.dx_stride = p.dx_stride, a.dx_slice = p.slice;
  a.dw = grad_weight, a.dw_type = grad_weight_type, a.dw_stride = grad_weight_stride, a.accumulate = accumulate;
  a.gave_up = reinterpret_cast<int*>(ws + p.flags), a.status = status;
  const int m_tiles = (int)(up(rows, kTile) / kTile), d_tiles = (int)(up(cols, kTile) / kTile);
  const int64_t chunks = (up(classes, kTile) + p.chunk - 1) / p.chunk;
  auto grad_job = [&](int64_t k) {
    const int64_t v0 = k * p.chunk, v1 = std::min(classes, v0 + p.chunk);
    const int n_tiles = (int)(up(v1 - v0, kTile) / kTile);
    return Job{kGrad, m_tiles * n_tiles, m_tiles, n_tiles, 1, (int)(up(cols, kStep) / kStep), (int)(k % p.buffers), (int)v0, (int)v1, 0,
               bf16 ? kGradSegment : kGradSegment / 2};
  };
  // Launch k makes chunk k's G beside the products of chunk k - 1: the long
  // tiles first, the short ones of G fill the last round.
  for (int64_t k = 0; k <= chunks; ++k) {
    a.jobs = 0;
    auto add = [&](const Job& j) { a.job[a.jobs++] = j; };
    if (k > 0) {
      Job g = grad_job(k - 1);
      if (grad_weight)
        add(Job{kGradW, g.n_tiles * d_tiles, g.n_tiles, d_tiles, 1, (int)(up(rows, kStep) / kStep) * planes, g.buffer, g.v0, g.v1, 0,
                !fp32_weight ? kLongSegment : !split ? kGradWSegment : bf16 ? kSplitSegment : kSplitSegment / 2});
      if (grad_x)
        add(Job{kGradX, m_tiles * d_tiles * p.splits, m_tiles, d_tiles, p.splits, (int)(up(g.v1 - g.v0, kStep) / kStep) * planes_x, g.buffer,
                g.v0, g.v1, k > 1, kLongSegment});
    }
    // The costliest first: the others even out what they leave.
    if (a.jobs == 2 && tile_cost(a.job[1]) > tile_cost(a.job[0])) std::swap(a.job[0], a.job[1]);
    if (k < chunks) add(grad_job(k));
    if ((e = launch_tiles(maps, a, pairs, s)) != cudaSuccess) return done(e);
  }
  if (split && fp32_weight &&
      (rc = add_share(classes, cols, target, index_type, static_cast<float*>(grad_weight), classes == 1 ? cols : grad_weight_stride, 1)))
    return rc;
  if (!grad_x) return LOPT_OK;
  const dim3 grid((unsigned)rows, (unsigned)((cols + 1023) / 1024));
  const int ctas = kMaxCtas;
  if (bf16)
    e = launch(k_linear_ce_grad_x<__nv_bfloat16>, grid, dim3(256), 0, s, true, 1, (const float*)a.dx, p.dx_stride, p.slice, p.splits,
               rows, (int)cols, (const float*)largest, target, index_type, (int)classes, row_weight, (const float*)(planes_x == 1 ? hit : nullptr), (int)split, (const __nv_bfloat16*)wp, wst,
               (const int*)a.gave_up, ctas, (__nv_bfloat16*)grad_x, grad_x_stride);
  else
    e = launch(k_linear_ce_grad_x<__half>, grid, dim3(256), 0, s, true, 1, (const float*)a.dx, p.dx_stride, p.slice, p.splits, rows,
               (int)cols, (const float*)largest, target, index_type, (int)classes, row_weight, (const float*)(planes_x == 1 ? hit : nullptr), (int)split, (const __half*)wp, wst,
               (const int*)a.gave_up, ctas, (__half*)grad_x, grad_x_stride);
  return done(e);
}

}  // extern "C"
