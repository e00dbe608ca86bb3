// What the products grouped by expert share: tile variants, loads, MMAs and the ring of operand stages
// (tcgen05 + TMEM + TMA), the walk over an expert's tiles, copies of operands whose rows do not start
// on 16 bytes, tensor maps and launches.  How the pieces work together stands in grouped_mm.cu.
#pragma once

#include <atomic>

#include <cudaTypedefs.h>

#include "device_common.cuh"
#include "element.cuh"
#include "kernels.h"
#include "row_blocks.h"

namespace muon {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kBM = 128;            // rows of operand A: M of the MMA
constexpr int kABytes = kBM * 128;  // 16 KB
constexpr int kBox = 64 * 128;      // an MN-major box: 64 k-rows of 128 bytes
constexpr int kTmemCols = 512;
constexpr int kAccCols = 256;       // TMEM columns of one accumulator, of two
constexpr int kMaxStages = 6;
constexpr long long kWaitBudget = 4000000000LL;  // ~2 s of SM clock per wait

// mm tile variants: kMaxN rows of one expert per tile at most, on single CTAs or pairs.
// Narrow: smaller stages leave room for more of the weight in flight, for experts with few
// rows, whose product is bound by streaming it, and stages of two k-blocks under one pair of
// barriers: a wait, an elected lane and a commit cost the issuing warps 250-400 cycles, more than
// the loads or MMAs of one narrow k-block (one token 12.5 -> 9.2 us).  Where the MMAs take 500
// cycles a k-block, the finer stages are ahead (Pair: 328 against 335 us on 98304 x 1408 -> 2048).
// kSegment16, kSegment32: most k-blocks per segment of a sum that is stored in 16 or 32 bits.  The
// MMAs wait where a segment ends before the last tile's stores have left the epilogue free: pairs,
// which multiply fastest, pay for short segments (24570 rows, 2048 -> 1408, 16-bit: 111 us with
// 11, 118 with 8; weight gradient of 98304 rows, 64 x 2048 x 1408: 403 us with 12, 422 with 8, 452
// with 6, 523 with 4), the others little (weight gradient of 24576 rows: 188 us with 12, 192 with
// 4; all of these while accumulators were handed back with a release, 411 with 6 since).  With kSegment32 the
// error is a plain fp32 product's or at most a rounding (2^-24) more.
struct Pair {
  static constexpr bool kPair = true, kSplit = false;
  static constexpr int kMaxN = 256, kBoxRows = 64, kStages = 6, kSub = 1;
  static constexpr int kSegment16 = 11, kSegment32 = 6;
};
struct Wide {
  static constexpr bool kPair = false, kSplit = false;
  static constexpr int kMaxN = 256, kBoxRows = 64, kStages = 4, kSub = 1;
  static constexpr int kSegment16 = 8, kSegment32 = 4;
};
struct Narrow {
  static constexpr bool kPair = false, kSplit = false;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 4, kSub = 2;
  static constexpr int kSegment16 = 8, kSegment32 = 4;
};
// Split: a cluster of CTAs shares one tile, each taking a part of k; then all of them add up
// shares of the tile, the parts in order, out of each other's shared memory.  For products of so
// few tiles that most SMs would have none: a k-block costs a CTA 0.2 us whatever the tile's
// width (the MMA reads 128 rows of the weight).
struct Split {
  static constexpr bool kPair = false, kSplit = true;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 4, kSub = 2;
  static constexpr int kSegment16 = 8, kSegment32 = 4;
};
// The same for weight gradients of few tiles and many rows: the CTAs share the rows.
struct SplitWide {
  static constexpr bool kPair = false, kSplit = true;
  static constexpr int kMaxN = 256, kStages = 4, kSub = 1, kSegment32 = 4;
};
constexpr int kMostParts = 8;  // portable cluster size

// What follows from a variant (wgrad uses Pair, Wide and SplitWide).
template <typename V>
struct Shape {
  static constexpr int kCtas = V::kPair ? 2 : 1;
  static constexpr int kM = kBM * kCtas;                   // M of the MMA
  [[maybe_unused]] static constexpr int kStepN = 16 * kCtas;  // N goes in steps of this (mm)
  static constexpr int kBlock = kABytes + V::kMaxN / kCtas * 128;  // bytes of a k-block
  static constexpr int kStage = kBlock * V::kSub;
  static constexpr int kBlocks = (V::kMaxN + 63) / 64;     // 32-column blocks per epilogue warp
};

// Barriers and flags of one CTA.
struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  // wgrad on pairs, last stage of a tile: the second CTA's own operands have landed, and it
  // has zeroed the rows that are not its expert's.
  uint64_t tail[kMaxStages], fixed[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
};

// Loads of one box to shared address dst, signalling the barrier at `bar`: of this CTA
// (kPair false), or of either CTA of the pair (a shared::cluster address).
template <bool kPair>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool kPair>
__device__ __forceinline__ void load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                        uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Arrives on an own barrier (given by its shared address), which then expects `bytes`.
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// Operand descriptors as two words (see smem_desc_sw128): the low one moves with the address.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (saddr & 0x3FFFF) >> 4 | (lbo >> 4) << 16;
}

// kind::f16 products of 16-bit operands; kFp8: kind::f8f6f4 of 8-bit ones.
#define MUON_MMA(group, kind)                                                                      \
  asm volatile(                                                                                    \
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"                                                 \
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"                \
      "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], a, b, %3, p;\n\t}" ::"r"(d),          \
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "n"(kDescHi)                                     \
      : "memory")
template <bool kPair, bool kFp8 = false>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                    uint32_t add) {
  if constexpr (kPair && kFp8) MUON_MMA("2", "f8f6f4");
  else if constexpr (kPair) MUON_MMA("2", "f16");
  else if constexpr (kFp8) MUON_MMA("1", "f8f6f4");
  else MUON_MMA("1", "f16");
}
#undef MUON_MMA

// One lane of the (whole) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Bounded wait of a whole warp.  The polling stays out of line: the kernels' code is large
// enough for instruction fetches to matter in short launches.
static __device__ __noinline__ bool wait_warp_slow(uint64_t* bar, uint32_t parity, int* err, int* abort) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitBudget, err, abort));
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* err, int* abort) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_warp_slow(bar, parity, err, abort);
}

// Arrives on `bar` (of both CTAs of a pair) when the MMAs issued so far complete.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kPair) tc_commit_pair(bar, (uint16_t)0x3);
  else tc_commit(bar);
}

// idesc_bf16 with both operand types cleared is the fp16 form.
__device__ __forceinline__ uint32_t idesc_16(bool bf16, int M, int N, int a_mn, int b_mn) {
  const uint32_t d = idesc_bf16(M, N, a_mn, b_mn);
  return bf16 ? d : d & ~((1u << 7) | (1u << 10));
}

// Waits for an arrival from the other CTA of the pair, acquiring what it wrote.
__device__ __forceinline__ bool wait_peer(uint64_t* bar, uint32_t parity, int* err,
                                          volatile int* abort) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitBudget) {
      atomicExch(err, kErrTimeout);
      *abort = 1;
      return false;
    }
  }
}

// Waits that ignore the abort flag: copies and MMAs in flight must end before the CTA does.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, int* err) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitBudget) {
      atomicExch(err, kErrTimeout);
      return;
    }
}

// Ends a producer: every copy it issued has landed (a pair's first CTA counts both CTAs') and,
// unless the launch is giving up, every stage has been handed back.  The second waits for the
// MMAs' arrivals on this CTA's own barriers, which come from the pair's first CTA: none may be
// on its way when this CTA ends and its shared memory goes to the next one.
template <typename V>
__device__ __forceinline__ void drain_ring(Control& c, int64_t fills, uint32_t rank, int* err) {
  for (int64_t f = fills - 1; f >= 0 && f >= fills - V::kStages; --f) {
    const int stage = (int)(f % V::kStages);
    const uint32_t phase = (uint32_t)((f / V::kStages) & 1);
    if (rank == 0) drain(&c.full[stage], phase, err);
    if (*reinterpret_cast<volatile int*>(&c.abort) == 0) drain(&c.empty[stage], phase, err);
  }
}

// Position in the ring of operand stages.
template <int kStages>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

template <bool kPair, int kWarps = kEpiWarps>
__device__ __forceinline__ void setup(Control& c, int warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
      mbar_init(&c.tail[s], 1);
      mbar_init(&c.fixed[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.acc_full[b], 1);
      mbar_init(&c.acc_empty[b], (kPair ? 2 : 1) * kWarps);
    }
    mbar_init(&c.mma_done, 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (kPair) {
      tmem_alloc_pair(&c.tmem, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&c.tmem, kTmemCols);
      tmem_relinquish();
    }
  }
}

// Barriers and TMEM are ready in every CTA that may signal them; or every CTA is done with the
// others' shared memory.
template <bool kCluster>
__device__ __forceinline__ void sync_ctas() {
  tc_fence_before();
  if constexpr (kCluster) cluster_sync(); else __syncthreads();
  tc_fence_after();
}

template <typename V>
__device__ __forceinline__ void teardown(Control& c, int warp) {
  sync_ctas<V::kPair || V::kSplit>();
  if (warp == 2) {
    if constexpr (V::kPair) tmem_dealloc_pair(c.tmem, kTmemCols);
    else tmem_dealloc(c.tmem, kTmemCols);
  }
}

// mbar_arrive_cluster without the release, which waits for all of the thread's stores to be visible to the
// cluster: where the arrival hands over no memory.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// An epilogue warp is done reading accumulator `ab`: its loads have completed (tmem_ld_wait), and no memory
// is handed over, so the arrival in the other CTA needs no release.  (With one, it waited for the warp's
// stores of the tile before: 1290 instead of 150 cycles.)
template <bool kPair>
__device__ __forceinline__ void release_acc(Control& c, int ab, uint32_t rank, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (!kPair || rank == 0) mbar_arrive(&c.acc_empty[ab]);
    else mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&c.acc_empty[ab]), 0));
  }
}

// Waits for accumulator use number `use` (epilogue warp).
__device__ __forceinline__ bool wait_acc(Control& c, uint32_t use, int* err) {
  if (!wait_warp(&c.acc_full[use & 1], use >> 1 & 1u, err, &c.abort)) return false;
  tc_fence_after();
  return true;
}

// 32 lanes x 16 consecutive 32-bit columns of TMEM.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// sum (+)= 32 accumulator columns from `col` on of this warp's lanes.  kWhole: the first ones in one load, which
// wants 32 registers more.
template <bool kWhole = true>
__device__ __forceinline__ void add_acc(uint32_t tmem, int ab, int q, int col, bool first,
                                        float (&sum)[32]) {
  const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kAccCols + col);
  if (kWhole && first) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(at, v);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; ++k) sum[k] = __uint_as_float(v[k]);
  } else {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(at + h, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k)
        sum[h + k] = !kWhole && first ? __uint_as_float(v[k]) : sum[h + k] + __uint_as_float(v[k]);
    }
  }
}

// Reads the row offsets into shared memory (whole block; null: one expert owns every row).  If they
// are not ascending within 0..rows, no expert gets a row and kErrRowOffsets is recorded.
__device__ __forceinline__ void load_offsets(const int64_t* offsets, int n_experts, int64_t rows,
                                             int32_t* off, int* err) {
  bool bad = false;
  for (int e = threadIdx.x; e <= n_experts; e += blockDim.x) {
    const int64_t o = offsets != nullptr ? offsets[e] : e > 0 ? rows : 0;
    bad |= o < 0 || o > rows || (e > 0 && offsets != nullptr && offsets[e - 1] > o);
    off[e] = (int32_t)o;
  }
  if (__syncthreads_or(bad)) {
    for (int e = threadIdx.x; e <= n_experts; e += blockDim.x) off[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(err, kErrRowOffsets);
    __syncthreads();
  }
}

// first[e] = row tiles of the experts before e, first[n_experts] = all (one warp).
__device__ __forceinline__ void count_tiles(const int32_t* off, int n_experts, int max_n, int lane,
                                            int32_t* first) {
  int32_t sum = 0;
  if (lane == 0) first[0] = 0;
  for (int base = 0; base < n_experts; base += 32) {
    const int e = base + lane;
    const int32_t rows = e < n_experts ? off[e + 1] - off[e] : 0;
    int32_t v = rows / max_n + (rows % max_n != 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (e < n_experts) first[e + 1] = sum + v;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
}

struct MmTile {
  int expert, row, rows;  // rows row .. row + rows - 1 of x and y, all of `expert`
  int n;                  // the MMA's N: rows in steps of kStepN
  int f0;                 // first column of y
};

// kCols: columns of y that one CTA's 128 accumulator lanes hold.
template <typename V, int kCols>
__device__ __forceinline__ MmTile mm_tile(uint32_t t, uint32_t f_tiles, int n_experts,
                                          const int32_t* off, const int32_t* first) {
  constexpr int kStep = Shape<V>::kStepN;
  const int rt = (int)(t / f_tiles);
  int lo = 0, hi = n_experts - 1;  // the expert with first[e] <= rt < first[e + 1]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (first[mid + 1] > rt) hi = mid; else lo = mid + 1;
  }
  const int rows = off[lo + 1] - off[lo], tiles = first[lo + 1] - first[lo];
  // Within the expert: groups of kGroup row tiles, in each every column tile of y, in each the
  // group's row tiles.  The CTAs at work at a time then share a few column tiles of the weight
  // and a group's rows, and the weight comes from HBM once per group.
  constexpr int kGroup = 8;
  uint32_t rest = t - (uint32_t)first[lo] * f_tiles;
  int group = 0, size = tiles;
  if (tiles > kGroup) {
    group = (int)(rest / (kGroup * f_tiles)) * kGroup;
    rest -= (uint32_t)group * f_tiles;
    size = min(kGroup, tiles - group);
  }
  int row_tile = 0, f_tile = (int)rest, width = rows;
  if (tiles > 1) {
    f_tile = (int)(rest / (uint32_t)size);
    row_tile = group + (int)rest - f_tile * size;
    width = (int)(((uint32_t)rows + (uint32_t)tiles - 1) / (uint32_t)tiles);
  }
  width = (width + kStep - 1) / kStep * kStep;
  const int begin = row_tile * width;
  MmTile m;
  m.expert = lo;
  m.row = off[lo] + begin;
  m.rows = min(width, rows - begin);
  m.n = (m.rows + kStep - 1) / kStep * kStep;
  m.f0 = f_tile * (kCols * Shape<V>::kCtas);
  return m;
}

// Index of the CTA in its cluster of `parts`, for Split.
struct Part {
  int index, parts;
};
template <typename V>
__device__ __forceinline__ Part split_part() {
  Part p{0, 1};
  if constexpr (V::kSplit) {
    p.index = (int)cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(p.parts));
  }
  return p;
}

// ---------------------------------------------------------------------------- operand copies
// Copies batches of row-major 16-bit matrices to rows that start on 16 bytes (TMA wants its
// pointers and strides in units of 16 bytes), zeros behind each row's last element.
struct AlignCopy {
  const uint16_t* src;
  uint4* dst;
  const int64_t* offsets;  // batches are experts: those without rows are left out (null: none is)
  int64_t ld, stride, rows, cols, chunks, total;  // 16-byte chunks per row; all rows (0: no copy)
  int64_t pitch;                                  // of the copy, in chunks
  int32_t lanes;           // threads that share a row
};

// Eight elements from s on, in the widest loads its alignment allows, as they are stored.
__device__ __forceinline__ uint4 load_unaligned(const uint16_t* s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(s);
  if (at % 8 == 0) {
    const uint2 a = *reinterpret_cast<const uint2*>(s), b = *reinterpret_cast<const uint2*>(s + 4);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  if (at % 4 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(s);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(s + 1);
  const uint32_t first = s[0], a = w[0], b = w[1], c = w[2], last = s[7];
  return make_uint4(first | a << 16, a >> 16 | b << 16, b >> 16 | c << 16, c >> 16 | last << 16);
}

__device__ __forceinline__ void align_rows(const AlignCopy& c) {
  const int lane = threadIdx.x % c.lanes, per = 256 / c.lanes;
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / c.lanes; row < c.total;
       row += (int64_t)gridDim.x * per) {
    const int64_t batch = row / c.rows;
    if (c.offsets != nullptr && c.offsets[batch + 1] <= c.offsets[batch]) continue;
    const uint16_t* s = c.src + batch * c.stride + (row - batch * c.rows) * c.ld;
    for (int64_t q = lane + (int64_t)blockIdx.y * c.lanes; q < c.chunks;
         q += (int64_t)gridDim.y * c.lanes) {
      const int64_t c0 = q * 8;
      uint4 v;
      if (c0 + 8 <= c.cols) {
        v = load_unaligned(s + c0);
      } else {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = c0 + k < c.cols ? s[c0 + k] : 0;
        v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
      c.dst[row * c.pitch + q] = v;
    }
  }
}

static __global__ void __launch_bounds__(256) align_rows_kernel(const AlignCopy a, const AlignCopy b) {
  if (a.total > 0) align_rows(a);
  if (b.total > 0) align_rows(b);
}

// One operand as the tensor maps see it: `batch` matrices of rows x cols.
struct Operand {
  const void* ptr;
  int64_t rows, cols, ld, batch, stride;
};

inline bool aligned(const Operand& o) {
  return reinterpret_cast<uintptr_t>(o.ptr) % 16 == 0 && o.ld % 8 == 0 &&
         (o.batch == 1 || o.stride % 8 == 0);
}

// Row pitch of a copy: whole 128-byte lines where a row fills one, so that no 128-byte box row
// straddles two.
inline int64_t copy_pitch(const Operand& o) {
  const int64_t unit = o.cols >= 64 ? 64 : 8;
  return (o.cols + unit - 1) / unit * unit;
}

inline size_t copy_bytes(const Operand& o) {
  if (aligned(o)) return 0;
  return (size_t)split_part_bytes(o.batch * o.rows * copy_pitch(o) * 2);
}

// Replaces an operand by its aligned copy at *at in the workspace, if it needs one; returns the
// copy to make.
inline AlignCopy align_operand(Operand* o, uint8_t** at, const int64_t* offsets) {
  AlignCopy c{};
  c.lanes = 1;
  const size_t bytes = copy_bytes(*o);
  if (bytes == 0) return c;
  c.src = static_cast<const uint16_t*>(o->ptr);
  c.dst = reinterpret_cast<uint4*>(*at);
  c.offsets = offsets;
  c.ld = o->ld;
  c.stride = o->stride;
  c.rows = o->rows;
  c.cols = o->cols;
  c.chunks = (o->cols + 7) / 8;
  c.total = o->batch * o->rows;
  c.pitch = copy_pitch(*o) / 8;
  while (c.lanes < 32 && c.lanes < c.chunks) c.lanes *= 2;
  o->ptr = *at;
  o->ld = c.pitch * 8;
  o->stride = o->rows * o->ld;
  *at += bytes;
  return c;
}

// Makes two operands' rows start on 16 bytes (either may be null); offsets: b's batches are experts.
// *at: where the workspace is still free.
inline cudaError_t align_operands(Operand* a, Operand* b, const int64_t* offsets, uint8_t** at, int sms,
                                  cudaStream_t st) {
  const AlignCopy none{nullptr, nullptr, nullptr, 0, 0, 0, 0, 0, 0, 0, 1};
  const AlignCopy ca = a != nullptr ? align_operand(a, at, nullptr) : none,
                  cb = b != nullptr ? align_operand(b, at, offsets) : none;
  const int64_t need = ca.total * ca.lanes > cb.total * cb.lanes ? ca.total * ca.lanes
                                                                 : cb.total * cb.lanes;
  if (need == 0) return cudaSuccess;
  // A thread takes one chunk of a row, more only where that is more than 8 blocks per SM.
  const int64_t chunks = ca.chunks > cb.chunks ? ca.chunks : cb.chunks;
  const int64_t cap = (int64_t)sms * 8, blocks = (need + 255) / 256 < cap ? (need + 255) / 256 : cap;
  const int64_t across = (chunks + 31) / 32, room = cap / blocks;
  align_rows_kernel<<<dim3((unsigned)blocks, (unsigned)(across < room ? across : room)), 256, 0, st>>>(
      ca, cb);
  return cudaGetLastError();
}

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  return fn;
}

// A tensor map with boxes of 128 bytes x box_rows rows (128-byte swizzle) over an operand whose
// rows start on 16 bytes; batched operands get a third dimension.
inline cudaError_t encode(CUtensorMap* map, const Operand& o, int32_t dtype, bool batched, uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t size = dtype == kF32 ? 4 : dtype == kE4m3 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.batch};
  // (The stride of a dimension of length 1 means nothing, but has to be a valid one.)
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * size,
                                 (cuuint64_t)(o.batch == 1 ? o.ld : o.stride) * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), box_rows, 1}, unit[3] = {1, 1, 1};
  const CUresult r = fn(map, dtype == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                             : dtype == kE4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                             : dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        batched ? 3 : 2, const_cast<void*>(o.ptr), dims, strides, box, unit,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launches at most one CTA per SM, in clusters of `ctas`, for `tiles` tiles; the kernel's
// shared-memory size is set once per device.
template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, int64_t tiles, int ctas, int sms, int smem,
                   std::atomic<uint64_t>* ready, cudaStream_t st, int threads = kThreads) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready->load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready->fetch_or(1ull << dev, std::memory_order_release);
  }
  const int64_t most = sms / ctas, units = tiles < 1 ? 1 : tiles < most ? tiles : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ctas), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The pitch of a single row means nothing: one that TMA takes.
inline Operand operand(const void* ptr, int64_t rows, int64_t cols, int64_t ld, int64_t batch,
                int64_t stride) {
  return {ptr, rows, cols, rows == 1 ? (cols + 7) / 8 * 8 : ld, batch, stride};
}

// At least as many tiles as the offsets can make of the rows, each `cols` columns of y per CTA wide.
template <typename V>
int64_t mm_tiles(const GroupedMm& g, int cols = kBM) {
  return (g.rows / V::kMaxN + (g.rows < g.n_experts ? g.rows : g.n_experts)) *
         ((g.n - 1) / (cols * Shape<V>::kCtas) + 1);
}

}  // namespace muon
