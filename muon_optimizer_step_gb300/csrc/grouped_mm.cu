// Products grouped by expert over ragged rows, on the tensor cores (tcgen05 + TMEM + TMA).
//
//   mm:    y[r, :] = x[r, :] W_e           (W_e stored k x n)
//          y[r, :] = x[r, :] W_e^T         (W_e stored n x k, trans)
//   wgrad: dW_e (+)= sum over the rows r of expert e of a[r, :]^T b[r, :]
//
// Expert e owns rows offsets[e] .. offsets[e + 1] - 1.  The offsets are on the device: every
// CTA reads and checks them, counts each expert's tiles and walks the same tile list, tile
// blockIdx.x + i * gridDim.x of it (one CTA per SM).  Rows of no expert (before offsets[0],
// from offsets[n_experts] on) get zeros.
//
// mm computes tiles of y^T: the MMA's M = 128 is 128 columns of y (the weight is operand A) and
// its N is up to kMaxN rows of one expert (x is operand B).  N goes in steps of 16 (32 on pairs)
// where M is fixed, so the ragged side wastes at most 15 (31) rows per tile instead of up to 127,
// and a single token costs an MMA of N = 16.  An expert's rows are dealt evenly to its tiles.  Both weight
// layouts are operand majors of the MMA (K-major or MN-major boxes), nothing is transposed.
// Rows that a tile's box reads past its expert are the next expert's; they reach accumulator
// columns that are not stored.
//
// wgrad reduces over an expert's rows: both operands are MN-major boxes of 64 rows.  The last
// box of an expert holds rows of the next one; MMAs of K = 16 that would see only those are
// not issued, and before the one that sees both kinds the issuing warp zeroes them in shared
// memory, in both operands (0 * NaN is NaN).
//
// Large products run on CTA pairs (a 2-CTA cluster, cta_group::2): each CTA holds 128 of the
// MMA's 256 rows and half of its N columns of operand B, so a k-block brings 32 KB instead of
// 48 KB into each SM for the same work (98304 rows, 1408 -> 2048, 64 experts: pairs 344 us,
// single CTAs 387).  The other tiles, and when they run, stand at the variants and launches below.
//
// The tensor core truncates when it adds to its accumulator, always towards zero, so the error
// of a sum grows with its number of steps (1.8e-6 of the result after 1536 rows).  Results are
// therefore summed in short segments, which the epilogue adds up in registers with rounding to
// nearest: 3.3e-7 whatever the length (3.6e-7 for a plain fp32 product of 1536 rows).  16-bit
// results in longer ones: of whole sums of 4096 terms one in 430 is stored in bf16 other than the
// exact sum would be, of 16384 terms one in 110; in segments one in 2000 whatever the length
// (98304 rows, 1408 -> 2048: 336 us in segments, 333 whole; 24570 rows, 2048 -> 1408: 111 and
// 109).
//
// CTA roles (384 threads): warp 0 issues the TMA loads, warp 1 the MMAs (on the first CTA of a
// pair), warp 2 owns TMEM, warps 4-11 drain the accumulators (two, in TMEM's 512 columns, so a
// tile's stores overlap the next one's MMAs).  Every wait on an mbarrier is bounded.  Those for the
// other CTAs of the cluster at the start and end, for TMEM and for a CTA's own stores are not: they
// end once the bounded ones have.
//
// The issuing warps walk their loops whole and elect a lane for each k-block: with one lane in
// a divergent loop, descriptors and barrier addresses went through vector registers and issue
// was the bound (a k-block took 750 cycles to load and 560 + 50 per MMA to multiply; the same
// product 489 us instead of 322).
//
// Measured, per pass (the loads fill the 64 bytes a cycle that an SM takes from L2 to about
// 90 %; in runs of more than a few ms the 1.4 kW limit lowers the clock to 1.35-1.5 GHz):
//   98304 rows, 1408 -> 2048, 64 experts  342 us  1.66 PFLOP/s, tensor pipe 82 % busy
//   4096 rows, 4096 -> 14336, 8 experts   306 us  1.57 PFLOP/s, 84 %
//   24570 rows, 2048 -> 1408, 64 experts  112 us  1.26 PFLOP/s and 4.8 TB/s
//   192 rows, 1408 -> 2048, 64 experts     54 us  6.5 TB/s (HBM)
//   6 rows, 2048 -> 1408, 64 experts      9.2 us  (4.5 us are launch, offsets and first load)
//   weight gradient of the first          452 us  1.25 PFLOP/s and 3.1 TB/s, 55 % (403 us with
//                                                 segments of 12: loads alone took 343, stores
//                                                 alone 288, MMAs alone 279)
#include <atomic>

#include <cudaTypedefs.h>

#include "device_common.cuh"
#include "element.cuh"
#include "kernels.h"
#include "row_blocks.h"

namespace muon {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kBM = 128;            // rows of operand A: M of the MMA
constexpr int kABytes = kBM * 128;  // 16 KB
constexpr int kBox = 64 * 128;      // an MN-major box: 64 k-rows of 128 bytes
constexpr int kAccCols = 256;       // TMEM columns of one accumulator
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
// 4).  With kSegment32 the error is a plain fp32 product's or at most a rounding (2^-24) more.
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

struct MmParams {
  CUtensorMap x;   // (k, rows): boxes of 64 x kBoxRows
  CUtensorMap w;   // (inner, outer, expert): boxes of 64 x 128 (trans) or 64 x 64
  GroupedMm g;
};

struct WgradParams {
  CUtensorMap a, b;  // (columns, rows): boxes of 64 x 64
  CUtensorMap dw;    // (column, row, expert) of the result: boxes of 32 x 32
  GroupedWgrad g;
  int32_t max_n;     // widest tile
  bool bulk;         // dw is written by TMA
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

template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                    uint32_t add) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "n"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "n"(kDescHi)
        : "memory");
}

// One lane of the (whole) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Bounded wait of a whole warp.  The polling stays out of line: the kernels' code is large
// enough for instruction fetches to matter in short launches.
__device__ __noinline__ bool wait_warp_slow(uint64_t* bar, uint32_t parity, int* err, int* abort) {
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

template <bool kPair>
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
      mbar_init(&c.acc_empty[b], (kPair ? 2 : 1) * kEpiWarps);
    }
    mbar_init(&c.mma_done, 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (kPair) {
      tmem_alloc_pair(&c.tmem, 2 * kAccCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&c.tmem, 2 * kAccCols);
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
    if constexpr (V::kPair) tmem_dealloc_pair(c.tmem, 2 * kAccCols);
    else tmem_dealloc(c.tmem, 2 * kAccCols);
  }
}

// An epilogue warp is done reading accumulator `ab`.
template <bool kPair>
__device__ __forceinline__ void release_acc(Control& c, int ab, uint32_t rank, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (!kPair || rank == 0) mbar_arrive(&c.acc_empty[ab]);
    else mbar_arrive_cluster(mapa_shared(smem_u32(&c.acc_empty[ab]), 0));
  }
}

// Waits for accumulator use number `use` (epilogue warp).
__device__ __forceinline__ bool wait_acc(Control& c, int use, int* err) {
  if (!wait_warp(&c.acc_full[use & 1], (use >> 1) & 1, err, &c.abort)) return false;
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

// sum (+)= 32 accumulator columns from `col` on of this warp's lanes.
__device__ __forceinline__ void add_acc(uint32_t tmem, int ab, int q, int col, bool first,
                                        float (&sum)[32]) {
  const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kAccCols + col);
  if (first) {
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
      for (int k = 0; k < 16; ++k) sum[h + k] += __uint_as_float(v[k]);
    }
  }
}

// Reads the row offsets into shared memory (whole block).  If they are not ascending within
// 0..rows, no expert gets a row and kErrRowOffsets is recorded.
__device__ __forceinline__ void load_offsets(const int64_t* offsets, int n_experts, int64_t rows,
                                             int32_t* off, int* err) {
  bool bad = false;
  for (int e = threadIdx.x; e <= n_experts; e += kThreads) {
    const int64_t o = offsets[e];
    bad |= o < 0 || o > rows || (e > 0 && offsets[e - 1] > o);
    off[e] = (int32_t)o;
  }
  if (__syncthreads_or(bad)) {
    for (int e = threadIdx.x; e <= n_experts; e += kThreads) off[e] = 0;
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

// ---------------------------------------------------------------------------- mm
struct MmTile {
  int expert, row, rows;  // rows row .. row + rows - 1 of x and y, all of `expert`
  int n;                  // the MMA's N: rows in steps of kStepN
  int f0;                 // first column of y
};

template <typename V>
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
  m.f0 = f_tile * Shape<V>::kM;
  return m;
}

// Stores accumulator columns 32 c .. 32 c + 31 (rows of y) of this warp's 32 lanes (columns
// f .. f + 31 of y): one coalesced access per row, whatever y's alignment.
template <typename O>
__device__ __forceinline__ void mm_store(const GroupedMm& g, const MmTile& m, int c, int f, int lane,
                                         const float (&v)[32]) {
  if (f + lane >= g.n) return;
  O* dst = static_cast<O*>(g.y) + ((int64_t)m.row + 32 * c) * g.ldy + f + lane;
  const int left = m.rows - 32 * c;
  if (left >= 32) {
#pragma unroll
    for (int t = 0; t < 32; ++t) put(dst + t * g.ldy, v[t]);
  } else {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (t < left) put(dst + t * g.ldy, v[t]);
  }
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

template <typename V, typename O>
__global__ void __launch_bounds__(kThreads, 1)
grouped_mm_kernel(const __grid_constant__ MmParams p) {
  using S = Shape<V>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GroupedMm& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = V::kPair ? cluster_ctarank() : 0u;
  const Part part_k = split_part<V>();
  if (threadIdx.x == 96) {  // warp 3: off the other warps' way
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.x);
  }
  setup<V::kPair>(c, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kMaxN, lane, first);
  __syncthreads();
  sync_ctas<V::kPair>();
  const uint32_t tmem = c.tmem;
  const uint32_t f_tiles = (uint32_t)(g.n - 1) / S::kM + 1, tiles = (uint32_t)first[g.n_experts] * f_tiles;
  int kb0 = 0, kb1 = (g.k - 1) / kBK + 1;  // this CTA's k-blocks
  uint32_t unit = blockIdx.x / S::kCtas, units = gridDim.x / S::kCtas;
  if constexpr (V::kSplit) {
    const int all = kb1;  // parts is a power of two
    const int shift = 31 - __clz(part_k.parts);
    kb0 = (int)((int64_t)all * part_k.index >> shift);
    kb1 = (int)((int64_t)all * (part_k.index + 1) >> shift);
    unit >>= shift;
    units >>= shift;
  }
  const int seg = segment_blocks(kb1 - kb0, sizeof(O) == 4 ? V::kSegment32 : V::kSegment16, V::kSub);

  if (warp == 0) {
    Ring<V::kStages> ring;
    int64_t fills = 0;
    bool ok = true;
    const uint32_t full0 = smem_u32(c.full), dst0 = smem_u32(smem);
    // A pair's second CTA signals the first one's barriers.
    const uint32_t sig0 = V::kPair ? mapa_shared(full0, 0) : full0;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V>(t, f_tiles, g.n_experts, off, first);
      const int part = m.n / S::kCtas;  // rows of x this CTA brings
      const int boxes = (part + V::kBoxRows - 1) / V::kBoxRows;
      const uint32_t bytes = S::kCtas * (kABytes + boxes * V::kBoxRows * 128);
      const int f = m.f0 + kBM * (int)rank, row = (int)((uint32_t)m.row + part * rank);
      for (int kb = kb0; kb < kb1; kb += V::kSub, ++fills) {
        ok = wait_warp(&c.empty[ring.stage], ring.phase ^ 1u, g.err, &c.abort);
        if (!ok) break;
        const uint32_t sig = sig0 + 8 * ring.stage, a = dst0 + ring.stage * S::kStage;
        const int blocks = min(V::kSub, kb1 - kb);
        if (elect_one()) {
          // Only the first CTA of a pair arrives, announcing both CTAs' bytes.
          if (rank == 0) expect(full0 + 8 * ring.stage, blocks * bytes);
#pragma unroll
          for (int j = 0; j < V::kSub; ++j) {
            if (j >= blocks) break;
            const int k0 = (kb + j) * kBK;
            const uint32_t aj = a + j * S::kBlock;
            if (g.trans) {
              load_3d<V::kPair>(aj, &p.w, k0, f, m.expert, sig);
            } else {
              load_3d<V::kPair>(aj, &p.w, f, k0, m.expert, sig);
              load_3d<V::kPair>(aj + kBox, &p.w, f + 64, k0, m.expert, sig);
            }
#pragma unroll
            for (int b = 0; b < V::kMaxN / S::kCtas / V::kBoxRows; ++b)
              if (b < boxes)
                load_2d<V::kPair>(aj + kABytes + b * V::kBoxRows * 128, &p.x, k0,
                                  (int)((uint32_t)row + b * V::kBoxRows), sig);
          }
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) drain_ring<V>(c, fills, rank, g.err);
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // The whole warp walks the k-blocks and one lane issues, so that descriptors and counters
    // stay warp-uniform.
    Ring<V::kStages> ring;
    int use = 0;
    bool ok = true;
    const uint32_t a_mn = g.trans ? 0 : 1, a_step = a_mn ? 16 * 128 / 16 : 32 / 16;
    const uint32_t a0 = desc_lo(smem_u32(smem), a_mn ? kBox : 16);
    const uint32_t b0 = desc_lo(smem_u32(smem) + kABytes, 16);
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V>(t, f_tiles, g.n_experts, off, first);
      const uint32_t idesc = idesc_16(g.dtype == kBf16, S::kM, m.n, a_mn, 0);
      for (int kb = kb0; kb < kb1;) {
        // One accumulator: a segment of the k-blocks.
        const int end = min(kb1, kb + seg);
        ok = wait_warp(&c.acc_empty[use & 1], ((use >> 1) & 1) ^ 1u, g.err, &c.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (use & 1) * kAccCols;
        uint32_t add = 0;
        for (; kb < end; kb += V::kSub) {
          ok = wait_warp(&c.full[ring.stage], ring.phase, g.err, &c.abort);
          if (!ok) break;
          const uint32_t a = a0 + ring.stage * (S::kStage / 16), b = b0 + ring.stage * (S::kStage / 16);
          const int blocks = min(V::kSub, kb1 - kb);
          if (elect_one()) {
            // Columns past k are zeros in both operands.
#pragma unroll
            for (int j = 0; j < V::kSub; ++j) {
              if (j >= blocks) break;
              const uint32_t aj = a + j * (S::kBlock / 16), bj = b + j * (S::kBlock / 16);
              mma<V::kPair>(d, aj, bj, idesc, j == 0 ? add : 1);
              mma<V::kPair>(d, aj + a_step, bj + 2, idesc, 1);
              mma<V::kPair>(d, aj + 2 * a_step, bj + 4, idesc, 1);
              mma<V::kPair>(d, aj + 3 * a_step, bj + 6, idesc, 1);
            }
            commit<V::kPair>(&c.empty[ring.stage]);
          }
          __syncwarp();
          add = 1;
          ring.next();
        }
        if (!ok) break;
        if (elect_one()) commit<V::kPair>(&c.acc_full[use & 1]);
        __syncwarp();
        ++use;
      }
    }
    if (elect_one()) {
      if constexpr (V::kPair) tc_commit_pair(&c.mma_done, (uint16_t)0x1);
      else tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;  // a quarter of the lanes, every second block
    int use = 0;
    bool ok = true;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V>(t, f_tiles, g.n_experts, off, first);
      const int f = m.f0 + kBM * (int)rank + 32 * q;
      float sum[S::kBlocks][32];
      for (int kb = kb0; kb < kb1; kb += seg, ++use) {
        ok = wait_acc(c, use, g.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < S::kBlocks; ++i)
          if ((2 * i + half) * 32 < m.n)
            add_acc(tmem, use & 1, q, (2 * i + half) * 32, kb == kb0, sum[i]);
        release_acc<V::kPair>(c, use & 1, rank, lane);
      }
      if (!ok) break;
      if constexpr (V::kSplit) {
        // The operand stages are free: this tile's MMAs were the last.
        if (half * 32 < m.n)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            reinterpret_cast<float*>(smem)[(q * V::kMaxN + half * 32 + k) * 32 + lane] = sum[0][k];
      } else {
#pragma unroll
        for (int i = 0; i < S::kBlocks; ++i)
          if ((2 * i + half) * 32 < m.n) mm_store<O>(g, m, 2 * i + half, f, lane, sum[i]);
      }
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x) {
      O* row = static_cast<O*>(g.y) + (z < head ? z : off[g.n_experts] + z - head) * g.ldy;
      for (int64_t f = threadIdx.x - 128; f < g.n; f += kEpiWarps * 32) put(&row[f], 0.f);
    }
  }
  if constexpr (V::kSplit) {
    // The parts of the tile are in the CTAs' shared memory, as [quarter][row of y][column]:
    // every CTA adds and stores a share, 8 columns per thread, the parts in order.
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && unit < tiles) {
      const MmTile m = mm_tile<V>(unit, f_tiles, g.n_experts, off, first);
      const int cols = g.n - m.f0;
      for (int i = threadIdx.x - 128 + part_k.index * kEpiWarps * 32; i < m.rows * 16;
           i += part_k.parts * kEpiWarps * 32) {
        const int r = i / 16, col = i % 16 * 8;
        const uint32_t at = smem_u32(smem) + ((col / 32 * V::kMaxN + r) * 32 + col % 32) * 4;
        float sum[8] = {};
        for (int q = 0; q < part_k.parts; ++q) {
          float v[8];
          const uint32_t from = mapa_shared(at, q);
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(from) : "memory");
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(from + 16) : "memory");
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[k] += v[k];
        }
        O* dst = static_cast<O*>(g.y) + (int64_t)(m.row + r) * g.ldy + m.f0 + col;
        if (col + 8 <= cols && reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
          __align__(16) O o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) put(&o[k], sum[k]);
#pragma unroll
          for (int k = 0; k < (int)sizeof(O) / 2; ++k)
            reinterpret_cast<uint4*>(dst)[k] = reinterpret_cast<const uint4*>(o)[k];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col + k < cols) put(&dst[k], sum[k]);
        }
      }
    }
    __syncwarp();
  }
  teardown<V>(c, warp);
}

// ---------------------------------------------------------------------------- wgrad
constexpr int kWgradStaging = 4096;  // per epilogue warp: a block of 32 x 32 floats
constexpr int kWgradStep = 32;       // tiles are whole blocks wide, but for the matrix's edge

struct WgradTile {
  int expert, row, rows;  // the expert's rows
  int i0, j0, cols, n;    // first row and column of dw, its columns, and the MMA's N
};

struct WgradGrid {
  uint32_t m_tiles, n_tiles;
  int width;
  int64_t tiles;
};

template <typename V>
__host__ __device__ __forceinline__ WgradGrid wgrad_grid(const GroupedWgrad& g, int max_n) {
  WgradGrid w;
  w.m_tiles = (g.m - 1) / Shape<V>::kM + 1;
  w.n_tiles = (uint32_t)(g.n - 1) / (uint32_t)max_n + 1;
  // Columns dealt evenly.
  w.width = (int)((uint32_t)(g.n - 1) / w.n_tiles + kWgradStep) / kWgradStep * kWgradStep;
  w.tiles = (int64_t)g.n_experts * w.m_tiles * w.n_tiles;
  return w;
}

// part: the share of the expert's k-blocks that a CTA of a split tile takes (all by default).
template <typename V>
__device__ __forceinline__ WgradTile wgrad_tile(const GroupedWgrad& g, const WgradGrid& w, uint32_t t,
                                                bool bad, const Part& part = Part{0, 1}) {
  // Row tiles first: the CTAs at work at a time share column panels of b (446 against 450 us on
  // 64 x 2048 x 1408 in a long run, 407 against 414 in a short one).
  const uint32_t per = w.m_tiles * w.n_tiles, e = t / per, r = t - e * per, j = r / w.m_tiles;
  WgradTile x;
  x.expert = e;
  x.row = bad ? 0 : (int)g.offsets[e];
  x.rows = bad ? 0 : (int)(g.offsets[e + 1] - g.offsets[e]);
  x.i0 = (int)(r - j * w.m_tiles) * Shape<V>::kM;
  x.j0 = (int)j * w.width;
  x.cols = min(w.width, g.n - x.j0);
  x.n = (x.cols + kWgradStep - 1) / kWgradStep * kWgradStep;
  if (V::kSplit && part.parts > 1) {
    const RowShare s = row_share(x.rows, part.index, 31 - __clz(part.parts));  // a power of two
    x.rows = s.rows;
    x.row += s.first;
  }
  return x;
}

// Zeroes rows left .. 15 of the last K = 16 step in each of a stage's boxes (whole warp).
__device__ __forceinline__ void zero_rows(uint8_t* stage, int left, int boxes, int lane) {
  const int rows = 16 - left % 16;
  uint8_t* z = stage + left * 128;
  for (int i = lane; i < boxes * rows * 8; i += 32)
    *reinterpret_cast<uint4*>(z + i / (rows * 8) * kBox + i % (rows * 8) * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// The 32 values from dst on that lane's row of a block holds (n of them inside the matrix).  A
// lane's loads cover whole 32-byte sectors where they can: beside the operand stages L1 has no
// room to keep the rest of one for the next load.
__device__ __forceinline__ void wgrad_load(const float* dst, int n, float (&v)[32]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(dst);
  if (n >= 32 && at % 32 == 0) {
#pragma unroll
    for (int k = 0; k < 32; k += 8)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[k]), "=f"(v[k + 1]), "=f"(v[k + 2]), "=f"(v[k + 3]), "=f"(v[k + 4]),
                     "=f"(v[k + 5]), "=f"(v[k + 6]), "=f"(v[k + 7])
                   : "l"(dst + k)
                   : "memory");
  } else if (n >= 32 && at % 16 == 0) {
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 q = *reinterpret_cast<const float4*>(dst + k);
      v[k] = q.x;
      v[k + 1] = q.y;
      v[k + 2] = q.z;
      v[k + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = k < n ? dst[k] : 0.f;
  }
}

// Writes, or (kAdd) adds to, the block dw[row .. row + 31, col .. col + 31] whose row `lane` the warp's
// lane holds.
// The block is turned around in `stage` (16-byte chunk k of row r in slot k ^ (r & 7), free of
// bank conflicts on the way in), so that every access covers one row.
template <bool kAdd>
__device__ __forceinline__ void wgrad_store(float* dw, int64_t lddw, int rows, int cols, int lane,
                                            const float (&v)[32], float4* stage) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    stage[8 * lane + (k ^ (lane & 7))] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  __syncwarp();
  // Element (r, lane) of the block.
  const auto at = [&](int r) {
    return reinterpret_cast<const float*>(stage + 8 * r + (lane >> 2 ^ (r & 7)))[lane & 3];
  };
  if (lane < cols) {
    dw += lane;
    if (rows >= 32 && !kAdd) {
#pragma unroll
      for (int r = 0; r < 32; ++r, dw += lddw) *dw = at(r);
    } else {
      rows = min(rows, 32);
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8, dw += 8 * lddw) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = kAdd && r0 + k < rows ? dw[k * lddw] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r0 + k < rows) dw[k * lddw] = o[k] + at(r0 + k);
      }
    }
  }
  __syncwarp();
}

// The same by TMA, which drops what lies outside the matrix: the warp's only waits are for the
// previous block to have left `stage`.  Every row of dw must start and end on 16 bytes.
__device__ __forceinline__ void wgrad_store_bulk(const CUtensorMap* map, int expert, int row, int col,
                                                 int lane, const float (&v)[32], float4* stage) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k)  // the 128-byte swizzle of the map
    stage[8 * lane + (k ^ (lane & 7))] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
        "r"(col), "r"(row), "r"(expert), "r"(smem_u32(stage))
        : "memory");
    bulk_commit();
  }
}

// A split tile's block i of epilogue warp `warp`, as [column][row], in a CTA's operand stages.
__device__ __forceinline__ float* wgrad_part(uint8_t* smem, int warp, int i) {
  return reinterpret_cast<float*>(smem) + (warp * 4 + i) * 1024;
}

// Adds the parts of a split tile, in order, out of the cluster's shared memory and writes them:
// the blocks are dealt to the epilogue warps of all its CTAs.
__device__ __forceinline__ void wgrad_join(const WgradParams& p, uint8_t* smem, float4* stage,
                                           const Part& split, uint32_t t, uint32_t tiles,
                                           const WgradGrid& w, bool bad, int lane, int warp) {
  if (t >= tiles) return;
  const GroupedWgrad& g = p.g;
  const WgradTile x = wgrad_tile<SplitWide>(g, w, t, bad);
  if (x.rows == 0 && g.accumulate) return;
  for (int b = split.index * kEpiWarps + warp; b < kEpiWarps * 4; b += split.parts * kEpiWarps) {
    const int from = b >> 2, i = b & 3;  // the warp and block that hold it
    const int row = x.i0 + 32 * (from & 3), col = (2 * i + (from >> 2)) * 32;
    if (col >= x.cols || row >= g.m) continue;
    float sum[32] = {};
    const uint32_t at = smem_u32(wgrad_part(smem, from, i)) + lane * 4;
    for (int q = 0; q < split.parts; ++q) {
      const uint32_t from_q = mapa_shared(at, q);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from_q + k * 128) : "memory");
        sum[k] += v;
      }
    }
    float* dw = g.dw + x.expert * g.dw_stride + (int64_t)row * g.lddw + x.j0 + col;
    if (p.bulk && !g.accumulate) wgrad_store_bulk(&p.dw, x.expert, row, x.j0 + col, lane, sum, stage);
    else if (g.accumulate) wgrad_store<true>(dw, g.lddw, g.m - row, x.cols - col, lane, sum, stage);
    else wgrad_store<false>(dw, g.lddw, g.m - row, x.cols - col, lane, sum, stage);
  }
}

template <typename V>
__global__ void __launch_bounds__(kThreads, 1)
grouped_wgrad_kernel(const __grid_constant__ WgradParams p) {
  using S = Shape<V>;
  static_assert(V::kSub == 1, "a stage is a k-block");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GroupedWgrad& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = V::kPair ? cluster_ctarank() : 0u;
  if (threadIdx.x == 96 && g.rows > 0) {
    prefetch_tmap(&p.a);
    prefetch_tmap(&p.b);
  }
  setup<V::kPair>(c, warp);
  bool bad = false;
  for (int e = threadIdx.x; e <= g.n_experts; e += kThreads) {
    const int64_t o = g.offsets[e];
    bad |= o < 0 || o > g.rows || (e > 0 && g.offsets[e - 1] > o);
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicExch(g.err, kErrRowOffsets);
  sync_ctas<V::kPair>();
  const uint32_t tmem = c.tmem;
  const WgradGrid w = wgrad_grid<V>(g, p.max_n);
  const Part split = split_part<V>();
  const uint32_t ctas = S::kCtas * split.parts, tiles = (uint32_t)w.tiles;
  const uint32_t unit = blockIdx.x / ctas, units = gridDim.x / ctas;

  if (warp == 0) {
    Ring<V::kStages> ring;
    int64_t fills = 0;
    uint32_t tails = 0, used = 0;  // per stage: parity of the next use of `tail`; any use
    bool ok = true;
    const uint32_t full0 = smem_u32(c.full), tail0 = smem_u32(c.tail), dst0 = smem_u32(smem);
    const uint32_t sig0 = V::kPair ? mapa_shared(full0, 0) : full0;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const WgradTile x = wgrad_tile<V>(g, w, t, bad, split);
      const int part = x.n / S::kCtas, boxes = (part + 63) / 64;  // columns of b this CTA brings
      const int i = x.i0 + kBM * (int)rank, j = x.j0 + part * (int)rank;
      for (int left = x.rows; left > 0; left -= kBK, ++fills) {
        ok = wait_warp(&c.empty[ring.stage], ring.phase ^ 1u, g.err, &c.abort);
        if (!ok) break;
        const uint32_t a = dst0 + ring.stage * S::kStage;
        const int y = x.row + (x.rows - left);
        // A last stage with rows to zero lands on each CTA's own barrier.
        const bool own = V::kPair && left < kBK && left % 16 != 0;
        if (own) {
          const uint32_t bar = (rank == 0 ? full0 : tail0) + 8 * ring.stage;
          if (elect_one()) {
            expect(bar, (2 + boxes) * kBox);
            for (int b = 0; b < 2; ++b) load_2d<false>(a + b * kBox, &p.a, i + 64 * b, y, bar);
            for (int b = 0; b < boxes; ++b)
              load_2d<false>(a + kABytes + b * kBox, &p.b, j + 64 * b, y, bar);
          }
          if (rank != 0) {
            tails ^= 1u << ring.stage;
            used |= 1u << ring.stage;
          }
        } else if (elect_one()) {
          const uint32_t sig = sig0 + 8 * ring.stage;
          if (rank == 0) expect(full0 + 8 * ring.stage, S::kCtas * (2 + boxes) * kBox);
          load_2d<V::kPair>(a, &p.a, i, y, sig);
          load_2d<V::kPair>(a + kBox, &p.a, i + 64, y, sig);
#pragma unroll
          for (int b = 0; b < V::kMaxN / S::kCtas / 64; ++b)
            if (b < boxes) load_2d<V::kPair>(a + kABytes + b * kBox, &p.b, j + 64 * b, y, sig);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) {
      drain_ring<V>(c, fills, rank, g.err);
      for (int s = 0; s < V::kStages; ++s)
        if (used >> s & 1) drain(&c.tail[s], (tails >> s & 1) ^ 1u, g.err);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    Ring<V::kStages> ring;
    int use = 0;
    uint32_t fixes = 0;  // per stage: parity of the next use of its `fixed` barrier
    bool ok = true;
    constexpr uint32_t kStep = 16 * 128 / 16;
    const uint32_t a0 = desc_lo(smem_u32(smem), kBox), b0 = desc_lo(smem_u32(smem) + kABytes, kBox);
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const WgradTile x = wgrad_tile<V>(g, w, t, bad, split);
      const uint32_t idesc = idesc_16(g.dtype == kBf16, S::kM, x.n, 1, 1);
      const int seg = segment_blocks(row_blocks(x.rows), V::kSegment32, 1);
      for (int left = x.rows; left > 0;) {
        ok = wait_warp(&c.acc_empty[use & 1], ((use >> 1) & 1) ^ 1u, g.err, &c.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (use & 1) * kAccCols;
        uint32_t add = 0;
        for (int in = 0; in < seg && left > 0; ++in, left -= kBK) {
          ok = wait_warp(&c.full[ring.stage], ring.phase, g.err, &c.abort);
          if (!ok) break;
          if (left < kBK && left % 16 != 0) {
            // The rows behind the expert's last are the next expert's.
            zero_rows(smem + ring.stage * S::kStage, left, 2 + (x.n / S::kCtas + 63) / 64, lane);
            if (V::kPair) {
              ok = __all_sync(0xffffffffu, wait_peer(&c.fixed[ring.stage], fixes >> ring.stage & 1,
                                                     g.err, &c.abort));
              if (!ok) break;
              fixes ^= 1u << ring.stage;
            }
          }
          const uint32_t a = a0 + ring.stage * (S::kStage / 16), b = b0 + ring.stage * (S::kStage / 16);
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (left > s * 16)
                mma<V::kPair>(d, a + s * kStep, b + s * kStep, idesc, s == 0 ? add : 1);
            commit<V::kPair>(&c.empty[ring.stage]);
          }
          __syncwarp();
          add = 1;
          ring.next();
        }
        if (!ok) break;
        if (elect_one()) commit<V::kPair>(&c.acc_full[use & 1]);
        __syncwarp();
        ++use;
      }
    }
    if (elect_one()) {
      if constexpr (V::kPair) tc_commit_pair(&c.mma_done, (uint16_t)0x1);
      else tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // Second CTA of a pair: zeroes its own part of a last k-block, then tells the first CTA.
    // A stage's barriers are used again only after the MMAs that waited for this.
    int64_t fills = 0;
    uint32_t tails = 0;  // per stage: parity of the next use of its `tail` barrier
    for (uint32_t t = unit; t < tiles; t += units) {
      const WgradTile x = wgrad_tile<V>(g, w, t, bad, split);
      fills += row_blocks(x.rows);
      const int left = x.rows % kBK;
      if (left % 16 == 0) continue;
      const int stage = (int)((fills - 1) % V::kStages);
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&c.tail[stage], tails >> stage & 1, kWaitBudget,
                                                     g.err, &c.abort)))
        break;
      tails ^= 1u << stage;
      zero_rows(smem + stage * S::kStage, left, 2 + (x.n / S::kCtas + 63) / 64, lane);
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&c.fixed[stage]), 0));
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    float4* stage =
        reinterpret_cast<float4*>(smem + V::kStages * S::kStage + (warp - 4) * kWgradStaging);
    int use = 0;
    bool ok = true;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const WgradTile x = wgrad_tile<V>(g, w, t, bad, split);
      if (x.rows == 0 && g.accumulate && !V::kSplit) continue;
      const int row = x.i0 + kBM * (int)rank + 32 * q;
      float* dw = g.dw + x.expert * g.dw_stride + (int64_t)row * g.lddw + x.j0;
      // The sums start from the old values, which arrive while the MMAs run.
      const bool old = g.accumulate && !V::kSplit;
      if (old && p.bulk && t + units < tiles && lane < S::kBlocks) {
        // The next tile's come to L2, a block per lane (64 x 2048 x 1408 from 24570 rows: 354
        // us without, 311 with).
        const WgradTile y = wgrad_tile<V>(g, w, t + units, bad, split);
        const int r = y.i0 + kBM * (int)rank + 32 * q, col = (2 * lane + half) * 32;
        if (r < g.m && col < y.cols)
          asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(&p.dw),
                       "r"(y.j0 + col), "r"(r), "r"(y.expert)
                       : "memory");
      }
      float sum[S::kBlocks][32];
      if (old || x.rows == 0)
#pragma unroll
        for (int i = 0; i < S::kBlocks; ++i)
          wgrad_load(dw + lane * g.lddw + (2 * i + half) * 32,
                     old && row + lane < g.m ? x.cols - (2 * i + half) * 32 : 0, sum[i]);
      const int blocks = row_blocks(x.rows), seg = segment_blocks(blocks, V::kSegment32, 1);
      for (int b = 0; b < blocks; b += seg, ++use) {
        ok = wait_acc(c, use, g.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < S::kBlocks; ++i)
          if ((2 * i + half) * 32 < x.n)
            add_acc(tmem, use & 1, q, (2 * i + half) * 32, b == 0 && !old, sum[i]);
        release_acc<V::kPair>(c, use & 1, rank, lane);
      }
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < S::kBlocks; ++i) {
        const int col = (2 * i + half) * 32;
        if (col >= x.cols || row >= g.m) continue;
        if (V::kSplit) {
          // The operand stages are free: this tile's MMAs were the last.
#pragma unroll
          for (int k = 0; k < 32; ++k) wgrad_part(smem, warp - 4, i)[k * 32 + lane] = sum[i][k];
        } else if (p.bulk) {
          wgrad_store_bulk(&p.dw, x.expert, row, x.j0 + col, lane, sum[i], stage);
        } else {
          wgrad_store<false>(dw + col, g.lddw, g.m - row, x.cols - col, lane, sum[i], stage);
        }
      }
    }
    if constexpr (V::kSplit) {
      // (The other warps wait at the same barrier below.)
      __syncwarp();
      cluster_sync();
      wgrad_join(p, smem, stage, split, unit, tiles, w, bad, lane, warp - 4);
    }
    // Shared memory must outlive the stores that read it.
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  if constexpr (V::kSplit) {
    __syncwarp();
    if (warp < 4) cluster_sync();
  }
  teardown<V>(c, warp);
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

__global__ void __launch_bounds__(256) align_rows_kernel(const AlignCopy a, const AlignCopy b) {
  if (a.total > 0) align_rows(a);
  if (b.total > 0) align_rows(b);
}

// One operand as the tensor maps see it: `batch` matrices of rows x cols.
struct Operand {
  const void* ptr;
  int64_t rows, cols, ld, batch, stride;
};

bool aligned(const Operand& o) {
  return reinterpret_cast<uintptr_t>(o.ptr) % 16 == 0 && o.ld % 8 == 0 &&
         (o.batch == 1 || o.stride % 8 == 0);
}

// Row pitch of a copy: whole 128-byte lines where a row fills one, so that no 128-byte box row
// straddles two.
int64_t copy_pitch(const Operand& o) {
  const int64_t unit = o.cols >= 64 ? 64 : 8;
  return (o.cols + unit - 1) / unit * unit;
}

size_t copy_bytes(const Operand& o) {
  if (aligned(o)) return 0;
  return (size_t)split_part_bytes(o.batch * o.rows * copy_pitch(o) * 2);
}

// Replaces an operand by its aligned copy at *at in the workspace, if it needs one; returns the
// copy to make.
AlignCopy align_operand(Operand* o, uint8_t** at, const int64_t* offsets) {
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

// Makes both operands' rows start on 16 bytes; offsets: b's batches are experts.
cudaError_t align_operands(Operand* a, Operand* b, const int64_t* offsets, void* workspace, int sms,
                           cudaStream_t st) {
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const AlignCopy ca = align_operand(a, &at, nullptr), cb = align_operand(b, &at, offsets);
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

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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
cudaError_t encode(CUtensorMap* map, const Operand& o, int32_t dtype, bool batched, uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t size = dtype == kF32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.batch};
  // (The stride of a dimension of length 1 means nothing, but has to be a valid one.)
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * size,
                                 (cuuint64_t)(o.batch == 1 ? o.ld : o.stride) * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), box_rows, 1}, unit[3] = {1, 1, 1};
  const CUresult r = fn(map, dtype == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
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
                   std::atomic<uint64_t>* ready, cudaStream_t st) {
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
  cfg.blockDim = dim3(kThreads, 1, 1);
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

// At least as many tiles as the offsets can make of the rows.
template <typename V>
int64_t mm_tiles(const GroupedMm& g) {
  return (g.rows / V::kMaxN + (g.rows < g.n_experts ? g.rows : g.n_experts)) *
         ((g.n - 1) / Shape<V>::kM + 1);
}

template <typename V, typename O>
cudaError_t launch_mm(const MmParams& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  return launch(grouped_mm_kernel<V, O>, p, mm_tiles<V>(p.g), Shape<V>::kCtas * parts, sms,
                V::kStages * Shape<V>::kStage + 1024, &ready, st);
}

template <typename V>
cudaError_t launch_mm_as(const MmParams& p, int parts, int sms, cudaStream_t st) {
  return p.g.out_dtype == kF32 ? launch_mm<V, float>(p, parts, sms, st)
         : p.g.out_dtype == kBf16 ? launch_mm<V, __nv_bfloat16>(p, parts, sms, st)
                                  : launch_mm<V, __half>(p, parts, sms, st);
}

template <typename V>
cudaError_t launch_wgrad(const WgradParams& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  return launch(grouped_wgrad_kernel<V>, p, wgrad_grid<V>(p.g, p.max_n).tiles,
                Shape<V>::kCtas * parts, sms,
                V::kStages * Shape<V>::kStage + kEpiWarps * kWgradStaging + 1024, &ready, st);
}

// The pitch of a single row means nothing: one that TMA takes.
Operand operand(const void* ptr, int64_t rows, int64_t cols, int64_t ld, int64_t batch,
                int64_t stride) {
  return {ptr, rows, cols, rows == 1 ? (cols + 7) / 8 * 8 : ld, batch, stride};
}
Operand x_of(const GroupedMm& g) { return operand(g.x, g.rows, g.k, g.ldx, 1, 0); }
Operand w_of(const GroupedMm& g) {
  return operand(g.w, g.trans ? g.n : g.k, g.trans ? g.k : g.n, g.ldw, g.n_experts, g.w_stride);
}
Operand a_of(const GroupedWgrad& g) { return operand(g.a, g.rows, g.m, g.lda, 1, 0); }
Operand b_of(const GroupedWgrad& g) { return operand(g.b, g.rows, g.n, g.ldb, 1, 0); }

}  // namespace

// The device counts tiles in 32 bits.
bool grouped_mm_fits(const GroupedMm& g) {
  return (g.rows / Narrow::kMaxN + g.n_experts) * (int64_t)((g.n - 1) / kBM + 1) <= INT32_MAX;
}

bool grouped_wgrad_fits(const GroupedWgrad& g) {
  return (int64_t)g.n_experts * ((g.m - 1) / kBM + 1) * ((g.n - 1) / 64 + 1) <= INT32_MAX;
}

size_t grouped_mm_workspace(const GroupedMm& g) {
  return g.rows == 0 ? 0 : copy_bytes(x_of(g)) + copy_bytes(w_of(g));
}

size_t grouped_wgrad_workspace(const GroupedWgrad& g) {
  return g.rows == 0 ? 0 : copy_bytes(a_of(g)) + copy_bytes(b_of(g));
}

cudaError_t launch_grouped_mm(const GroupedMm& g, void* workspace, int sms, cudaStream_t st) {
  MmParams p;
  p.g = g;
  Operand x = x_of(g), w = w_of(g);
  cudaError_t e = align_operands(&x, &w, g.offsets, workspace, sms, st);
  // Which tiles (us, by rows of the whole product):
  //  - A k-split where every cluster gets an SM for each of its CTAs, and one tile (6 rows,
  //    2048 -> 1408: 13.8 without, 9.2 with; 1 row: 13.5 and 5.9).
  //  - Few rows per expert, up to a narrow tile's: streaming the weights is the whole cost
  //    (64 experts, 2048 -> 1408, average rows 32: narrow 59.8, pairs 66.9; 64: 65.1 and 69.4;
  //    80: 76.2 and 70.9).  Few tiles: the more SMs work (1 expert, 512 rows, 2048 -> 2048:
  //    narrow 11.2, wide 14.8).
  //  - Pairs for 16-bit results, from two tiles for each pair of SMs on (8 experts, 2048 -> 2048,
  //    2048 rows: 128 tiles, pairs 25.6, wide 25.9; 4096 rows: 36.2 and 39.4; 64 experts, 2048 ->
  //    1408, 24570 rows: 117 and 129).  The shorter segments of fp32 results hold pairs up (the last
  //    two: 53.0 and 45.4, 147 and 142; 98304 rows, 1408 -> 2048: 425 and 437).
  int parts = 1;
  while (parts < kMostParts && mm_tiles<Split>(g) * parts * 2 <= sms && g.k >= 4 * kBK * parts * 2)
    parts *= 2;
  const bool narrow = g.rows <= Narrow::kMaxN * (int64_t)g.n_experts || mm_tiles<Narrow>(g) <= sms;
  const bool pair = !narrow && g.out_dtype != kF32 && g.n > kBM && mm_tiles<Pair>(g) >= sms;
  if (e == cudaSuccess)
    e = encode(&p.x, x, g.dtype, false, parts > 1 || narrow ? Narrow::kBoxRows : Wide::kBoxRows);
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, g.trans ? kBM : 64);
  if (e != cudaSuccess) return e;
  return parts > 1 ? launch_mm_as<Split>(p, parts, sms, st)
         : narrow  ? launch_mm_as<Narrow>(p, 1, sms, st)
         : !pair   ? launch_mm_as<Wide>(p, 1, sms, st)
         : g.out_dtype == kBf16 ? launch_mm<Pair, __nv_bfloat16>(p, 1, sms, st)
                                : launch_mm<Pair, __half>(p, 1, sms, st);
}

cudaError_t launch_grouped_wgrad(const GroupedWgrad& g, void* workspace, int sms, cudaStream_t st) {
  WgradParams p;
  p.g = g;
  Operand a = a_of(g), b = b_of(g);
  cudaError_t e = cudaSuccess;
  if (g.rows > 0) {  // without rows nothing is loaded: the maps stay unused
    e = align_operands(&a, &b, nullptr, workspace, sms, st);
    if (e == cudaSuccess) e = encode(&p.a, a, g.dtype, false, 64);
    if (e == cudaSuccess) e = encode(&p.b, b, g.dtype, false, 64);
  }
  // Written by TMA where every row of dw starts and ends on 16 bytes: a store fills the last 16
  // bytes of a row whole, with what lies behind the row's end in them.
  p.bulk = reinterpret_cast<uintptr_t>(g.dw) % 16 == 0 && g.lddw % 4 == 0 && g.n % 4 == 0 &&
           (g.n_experts == 1 || g.dw_stride % 4 == 0);
  if (e == cudaSuccess && p.bulk)
    e = encode(&p.dw, {g.dw, g.m, g.n, g.lddw, g.n_experts, g.dw_stride}, kF32, true, 32);
  if (e != cudaSuccess) return e;
  p.max_n = 256;
  // Pairs for many rows (64 experts of 2048 x 1408, average rows 768: pairs 279, wide 286 us, adding
  // 421 and 449; 384: 195 and 190, adding 333 and 313).
  if (g.m > kBM && wgrad_grid<Pair>(g, 256).tiles >= sms / 2 && g.rows >= 512 * (int64_t)g.n_experts)
    return launch_wgrad<Pair>(p, 1, sms, st);
  // Few tiles: with many rows several CTAs for each (32 x 216 from 7855 rows 33.6 -> 12.6 us),
  // then narrower ones, while every SM gets at most one (13 experts of 130 x 520 from 154 rows
  // each 16.3 -> 10.5 us).
  int parts = 1;
  while (parts < kMostParts && wgrad_grid<Wide>(g, 256).tiles * parts * 2 <= sms &&
         g.rows >= (int64_t)g.n_experts * parts * 8 * kBK)
    parts *= 2;
  while (p.max_n > 64 && wgrad_grid<Wide>(g, p.max_n / 2).tiles * parts <= sms) p.max_n /= 2;
  return parts > 1 ? launch_wgrad<SplitWide>(p, parts, sms, st) : launch_wgrad<Wide>(p, 1, sms, st);
}

}  // namespace muon
