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
// its N is up to kMaxN rows of one expert (x is operand B).  N goes in steps of 16 where M is
// fixed, so the ragged side wastes at most 15 rows per tile instead of up to 127, and a single
// token costs an MMA of N = 16.  An expert's rows are dealt evenly to its tiles.  Both weight
// layouts are operand majors of the MMA (K-major or MN-major boxes), nothing is transposed.
// Rows that a tile's box reads past its expert are the next expert's; they reach accumulator
// columns that are not stored.
//
// wgrad reduces over an expert's rows: both operands are MN-major boxes of 64 rows.  The last
// box of an expert holds rows of the next one; MMAs of K = 16 that would see only those are
// not issued, and before the one that sees both kinds the issuing warp zeroes them in shared
// memory, in both operands (0 * NaN is NaN).
//
// CTA roles (384 threads): warp 0 issues the TMA loads, warp 1 the MMAs, warp 2 owns TMEM,
// warps 4-11 drain the accumulators (two, in TMEM's 512 columns,
// so a tile's stores overlap the next one's MMAs).  Every wait is bounded.
#include <atomic>

#include <cudaTypedefs.h>

#include "device_common.cuh"
#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kBM = 128;            // rows of operand A: M of the MMA
constexpr int kBK = 64;             // k-block: 128 bytes of a 16-bit row
constexpr int kABytes = kBM * 128;  // 16 KB
constexpr int kBox = 64 * 128;      // an MN-major box: 64 k-rows of 128 bytes
constexpr int kAccCols = 256;       // TMEM columns of one accumulator
constexpr int kStagingBytes = 2048; // per epilogue warp (mm)
constexpr long long kWaitBudget = 4000000000LL;  // ~2 s of SM clock per wait

// mm tile variants.  Wide: up to 256 rows per tile, for experts with many rows.  Narrow: up to
// 64, whose smaller stages leave room for more of the weight in flight: with few rows the
// product is bound by streaming it.
struct Wide {
  static constexpr int kMaxN = 256, kBoxRows = 64, kStages = 4;
};
struct Narrow {
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 8;
};

struct MmParams {
  CUtensorMap x;   // (k, rows): boxes of 64 x kBoxRows
  CUtensorMap w;   // (inner, outer, expert): boxes of 64 x 128 (trans) or 64 x 64
  GroupedMm g;
};

struct WgradParams {
  CUtensorMap a, b;  // (columns, rows): boxes of 64 x 64
  GroupedWgrad g;
};

// Barriers and flags of one CTA.
struct Control {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// idesc_bf16 with both operand types cleared is the fp16 form.
__device__ __forceinline__ uint32_t idesc_16(bool bf16, int N, int a_mn, int b_mn) {
  const uint32_t d = idesc_bf16(kBM, N, a_mn, b_mn);
  return bf16 ? d : d & ~((1u << 7) | (1u << 10));
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

__device__ __forceinline__ void setup(Control& c, int stages, int warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.acc_full[b], 1);
      mbar_init(&c.acc_empty[b], kEpiWarps);
    }
    mbar_init(&c.mma_done, 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&c.tmem, 2 * kAccCols);
    tmem_relinquish();
  }
}

__device__ __forceinline__ void teardown(Control& c, int warp) {
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(c.tmem, 2 * kAccCols);
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
  int n;                  // the MMA's N: rows in steps of 16
  int f0;                 // first column of y
};

__device__ __forceinline__ MmTile mm_tile(int64_t t, int f_tiles, int n_experts, const int32_t* off,
                                          const int32_t* first) {
  const int rt = (int)(t / f_tiles);
  int lo = 0, hi = n_experts - 1;  // the expert with first[e] <= rt < first[e + 1]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (first[mid + 1] > rt) hi = mid; else lo = mid + 1;
  }
  MmTile m;
  m.expert = lo;
  const int rows = off[lo + 1] - off[lo], tiles = first[lo + 1] - first[lo];
  const int width = ((rows + tiles - 1) / tiles + 15) & ~15;
  const int begin = (rt - first[lo]) * width;
  m.row = off[lo] + begin;
  m.rows = min(width, rows - begin);
  m.n = (m.rows + 15) & ~15;
  m.f0 = (int)(t % f_tiles) * kBM;
  return m;
}

// Stores accumulator columns 32 c .. 32 c + 31 (rows of y) of this warp's 32 lanes (columns
// f .. f + 31 of y): the block is turned around in `stage` (2 KB), so that 64 or 128
// consecutive bytes of a row of y leave together.
template <typename O>
__device__ __forceinline__ void mm_store(const GroupedMm& g, const MmTile& m, int c, int f, int lane,
                                         const uint32_t (&v)[32], O* stage) {
  constexpr int kRows = kStagingBytes / (32 * sizeof(O));  // rows staged at a time
  constexpr int kPer = 16 / sizeof(O), kChunks = 32 / kPer, kPass = 32 / kChunks;
#pragma unroll
  for (int h = 0; h < 32 / kRows; ++h) {
    if (c * 32 + h * kRows >= m.rows) break;
#pragma unroll
    for (int t = 0; t < kRows; ++t) put(&stage[t * 32 + lane], __uint_as_float(v[h * kRows + t]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRows / kPass; ++i) {
      const int t = i * kPass + lane / kChunks, q = lane % kChunks * kPer;
      const int r = c * 32 + h * kRows + t, col = f + q;
      if (r < m.rows && col < g.n) {
        O* dst = static_cast<O*>(g.y) + (int64_t)(m.row + r) * g.ldy + col;
        const O* src = stage + t * 32 + q;
        if (col + kPer <= g.n && reinterpret_cast<uintptr_t>(dst) % 16 == 0)
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else
          for (int e = 0; e < kPer && col + e < g.n; ++e) dst[e] = src[e];
      }
    }
    __syncwarp();
  }
}

template <typename V, typename O>
__global__ void __launch_bounds__(kThreads, 1)
grouped_mm_kernel(const __grid_constant__ MmParams p) {
  constexpr int kStageBytes = kABytes + V::kMaxN * 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GroupedMm& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  setup(c, V::kStages, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kMaxN, lane, first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort = &c.abort;
  const int f_tiles = (g.n - 1) / kBM + 1, k_blocks = (g.k - 1) / kBK + 1;
  const int64_t tiles = (int64_t)first[g.n_experts] * f_tiles;

  if (warp == 0) {
    if (lane == 0) {
      Ring<V::kStages> ring;
      int64_t fills = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const MmTile m = mm_tile(t, f_tiles, g.n_experts, off, first);
        const int boxes = (m.n + V::kBoxRows - 1) / V::kBoxRows;
        const uint32_t bytes = kABytes + boxes * V::kBoxRows * 128;
        for (int kb = 0; kb < k_blocks; ++kb, ++fills) {
          uint64_t* full = &c.full[ring.stage];
          if (!mbar_wait_bounded(&c.empty[ring.stage], ring.phase ^ 1u, kWaitBudget, g.err, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full, bytes);
          uint8_t* sa = smem + ring.stage * kStageBytes;
          const int k0 = kb * kBK;
          if (g.trans) {
            tma_load_3d(sa, &p.w, k0, m.f0, m.expert, full);
          } else {
            tma_load_3d(sa, &p.w, m.f0, k0, m.expert, full);
            tma_load_3d(sa + kBox, &p.w, m.f0 + 64, k0, m.expert, full);
          }
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sa + kABytes + b * V::kBoxRows * 128, &p.x, k0, m.row + b * V::kBoxRows,
                        full);
          ring.next();
        }
      }
      for (int64_t f = fills - 1; f >= 0 && f >= fills - V::kStages; --f)
        drain(&c.full[f % V::kStages], (uint32_t)((f / V::kStages) & 1), g.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      Ring<V::kStages> ring;
      int local = 0;
      bool ok = true;
      const uint32_t sbase = smem_u32(smem);
      const int a_mn = g.trans ? 0 : 1;
      const uint32_t a_step = a_mn ? 16 * 128 : 32, a_lbo = a_mn ? kBox : 16;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++local) {
        const MmTile m = mm_tile(t, f_tiles, g.n_experts, off, first);
        const uint32_t idesc = idesc_16(g.dtype == kBf16, m.n, a_mn, 0);
        const int ab = local & 1;
        if (!mbar_wait_bounded(&c.acc_empty[ab], ((local >> 1) & 1) ^ 1u, kWaitBudget, g.err, abort))
          break;
        tc_fence_after();
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait_bounded(&c.full[ring.stage], ring.phase, kWaitBudget, g.err, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = sbase + ring.stage * kStageBytes, sb = sa + kABytes;
          const int steps = min(4, (g.k - kb * kBK + 15) / 16);
          for (int s = 0; s < steps; ++s)
            tc_mma_f16(tmem + ab * kAccCols, smem_desc_sw128(sa + s * a_step, a_lbo, 1024),
                       smem_desc_sw128(sb + s * 32, 16, 1024), idesc, (kb | s) != 0);
          tc_commit(&c.empty[ring.stage]);
          ring.next();
        }
        if (ok) tc_commit(&c.acc_full[ab]);
      }
      tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;  // a quarter of the lanes, every second block
    O* stage = reinterpret_cast<O*>(smem + V::kStages * kStageBytes + (warp - 4) * kStagingBytes);
    int local = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++local) {
      const MmTile m = mm_tile(t, f_tiles, g.n_experts, off, first);
      const int ab = local & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&c.acc_full[ab], (local >> 1) & 1, kWaitBudget,
                                                     g.err, abort)))
        break;
      tc_fence_after();
      for (int b = half; b * 32 < m.n; b += 2) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kAccCols + 32 * b), v);
        tmem_ld_wait();
        mm_store<O>(g, m, b, m.f0 + 32 * q, lane, v, stage);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.acc_empty[ab]);
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x) {
      O* row = static_cast<O*>(g.y) + (z < head ? z : off[g.n_experts] + z - head) * g.ldy;
      for (int64_t f = threadIdx.x - 128; f < g.n; f += kEpiWarps * 32) put(&row[f], 0.f);
    }
  }
  teardown(c, warp);
}

// ---------------------------------------------------------------------------- wgrad
constexpr int kWgradStages = 4;
constexpr int kWgradStage = kABytes + 256 * 128;

struct WgradTile {
  int expert, row, rows;  // the expert's rows
  int i0, j0, cols, n;    // first row and column of dw, its columns, and the MMA's N
};

struct WgradGrid {
  int m_tiles, n_tiles, width;
  int64_t tiles;
};

__host__ __device__ __forceinline__ WgradGrid wgrad_grid(const GroupedWgrad& g) {
  WgradGrid w;
  w.m_tiles = (g.m - 1) / kBM + 1;
  w.n_tiles = (g.n - 1) / 256 + 1;
  w.width = ((g.n - 1) / w.n_tiles + 1 + 15) & ~15;  // columns dealt evenly, in steps of 16
  w.tiles = (int64_t)g.n_experts * w.m_tiles * w.n_tiles;
  return w;
}

__device__ __forceinline__ WgradTile wgrad_tile(const GroupedWgrad& g, const WgradGrid& w, int64_t t,
                                                const int32_t* off) {
  const int64_t per = (int64_t)w.m_tiles * w.n_tiles;
  const int e = (int)(t / per);
  const int64_t r = t - e * per;
  WgradTile x;
  x.expert = e;
  x.row = off[e];
  x.rows = off[e + 1] - off[e];
  x.i0 = (int)(r / w.n_tiles) * kBM;
  x.j0 = (int)(r % w.n_tiles) * w.width;
  x.cols = min(w.width, g.n - x.j0);
  x.n = (x.cols + 15) & ~15;
  return x;
}

__global__ void __launch_bounds__(kThreads, 1)
grouped_wgrad_kernel(const __grid_constant__ WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ int32_t off[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GroupedWgrad& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  setup(c, kWgradStages, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort = &c.abort;
  const WgradGrid w = wgrad_grid(g);

  if (warp == 0) {
    if (lane == 0) {
      Ring<kWgradStages> ring;
      int64_t fills = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < w.tiles && ok; t += gridDim.x) {
        const WgradTile x = wgrad_tile(g, w, t, off);
        const int boxes = (x.n + 63) / 64;
        for (int r = 0; r < x.rows; r += kBK, ++fills) {
          uint64_t* full = &c.full[ring.stage];
          if (!mbar_wait_bounded(&c.empty[ring.stage], ring.phase ^ 1u, kWaitBudget, g.err, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full, (2 + boxes) * kBox);
          uint8_t* sa = smem + ring.stage * kWgradStage;
          for (int b = 0; b < 2; ++b)
            tma_load_2d(sa + b * kBox, &p.a, x.i0 + 64 * b, x.row + r, full);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sa + kABytes + b * kBox, &p.b, x.j0 + 64 * b, x.row + r, full);
          ring.next();
        }
      }
      for (int64_t f = fills - 1; f >= 0 && f >= fills - kWgradStages; --f)
        drain(&c.full[f % kWgradStages], (uint32_t)((f / kWgradStages) & 1), g.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // The whole warp waits, lane 0 issues: the last k-block of an expert needs all lanes.
    Ring<kWgradStages> ring;
    int local = 0;
    bool ok = true;
    const uint32_t sbase = smem_u32(smem);
    for (int64_t t = blockIdx.x; t < w.tiles && ok; t += gridDim.x) {
      const WgradTile x = wgrad_tile(g, w, t, off);
      if (x.rows == 0) continue;
      const uint32_t idesc = idesc_16(g.dtype == kBf16, x.n, 1, 1);
      const int ab = local & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&c.acc_empty[ab], ((local >> 1) & 1) ^ 1u,
                                                     kWaitBudget, g.err, abort));
      ++local;
      tc_fence_after();
      for (int r = 0; r < x.rows && ok; r += kBK) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&c.full[ring.stage], ring.phase, kWaitBudget,
                                                       g.err, abort));
        if (!ok) break;
        const int left = x.rows - r, steps = min(4, (left + 15) / 16);
        if (left < kBK && left % 16 != 0) {
          // Rows left .. 16 steps - 1 of every box (A's two, then B's) are the next expert's.
          const int rows = 16 * steps - left, boxes = 2 + (x.n + 63) / 64;
          uint8_t* z = smem + ring.stage * kWgradStage + left * 128;
          for (int i = lane; i < boxes * rows * 8; i += 32)
            *reinterpret_cast<uint4*>(z + i / (rows * 8) * kBox + i % (rows * 8) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = sbase + ring.stage * kWgradStage, sb = sa + kABytes;
          for (int s = 0; s < steps; ++s)
            tc_mma_f16(tmem + ab * kAccCols, smem_desc_sw128(sa + s * 16 * 128, kBox, 1024),
                       smem_desc_sw128(sb + s * 16 * 128, kBox, 1024), idesc, (r | s) != 0);
          tc_commit(&c.empty[ring.stage]);
        }
        ring.next();
      }
      if (ok && lane == 0) tc_commit(&c.acc_full[ab]);
    }
    if (lane == 0) {
      tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    int local = 0;
    for (int64_t t = blockIdx.x; t < w.tiles; t += gridDim.x) {
      const WgradTile x = wgrad_tile(g, w, t, off);
      if (x.rows == 0 && g.accumulate) continue;
      const int ab = local & 1;
      if (x.rows > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&c.acc_full[ab], (local >> 1) & 1,
                                                       kWaitBudget, g.err, abort)))
          break;
        ++local;
        tc_fence_after();
      }
      const int i = x.i0 + 32 * q + lane;
      float* row = g.dw + x.expert * g.dw_stride + (int64_t)i * g.lddw + x.j0;
      for (int b = half; b * 32 < x.n; b += 2) {
        uint32_t v[32];
        if (x.rows > 0) {
          tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kAccCols + 32 * b),
                             v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0u;
        }
        if (i >= g.m) continue;
        float* dst = row + 32 * b;
        if (b * 32 + 32 <= x.cols && reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
          float4 o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = g.accumulate ? __ldcs(reinterpret_cast<const float4*>(dst) + k)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            o[k].x += __uint_as_float(v[4 * k]);
            o[k].y += __uint_as_float(v[4 * k + 1]);
            o[k].z += __uint_as_float(v[4 * k + 2]);
            o[k].w += __uint_as_float(v[4 * k + 3]);
            __stcs(reinterpret_cast<float4*>(dst) + k, o[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (b * 32 + k < x.cols)
              dst[k] = g.accumulate ? dst[k] + __uint_as_float(v[k]) : __uint_as_float(v[k]);
        }
      }
      if (x.rows > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.acc_empty[ab]);
      }
    }
  }
  teardown(c, warp);
}

// ---------------------------------------------------------------------------- operand copies
// Copies a batch of row-major 16-bit matrices to rows that start on 16 bytes (TMA wants its
// pointers and strides in units of 16 bytes), zeros behind each row's last element.
__global__ void __launch_bounds__(256)
align_rows_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t stride, int64_t rows,
                  int64_t cols, int64_t chunks, int64_t total, uint4* __restrict__ dst) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / chunks, c0 = (i - row * chunks) * 8;
    const int64_t batch = row / rows;
    const uint16_t* s = src + batch * stride + (row - batch * rows) * ld + c0;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = c0 + 2 * e < cols ? s[2 * e] : 0, hi = c0 + 2 * e + 1 < cols ? s[2 * e + 1] : 0;
      v[e] = lo | hi << 16;
    }
    dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
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

size_t copy_bytes(const Operand& o) {
  if (aligned(o)) return 0;
  return (size_t)split_part_bytes(o.batch * o.rows * ((o.cols + 7) / 8) * 16);
}

// Replaces an operand by its aligned copy at *at in the workspace, if it needs one.
cudaError_t align_operand(Operand* o, uint8_t** at, int sms, cudaStream_t st) {
  const size_t bytes = copy_bytes(*o);
  if (bytes == 0) return cudaSuccess;
  const int64_t chunks = (o->cols + 7) / 8, total = o->batch * o->rows * chunks;
  const int64_t blocks = (total + 255) / 256, cap = (int64_t)sms * 8;
  align_rows_kernel<<<(int)(blocks < cap ? blocks : cap), 256, 0, st>>>(
      static_cast<const uint16_t*>(o->ptr), o->ld, o->stride, o->rows, o->cols, chunks, total,
      reinterpret_cast<uint4*>(*at));
  o->ptr = *at;
  o->ld = chunks * 8;
  o->stride = o->rows * o->ld;
  *at += bytes;
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

// A tensor map over an aligned operand with boxes of 64 columns x box_rows rows (128-byte
// swizzle); batched operands get a third dimension.
cudaError_t encode(CUtensorMap* map, const Operand& o, int32_t dtype, bool batched, uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.batch};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2,
                                 (cuuint64_t)(o.batch == 1 ? o.rows * o.ld : o.stride) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1}, unit[3] = {1, 1, 1};
  const CUresult r = fn(map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        batched ? 3 : 2, const_cast<void*>(o.ptr), dims, strides, box, unit,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launches a persistent kernel; its shared-memory size is set once per device.
template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, int grid, int smem, std::atomic<uint64_t>* ready,
                   cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready->load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready->fetch_or(1ull << dev, std::memory_order_release);
  }
  kernel<<<grid, kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

int grid_for(int64_t tiles, int sms) { return (int)(tiles < 1 ? 1 : tiles < sms ? tiles : sms); }

template <typename V, typename O>
cudaError_t launch_mm(const MmParams& p, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const GroupedMm& g = p.g;
  const int64_t row_tiles = g.rows / V::kMaxN + (g.rows < g.n_experts ? g.rows : g.n_experts);
  const int64_t tiles = row_tiles * ((g.n - 1) / kBM + 1);
  const int smem = V::kStages * (kABytes + V::kMaxN * 128) + kEpiWarps * kStagingBytes + 1024;
  return launch(grouped_mm_kernel<V, O>, p, grid_for(tiles, sms), smem, &ready, st);
}

template <typename V>
cudaError_t launch_mm_as(const MmParams& p, int sms, cudaStream_t st) {
  return p.g.out_dtype == kF32 ? launch_mm<V, float>(p, sms, st)
         : p.g.out_dtype == kBf16 ? launch_mm<V, __nv_bfloat16>(p, sms, st)
                                  : launch_mm<V, __half>(p, sms, st);
}

Operand x_of(const GroupedMm& g) { return {g.x, g.rows, g.k, g.ldx, 1, 0}; }
Operand w_of(const GroupedMm& g) {
  return {g.w, g.trans ? g.n : g.k, g.trans ? g.k : g.n, g.ldw, g.n_experts, g.w_stride};
}
Operand a_of(const GroupedWgrad& g) { return {g.a, g.rows, g.m, g.lda, 1, 0}; }
Operand b_of(const GroupedWgrad& g) { return {g.b, g.rows, g.n, g.ldb, 1, 0}; }

}  // namespace

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
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = align_operand(&x, &at, sms, st);
  if (e == cudaSuccess) e = align_operand(&w, &at, sms, st);
  // Few rows per expert: streaming the weights is the whole cost.
  const bool narrow = g.rows <= 64 || g.rows <= 32 * (int64_t)g.n_experts;
  if (e == cudaSuccess)
    e = encode(&p.x, x, g.dtype, false, narrow ? Narrow::kBoxRows : Wide::kBoxRows);
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, g.trans ? kBM : 64);
  if (e != cudaSuccess) return e;
  return narrow ? launch_mm_as<Narrow>(p, sms, st) : launch_mm_as<Wide>(p, sms, st);
}

cudaError_t launch_grouped_wgrad(const GroupedWgrad& g, void* workspace, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  WgradParams p;
  p.g = g;
  Operand a = a_of(g), b = b_of(g);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (g.rows > 0) {  // without rows nothing is loaded: the maps stay unused
    e = align_operand(&a, &at, sms, st);
    if (e == cudaSuccess) e = align_operand(&b, &at, sms, st);
    if (e == cudaSuccess) e = encode(&p.a, a, g.dtype, false, 64);
    if (e == cudaSuccess) e = encode(&p.b, b, g.dtype, false, 64);
  }
  if (e != cudaSuccess) return e;
  return launch(grouped_wgrad_kernel, p, grid_for(wgrad_grid(g).tiles, sms),
                kWgradStages * kWgradStage + 1024, &ready, st);
}

}  // namespace muon
