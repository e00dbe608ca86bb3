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
//   weight gradient of the first          411 us  1.38 PFLOP/s and 3.4 TB/s (loads alone took 343,
//                                                 stores alone 288, MMAs alone 279; 452 while a
//                                                 pair's second CTA handed its accumulators back with
//                                                 a release, see release_acc)
#include "grouped_kernel.cuh"

namespace muon {

namespace {

struct WgradParams {
  CUtensorMap a, b;  // (columns, rows): boxes of 64 x 64
  CUtensorMap dw;    // (column, row, expert) of the result: boxes of 32 x 32
  GroupedWgrad g;
  int32_t max_n;     // widest tile
  bool bulk;         // dw is written by TMA
};

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

template <typename V>
cudaError_t launch_wgrad(const WgradParams& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  return launch(grouped_wgrad_kernel<V>, p, wgrad_grid<V>(p.g, p.max_n).tiles,
                Shape<V>::kCtas * parts, sms,
                V::kStages * Shape<V>::kStage + kEpiWarps * kWgradStaging + 1024, &ready, st);
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
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = align_operands(&x, &w, g.offsets, &at, sms, st);
  const MmChoice c = choose_tiles<Plain<float>>(g, g.out_dtype == kF32, sms);
  if (e == cudaSuccess) e = encode(&p.x, x, g.dtype, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, g.trans ? kBM : 64);
  if (e != cudaSuccess) return e;
  return g.out_dtype == kF32 ? launch_tiles<Plain<float>, false>(p, c, sms, st)
         : g.out_dtype == kBf16 ? launch_tiles<Plain<__nv_bfloat16>, true>(p, c, sms, st)
                                : launch_tiles<Plain<__half>, true>(p, c, sms, st);
}

cudaError_t launch_grouped_wgrad(const GroupedWgrad& g, void* workspace, int sms, cudaStream_t st) {
  WgradParams p;
  p.g = g;
  Operand a = a_of(g), b = b_of(g);
  cudaError_t e = cudaSuccess;
  if (g.rows > 0) {  // without rows nothing is loaded: the maps stay unused
    uint8_t* at = static_cast<uint8_t*>(workspace);
    e = align_operands(&a, &b, nullptr, &at, sms, st);
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
