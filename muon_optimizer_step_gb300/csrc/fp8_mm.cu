// Products of 8-bit operands (e4m3) grouped by expert, with a scale for each 128 columns of a row of x and
// for each block of 128 x 128 of a weight.
//
//   y[r, c] = sum over the blocks b of 128 along k of
//             x_scale[b][r] w_scale[e][c / 128][b] (sum over b's k of x[r, k] w_e[c, k])
//
// A k-block is 128 bytes of a row, one block of the scales: each is an accumulator of its own (two in turn), and
// the epilogue warps add it to the sums in registers, times its row's scale and the weight's.  So every 128 terms
// are summed in the tensor core, the blocks in fp32 with rounding to nearest.
//
// Few rows per expert: tiles of y^T as in the grouped products of 16-bit operands (see grouped_mm.cu), 128
// columns of y (the weight, operand A) by up to 64 rows of one expert, or a cluster of CTAs that share the
// k-blocks of one.  Streaming the weight bounds them.  Many: tiles of y, below.
//
// Warp 3 brings the scales into a ring of slots in shared memory, several k-blocks ahead (cp.async).  It also looks
// for scales whose product is so far from 1 that it takes more than one factor (see Factors).
#include <cstddef>

#include "grouped_kernel.cuh"

namespace muon {

namespace {

constexpr int kBK8 = 128;   // elements of a k-block: 128 bytes
// Slots of scales.  (With 8 the next k-block's waited for the epilogue: 3600 rows, 2048 -> 1408, 50.3 us against 47.3.)
constexpr int kSlots = 16;
constexpr int kAhead = 6;   // k-blocks that scales are asked for ahead
constexpr int kStaging8 = 1024;          // bytes of each epilogue warp: 8 rows of its 32 columns

struct Fp8Params {
  CUtensorMap x, w;  // (k, rows) and (k, columns of y, expert): boxes of 128 x 16 and 128 x 128, or (tiles
                     // of y) 128 x 128 and 128 x 64
  Fp8Mm g;
};

// Few rows per expert: the tiles of y^T, as for 16-bit operands (see grouped_tiles.cuh), with a k-block per
// stage.
struct Narrow8 {
  static constexpr bool kPair = false, kSplit = false;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 6, kSub = 1;
};
struct Split8 {
  static constexpr bool kPair = false, kSplit = true;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 6, kSub = 1;
};

struct Scales {
  alignas(16) float slot[kSlots][64];  // read 16 bytes at a time
  float first[kSlots][64], again[kSlots][64];  // where `far`, see Factors (the slot then holds zeros)
  int far[kSlots];
  float weight[kSlots][32];  // the weight's scale, a copy for each lane of warp 3
  uint64_t full[kSlots], empty[kSlots];
};

static_assert(alignof(Scales) >= 16 && offsetof(Scales, slot) % 16 == 0, "add_block reads the slots in 16-byte units");

// What a block's sum is multiplied by: the product of its two scales, or, where that leaves 2^-100 .. 2^100, the
// product by 2^-128 (2^128) and twice 2^64 (2^-64).  A sum is 0 or of 2^-18 .. 2^25, so that nothing on the way
// leaves fp32's normal range unless the result does: a product of 2^128 and more would make NaN of a sum of 0, one
// below 2^-126 would lose bits.
struct Factors {
  float first, again;
};
constexpr float kNearOne = 0x1p100f;
__device__ __forceinline__ bool near_one(float product) {
  return fabsf(product) >= 1.f / kNearOne && fabsf(product) <= kNearOne;
}
__device__ __forceinline__ Factors factors(float x, float w) {
  const float p = x * w;
  if (near_one(p) || x == 0.f || w == 0.f) return {p, 1.f};
  return fabsf(p) > 1.f ? Factors{x * 0x1p-64f * (w * 0x1p-64f), 0x1p64f}
                        : Factors{x * 0x1p64f * (w * 0x1p64f), 0x1p-64f};
}

__device__ __forceinline__ void copy_4(void* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ float low(f32x2 v) { return parts(v).x; }
__device__ __forceinline__ float high(f32x2 v) { return parts(v).y; }

__device__ __forceinline__ f32x2 pair_of(const uint32_t* v) {
  return pair(__uint_as_float(v[0]), __uint_as_float(v[1]));
}

// sum += 32 accumulator columns in v, times their scales from s on (16-byte aligned).
__device__ __forceinline__ void add_block(f32x2 (&sum)[16], const uint32_t (&v)[32], const float* s) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    f32x2 x, y;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(smem_u32(s + k)));
    sum[k / 2] = fma2(pair_of(v + k), x, sum[k / 2]);
    sum[k / 2 + 1] = fma2(pair_of(v + k + 2), y, sum[k / 2 + 1]);
  }
}
// sum += a lane's 32 accumulator columns from `at` on, times both factors of their scales.  Out of line, the sums in
// memory: few calls have any.
static __device__ __noinline__ void add_far_block(f32x2* sum, uint32_t at, const float* first, const float* again) {
#pragma unroll 1
  for (int h = 0; h < 32; h += 16) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(at + h, v);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const f32x2 f = pair(first[h + k], first[h + k + 1]), t = pair(again[h + k], again[h + k + 1]);
      sum[(h + k) / 2] = fma2(mul2(mul2(pair_of(v + k), f), t), t, sum[(h + k) / 2]);
    }
  }
}
// The factors of two rows of a slot; whether any of the warp's goes beyond the product (then they are stored).
static __device__ __noinline__ bool far_slot(float* first, float* again, float x0, float x1, float w) {
  const Factors f0 = factors(x0, w), f1 = factors(x1, w);
  if (!__any_sync(0xffffffffu, f0.again != 1.f || f1.again != 1.f)) return false;
  first[0] = f0.first, again[0] = f0.again;
  first[32] = f1.first, again[32] = f1.again;
  return true;
}
// f(the sums in memory): where sums in registers meet a function that is out of line.
template <int kN, typename F>
__device__ __forceinline__ void in_memory(f32x2 (&sum)[kN], const F& f) {
  f32x2 there[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) there[k] = sum[k];
  f(there);
#pragma unroll
  for (int k = 0; k < kN; ++k) sum[k] = there[k];
}

template <typename V, typename O>
__global__ void __launch_bounds__(kThreads, 1) fp8_mm_kernel(const __grid_constant__ Fp8Params p) {
  using S = Shape<V>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ Scales sc;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Fp8Mm& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part part_k = split_part<V>();
  if (threadIdx.x == 96) {
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.x);
  }
  if (warp == 3 && lane < kSlots) {
    mbar_init(&sc.full[lane], 1);
    mbar_init(&sc.empty[lane], kEpiWarps);
    fence_mbar_init();
  }
  setup<false>(c, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kMaxN, lane, first);
  __syncthreads();
  sync_ctas<false>();
  const uint32_t tmem = c.tmem;
  const uint32_t f_tiles = (uint32_t)(g.n - 1) / S::kM + 1, tiles = (uint32_t)first[g.n_experts] * f_tiles;
  const int blocks = (g.k - 1) / kBK8 + 1;
  int kb0 = 0, kb1 = blocks;  // this CTA's k-blocks
  uint32_t unit = blockIdx.x, units = gridDim.x;
  if constexpr (V::kSplit) {
    const int shift = 31 - __clz(part_k.parts);  // parts is a power of two
    kb0 = (int)((int64_t)blocks * part_k.index >> shift);
    kb1 = (int)((int64_t)blocks * (part_k.index + 1) >> shift);
    unit >>= shift;
    units >>= shift;
  }

  if (warp == 0) {
    Ring<V::kStages> ring;
    int64_t fills = 0;
    bool ok = true;
    const uint32_t full0 = smem_u32(c.full), dst0 = smem_u32(smem);
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const int boxes = (m.n + V::kBoxRows - 1) / V::kBoxRows;
      const uint32_t bytes = kABytes + boxes * V::kBoxRows * 128;
      for (int kb = kb0; kb < kb1; ++kb, ++fills) {
        ok = wait_warp(&c.empty[ring.stage], ring.phase ^ 1u, g.err, &c.abort);
        if (!ok) break;
        const uint32_t sig = full0 + 8 * ring.stage, a = dst0 + ring.stage * S::kStage;
        if (elect_one()) {
          expect(sig, bytes);
          load_3d<false>(a, &p.w, kb * kBK8, m.f0, m.expert, sig);
#pragma unroll
          for (int b = 0; b < V::kMaxN / V::kBoxRows; ++b)
            if (b < boxes)
              load_2d<false>(a + kABytes + b * V::kBoxRows * 128, &p.x, kb * kBK8,
                             (int)((uint32_t)m.row + b * V::kBoxRows), sig);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) drain_ring<V>(c, fills, 0, g.err);
    __syncwarp();
  } else if (warp == 1) {
    Ring<V::kStages> ring;
    uint32_t use = 0;
    bool ok = true;
    const uint32_t a0 = desc_lo(smem_u32(smem), 16), b0 = desc_lo(smem_u32(smem) + kABytes, 16);
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const uint32_t idesc = idesc_16(false, S::kM, m.n, 0, 0);  // e4m3 has the same code as fp16
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        ok = wait_warp(&c.acc_empty[use & 1], (use >> 1 & 1u) ^ 1u, g.err, &c.abort) &&
             wait_warp(&c.full[ring.stage], ring.phase, g.err, &c.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (use & 1) * kAccCols;
        const uint32_t a = a0 + ring.stage * (S::kStage / 16), b = b0 + ring.stage * (S::kStage / 16);
        if (elect_one()) {
          // K = 32 each; columns past k are zeros in both operands.
          mma<false, true>(d, a, b, idesc, 0);
          mma<false, true>(d, a + 2, b + 2, idesc, 1);
          mma<false, true>(d, a + 4, b + 4, idesc, 1);
          mma<false, true>(d, a + 6, b + 6, idesc, 1);
          commit<false>(&c.empty[ring.stage]);
          commit<false>(&c.acc_full[use & 1]);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) {
      tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp == 3) {
    // Scales: k-block number `use` goes to slot use % kSlots.
    int64_t use = 0;
    bool ok = true;
    const auto ready = [&](int64_t u) {  // multiplies what this lane has brought, and hands the slot over
      const int s = (int)(u % kSlots);
      const float w = sc.weight[s][lane], x0 = sc.slot[s][lane], x1 = sc.slot[s][32 + lane];
      float p0 = x0 * w, p1 = x1 * w;
      bool far = false;
      if (__any_sync(0xffffffffu, !near_one(p0) || !near_one(p1))) {
        far = far_slot(sc.first[s] + lane, sc.again[s] + lane, x0, x1, w);
        p0 = far ? 0.f : p0;
        p1 = far ? 0.f : p1;
      }
      sc.slot[s][lane] = p0;
      sc.slot[s][32 + lane] = p1;
      if (lane == 0) sc.far[s] = far;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.full[s]);
    };
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const float* ws = g.w_scale + ((int64_t)m.expert * ((g.n - 1) / 128 + 1) + m.f0 / 128) * blocks;
      const float* xs = g.x_scale + m.row;
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        const int s = (int)(use % kSlots);
        ok = wait_warp(&sc.empty[s], (uint32_t)((use / kSlots) & 1) ^ 1u, g.err, &c.abort);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 64; k += 32)
          if (k + lane < m.rows) copy_4(&sc.slot[s][k + lane], xs + (int64_t)kb * g.ld_x_scale + k + lane);
          else sc.slot[s][k + lane] = 1.f;  // (no row: nothing that counts as far)
        copy_4(&sc.weight[s][lane], ws + kb);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (use >= kAhead) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
          ready(use - kAhead);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok)
      for (int64_t u = use < kAhead ? 0 : use - kAhead; u < use; ++u) ready(u);
  } else if (warp >= 4) {
    // A quarter of the lanes, and one of two blocks of 32 columns.
    const int q = warp & 3, group = (warp - 4) >> 2;
    uint32_t use = 0;
    bool ok = true;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const int f = m.f0 + 32 * q;
      f32x2 sum[16] = {};  // pairs
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        const uint32_t s = use % kSlots;
        ok = wait_warp(&sc.full[s], use / kSlots & 1u, g.err, &c.abort) &&
             wait_acc(c, use, g.err);
        if (!ok) break;
        if (32 * group < m.n) {
          const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (use & 1) * kAccCols + 32u * group;
          const int far = sc.far[s];
          uint32_t v[32];
          tmem_ld_32x32b_x32(at, v);
          tmem_ld_wait();
          add_block(sum, v, &sc.slot[s][32 * group]);
          if (__any_sync(0xffffffffu, far))
            in_memory(sum, [&](f32x2* to) { add_far_block(to, at, &sc.first[s][32 * group], &sc.again[s][32 * group]); });
        }
        release_acc<false>(c, use & 1, 0, lane);
        if (lane == 0) mbar_arrive(&sc.empty[s]);
      }
      if (!ok) break;
      if constexpr (V::kSplit) {
        // The operand stages are free: this tile's MMAs were the last.
        if (group * 32 < m.n)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            reinterpret_cast<float*>(smem)[(q * V::kMaxN + group * 32 + k) * 32 + lane] =
                k & 1 ? high(sum[k / 2]) : low(sum[k / 2]);
      } else {
        const int col = f + lane % 4 * 8, inside = g.n - col;
        O* y = static_cast<O*>(g.y) + (int64_t)m.row * g.ldy + col;
        by_rows<1, 8, 2>(
            reinterpret_cast<float*>(smem + V::kStages * S::kStage + (warp - 4) * kStaging8), lane, m.rows, group,
            [&](int, int k) { return k & 1 ? high(sum[k / 2]) : low(sum[k / 2]); },
            [&](int r, const float (&v)[8]) { store_8(y + r * g.ldy, inside, v); });
      }
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x)
      Store<O>::zero_row(p, z < head ? z : off[g.n_experts] + z - head, (int)threadIdx.x - 128);
  }
  if constexpr (V::kSplit) {
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && unit < tiles)
      Store<O>::template join<V>(p, mm_tile<V, kBM>(unit, f_tiles, g.n_experts, off, first), part_k, smem);
    __syncwarp();
  }
  teardown<V>(c, warp);
}

// ---------------------------------------------------------------------------- many rows
// Tiles of y itself: 128 rows of one expert (x, operand A) by up to 256 columns (the weight, operand B).  An
// accumulator lane is then a row of y and its scale one value of the thread's, where tiles of y^T need one
// for each column out of shared memory, whose bandwidth the MMAs want for their operands (98304 rows,
// 1408 -> 2048: 501 us with those, 335 with these).  The operands bound them, 48 KB a k-block out of L2 (273 us
// with nothing read from the accumulators, 12.6 TB/s), and on top of that adding up the accumulators (loads of
// them alone 313, multiply-adds alone 319); the MMAs themselves would take 150.  On pairs of CTAs, which load a
// third less, the same takes 364 us, as a k-block waits for two epilogues.
constexpr int kRowStage = 2048;  // bytes of each epilogue warp: 64 bytes of its 32 rows
constexpr int kGroup = 8;        // k-blocks whose scales come together
constexpr int kGroups = 3;

struct Rows8 {
  static constexpr int kTileRows = kBM, kTileCols = 256, kStages = 3;
  static constexpr int kStage = kABytes + kTileCols * 128;
};

struct RowScales {
  float x[kGroups][kGroup][kBM];
  float w[kGroups][2][kGroup];  // of the tile's two blocks of 128 columns
  int far[kGroups];  // whether a product of theirs may be far from 1
  uint64_t full[kGroups], empty[kGroups];
};

// The tile's rows row .. row + rows - 1 of expert `expert` and its first column.
struct RowTile {
  int expert = 0, row, rows, f0;
};
// Tiles are asked for in ascending order: the search for the expert goes on from the last one's.
template <int kRows>
__device__ __forceinline__ void row_tile(RowTile& m, uint32_t t, uint32_t f_tiles, const int32_t* off,
                                         const int32_t* first) {
  const int rt = (int)(t / f_tiles);
  int lo = m.expert;  // first[lo] <= rt < first[lo + 1]
  while (first[lo + 1] <= rt) ++lo;
  // Groups of 8 row tiles, in each every column tile, in each the group's row tiles (as mm_tile).
  const uint32_t tiles = (uint32_t)(first[lo + 1] - first[lo]);
  uint32_t rest = t - (uint32_t)first[lo] * f_tiles;
  const uint32_t group = rest / (8 * f_tiles) * 8, size = min(8u, tiles - group);
  rest -= group * f_tiles;
  const uint32_t f = rest / size, r = group + rest - f * size;
  m.expert = lo;
  m.row = off[lo] + (int)(r * kRows);
  m.rows = min(kRows, off[lo + 1] - m.row);
  m.f0 = (int)f * 256;
}

// 16 bytes of results: vectors of O.
template <typename O>
__device__ __forceinline__ uint4 pack_16(const f32x2* v) {
  const float2 a = parts(v[0]), b = parts(v[1]);
  if constexpr (sizeof(O) == 4) {
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    const float2 c = parts(v[2]), d = parts(v[3]);
    return make_uint4(pack_2<O>(a.x, a.y), pack_2<O>(b.x, b.y), pack_2<O>(c.x, c.y), pack_2<O>(d.x, d.y));
  }
}

// sum += the lane's row of `count` accumulators from use number `use` on, 128 columns from `at` on (in the first of the
// two), times both factors of their scales.  Out of line, the sums in memory: the ordinary case has no registers for
// it.  False where a wait gave up.
static __device__ __noinline__ bool add_far_group(f32x2* sum, Control& c, uint32_t use, int count, uint32_t at, bool on,
                                                  const float* x, const float* w, int lane, int* err) {
#pragma unroll 1
  for (int i = 0; i < count; ++i, ++use) {
    if (!wait_acc(c, use, err)) return false;
    const Factors f = factors(x[i * kBM], w[i]);
    const f32x2 first = pair(f.first, f.first), again = pair(f.again, f.again);
#pragma unroll 1
    for (int h = 0; on && h < 128; h += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(at + (use & 1) * kAccCols + h, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; k += 2)
        sum[(h + k) / 2] = fma2(mul2(mul2(pair_of(v + k), first), again), again, sum[(h + k) / 2]);
    }
    release_acc<false>(c, use & 1, 0, lane);
  }
  return true;
}

template <typename O>
__global__ void __launch_bounds__(kThreads, 1) fp8_rows_kernel(const __grid_constant__ Fp8Params p) {
  using V = Rows8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ RowScales sc;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Fp8Mm& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 96) {
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.x);
  }
  if (threadIdx.x == 0)
    for (int s = 0; s < kGroups; ++s) {
      mbar_init(&sc.full[s], 1);
      mbar_init(&sc.empty[s], kEpiWarps);
    }
  setup<false>(c, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kTileRows, lane, first);
  __syncthreads();
  sync_ctas<false>();
  const uint32_t tmem = c.tmem;
  const uint32_t f_tiles = (uint32_t)(g.n - 1) / 256 + 1, tiles = (uint32_t)first[g.n_experts] * f_tiles;
  const int blocks = (g.k - 1) / kBK8 + 1;
  // The MMA's N: the tile's columns in steps of 32.
  const auto columns = [&](const RowTile& m) { return min(256, (g.n - m.f0 + 31) / 32 * 32); };

  if (warp == 0) {
    Ring<V::kStages> ring;
    int64_t fills = 0;
    bool ok = true;
    const uint32_t full0 = smem_u32(c.full), dst0 = smem_u32(smem);
    RowTile m;
    for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      row_tile<V::kTileRows>(m, t, f_tiles, off, first);
      const int boxes = (columns(m) + 63) / 64;
      for (int kb = 0; kb < blocks; ++kb, ++fills) {
        ok = wait_warp(&c.empty[ring.stage], ring.phase ^ 1u, g.err, &c.abort);
        if (!ok) break;
        const uint32_t sig = full0 + 8 * ring.stage, a = dst0 + ring.stage * V::kStage;
        if (elect_one()) {
          expect(sig, kABytes + boxes * kBox);
          load_2d<false>(a, &p.x, kb * kBK8, m.row, sig);
#pragma unroll
          for (int b = 0; b < V::kTileCols / 64; ++b)
            if (b < boxes) load_3d<false>(a + kABytes + b * kBox, &p.w, kb * kBK8, m.f0 + 64 * b, m.expert, sig);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) drain_ring<V>(c, fills, 0, g.err);
    __syncwarp();
  } else if (warp == 1) {
    Ring<V::kStages> ring;
    uint32_t use = 0;
    bool ok = true;
    const uint32_t a0 = desc_lo(smem_u32(smem), 16), b0 = desc_lo(smem_u32(smem) + kABytes, 16);
    RowTile m;
    for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      row_tile<V::kTileRows>(m, t, f_tiles, off, first);
      const uint32_t idesc = idesc_16(false, V::kTileRows, columns(m), 0, 0);  // e4m3 has the same code as fp16
      for (int kb = 0; kb < blocks; ++kb, ++use) {
        ok = wait_warp(&c.acc_empty[use & 1], (use >> 1 & 1u) ^ 1u, g.err, &c.abort) &&
             wait_warp(&c.full[ring.stage], ring.phase, g.err, &c.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (use & 1) * kAccCols;
        const uint32_t a = a0 + ring.stage * (V::kStage / 16), b = b0 + ring.stage * (V::kStage / 16);
        if (elect_one()) {
          mma<false, true>(d, a, b, idesc, 0);
          mma<false, true>(d, a + 2, b + 2, idesc, 1);
          mma<false, true>(d, a + 4, b + 4, idesc, 1);
          mma<false, true>(d, a + 6, b + 6, idesc, 1);
          commit<false>(&c.acc_full[use & 1]);
          commit<false>(&c.empty[ring.stage]);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) {
      tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp == 3) {
    // Scales, kGroup k-blocks at a time.  A group is handed over when the next one has been asked for.
    uint32_t use = 0;
    bool ok = true;
    const auto ready = [&](uint32_t u) {
      // The largest and the smallest magnitudes (but 0) of what this lane has brought, and of all.
      const uint32_t s = u % kGroups, inf = 0x7f800000u;
      uint32_t x_most = 0, x_least = inf, w_most = 0, w_least = inf;
      const auto look = [&](float v, uint32_t& most, uint32_t& least) {
        const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
        most = max(most, b);
        least = b == 0 ? least : min(least, b);
      };
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
#pragma unroll
        for (int r = 0; r < kBM; r += 32) look(sc.x[s][i][r + lane], x_most, x_least);
      if (lane < 2 * kGroup) look(sc.w[s][lane / kGroup][lane % kGroup], w_most, w_least);
      const auto most = [](uint32_t v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, v)); };
      const auto least = [](uint32_t v) { return __uint_as_float(__reduce_min_sync(0xffffffffu, v)); };
      const float high = most(x_most) * most(w_most), low = least(x_least) * least(w_least);
      if (lane == 0) sc.far[s] = !(high <= kNearOne && low >= 1.f / kNearOne);
      __syncwarp();  // every lane's copies have landed
      if (lane == 0) mbar_arrive(&sc.full[s]);
    };
    const int64_t n_blocks = (g.n - 1) / 128 + 1;
    RowTile m;
    for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      row_tile<V::kTileRows>(m, t, f_tiles, off, first);
      const float* xs = g.x_scale + m.row;
      for (int kb = 0; kb < blocks; kb += kGroup, ++use) {
        const uint32_t s = use % kGroups;
        ok = wait_warp(&sc.empty[s], (use / kGroups & 1u) ^ 1u, g.err, &c.abort);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int r = 0; r < kBM; r += 32) {
            float* to = &sc.x[s][i][r + lane];
            if (kb + i < blocks && r + lane < m.rows) copy_4(to, xs + (int64_t)(kb + i) * g.ld_x_scale + r + lane);
            else *to = 0.f;
          }
        const int half = lane / kGroup, b = lane % kGroup;
        if (half < 2) {
          float* to = &sc.w[s][half][b];
          if (kb + b < blocks && m.f0 / 128 + half < n_blocks)
            copy_4(to, g.w_scale + ((int64_t)m.expert * n_blocks + m.f0 / 128 + half) * blocks + kb + b);
          else *to = 0.f;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (use > 0) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          ready(use - 1);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok && use > 0) ready(use - 1);
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;  // a quarter of the lanes, 128 columns
    uint4* stage = reinterpret_cast<uint4*>(smem + V::kStages * V::kStage + (warp - 4) * kRowStage);
    uint32_t use = 0, groups = 0;
    bool ok = true;
    RowTile m;
    for (uint32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      row_tile<V::kTileRows>(m, t, f_tiles, off, first);
      const bool on = 128 * half < columns(m);
      f32x2 sum[64];
#pragma unroll
      for (int k = 0; k < 64; ++k) sum[k] = 0;
      const uint32_t at0 = tmem + ((uint32_t)(32 * q) << 16) + 128u * half;
      for (int kb = 0; kb < blocks; kb += kGroup, ++groups) {
        const uint32_t s = groups % kGroups;
        ok = wait_warp(&sc.full[s], groups / kGroups & 1u, g.err, &c.abort);
        if (!ok) break;
        const int count = min(kGroup, blocks - kb);
        if (__any_sync(0xffffffffu, sc.far[s])) {
          in_memory(sum, [&](f32x2* to) {
            ok = add_far_group(to, c, use, count, at0, on, &sc.x[s][0][32 * q + lane], sc.w[s][half], lane, g.err);
          });
          use += count;
        } else {
          for (int i = 0; i < count; ++i, ++use) {
            ok = wait_acc(c, use, g.err);
            if (!ok) break;
            if (on) {
              const float scale = sc.x[s][i][32 * q + lane] * sc.w[s][half][i];
              const f32x2 both = pair(scale, scale);
              const uint32_t at = at0 + (use & 1) * kAccCols;
#pragma unroll
              for (int h = 0; h < 128; h += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(at + h, v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; k += 2) sum[(h + k) / 2] = fma2(pair_of(v + k), both, sum[(h + k) / 2]);
              }
            }
            release_acc<false>(c, use & 1, 0, lane);
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sc.empty[s]);
      }
      if (!ok) break;
      if (!on) continue;
      // 64 bytes of the warp's 32 rows at a time, so that a store covers whole sectors of 8 rows: 16-byte
      // chunk c of row r stands in slot c ^ (r / 2 % 4), free of bank conflicts.
      constexpr int kValues = 16 / (int)sizeof(O), kPasses = 128 / (4 * kValues);
      const int left = m.rows - 32 * q;
      O* y = static_cast<O*>(g.y) + ((int64_t)m.row + 32 * q) * g.ldy;
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          stage[4 * lane + (ch ^ (lane >> 1 & 3))] = pack_16<O>(&sum[(pass * 4 + ch) * kValues / 2]);
        __syncwarp();
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 8) {
          const int r = r0 + lane / 4, ch = lane % 4;
          const uint4 v = stage[4 * r + (ch ^ (r >> 1 & 3))];
          const int col = m.f0 + 128 * half + (pass * 4 + ch) * kValues, inside = g.n - col;
          if (r >= left || inside <= 0) continue;
          O* at = y + r * g.ldy + col;
          if (inside >= kValues && reinterpret_cast<uintptr_t>(at) % 16 == 0) {
            *reinterpret_cast<uint4*>(at) = v;
          } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < kValues; ++k) {
              if (k >= inside) break;
              if constexpr (sizeof(O) == 4) reinterpret_cast<uint32_t*>(at)[k] = w[k];
              else reinterpret_cast<uint16_t*>(at)[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
            }
          }
        }
      }
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x)
      Store<O>::template zero_row<kEpiWarps>(p, z < head ? z : off[g.n_experts] + z - head,
                                             (int)threadIdx.x - 128);
  }
  sync_ctas<false>();
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
}

template <typename O>
cudaError_t launch_rows(const Fp8Params& p, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  // At least as many tiles as the offsets can make of the rows.
  const int64_t tiles = (p.g.rows / Rows8::kTileRows + (p.g.rows < p.g.n_experts ? p.g.rows : p.g.n_experts)) *
                        (((int64_t)p.g.n - 1) / Rows8::kTileCols + 1);
  return launch(fp8_rows_kernel<O>, p, tiles, 1, sms,
                Rows8::kStages * Rows8::kStage + kEpiWarps * kRowStage + 1024, &ready, st);
}

template <typename V, typename O>
cudaError_t launch_as(const Fp8Params& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  return launch(fp8_mm_kernel<V, O>, p, mm_tiles<V>(p.g), parts, sms,
                V::kStages * Shape<V>::kStage + (V::kSplit ? 0 : kEpiWarps * kStaging8) + 1024, &ready, st);
}

template <typename O>
cudaError_t launch_type(const Fp8Params& p, int parts, bool narrow, int sms, cudaStream_t st) {
  return parts > 1 ? launch_as<Split8, O>(p, parts, sms, st)
         : narrow  ? launch_as<Narrow8, O>(p, 1, sms, st) : launch_rows<O>(p, sms, st);
}

}  // namespace

cudaError_t launch_fp8_mm(const Fp8Mm& g, int sms, cudaStream_t st) {
  Fp8Params p;
  p.g = g;
  // (The pitch of a single row means nothing: one that TMA takes.)
  const int64_t line = ((int64_t)g.k + 15) / 16 * 16;
  const Operand x{g.x, g.rows, g.k, g.rows == 1 ? line : g.ldx, 1, 0};
  const Operand w{g.w, g.n, g.k, g.n == 1 ? line : g.ldw, g.n_experts, g.w_stride};
  // The rules of the 16-bit products (see choose_tiles), and tiles of y itself where those take wide ones.
  int parts = 1;
  while (parts < kMostParts && mm_tiles<Split8>(g) * parts * 2 <= sms && g.k >= 4 * kBK8 * parts * 2) parts *= 2;
  const bool narrow = g.rows <= Narrow8::kMaxN * (int64_t)g.n_experts || mm_tiles<Narrow8>(g) <= sms;
  const bool few = parts > 1 || narrow;
  cudaError_t e = encode(&p.x, x, kE4m3, false, few ? Narrow8::kBoxRows : kBM);
  if (e == cudaSuccess) e = encode(&p.w, w, kE4m3, true, few ? kBM : 64);
  if (e != cudaSuccess) return e;
  return g.out_dtype == kF32 ? launch_type<float>(p, parts, narrow, sms, st)
         : g.out_dtype == kBf16 ? launch_type<__nv_bfloat16>(p, parts, narrow, sms, st)
                                : launch_type<__half>(p, parts, narrow, sms, st);
}

}  // namespace muon
