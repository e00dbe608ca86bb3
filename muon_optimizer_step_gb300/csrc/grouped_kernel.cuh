// The kernel of the products grouped by expert (see grouped_mm.cu), over what it does with a tile:
// an Op says which tensor maps the loads take (Params, x_map, w_map; kPasses: products whose sums are
// added; kGated: two weights, 64 columns of each in a tile's 128 lanes), how many columns of the result a
// CTA's tile is wide (kCols), whether sums are kept in short segments (fine), how many warps the epilogue has
// (kWarps) and what becomes of the accumulators (agree: whether warps that finish a tile together all have
// it; finish; join for tiles that a cluster shares; zero_row).
//
// kFromTmem: a tile's sums go back into TMEM, over its last segment, and finish takes them from there a few
// columns at a time.  With all sums in registers an epilogue that computes a lot beside them spills, and what
// spills has no L1 to go to beside the stages (98304 x 2048 -> 1408 backward: 1706 us with, 633 without).
// kKeep: the last block of a warp's columns stays in registers, so that the accumulator is handed back
// earlier, where the epilogue has them to spare (4096 x 4096 -> 14336 forward: 531 -> 526 us).
#pragma once

#include "grouped_tiles.cuh"

namespace muon {

// The variant with as many stages as the shared memory beside an Op's staging holds (what is left
// of 227 KB are the barriers and the experts' offsets).
template <typename V, int kStaging>
struct Fit : V {
  static constexpr int kRoom = (217 * 1024 - kStaging) / Shape<V>::kStage;
  static constexpr int kStages = kRoom < V::kStages ? kRoom : V::kStages;
};

// Writes 16 accumulator columns of this warp's lanes.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <typename V, typename Op>
__global__ void __launch_bounds__(128 + 32 * Op::kWarps, 1)
grouped_mm_kernel(const __grid_constant__ typename Op::Params p) {
  using S = Shape<V>;
  constexpr int kCols = Op::kCols;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const auto& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = V::kPair ? cluster_ctarank() : 0u;
  const Part part_k = split_part<V>();
  if (threadIdx.x == 96) {  // warp 3: off the other warps' way
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.x);
  }
  setup<V::kPair, Op::kWarps>(c, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kMaxN, lane, first);
  __syncthreads();
  sync_ctas<V::kPair>();
  const uint32_t tmem = c.tmem;
  const uint32_t f_tiles = (uint32_t)(g.n - 1) / (kCols * S::kCtas) + 1, tiles = (uint32_t)first[g.n_experts] * f_tiles;
  const int pass_blocks = (g.k - 1) / kBK + 1;
  int kb0 = 0, kb1 = Op::kPasses * pass_blocks;  // this CTA's k-blocks
  uint32_t unit = blockIdx.x / S::kCtas, units = gridDim.x / S::kCtas;
  if constexpr (V::kSplit) {
    const int all = kb1;  // parts is a power of two
    const int shift = 31 - __clz(part_k.parts);
    kb0 = (int)((int64_t)all * part_k.index >> shift);
    kb1 = (int)((int64_t)all * (part_k.index + 1) >> shift);
    unit >>= shift;
    units >>= shift;
  }
  const int seg = segment_blocks(kb1 - kb0, Op::fine(p) ? V::kSegment32 : V::kSegment16, V::kSub);

  if (warp == 0) {
    Ring<V::kStages> ring;
    int64_t fills = 0;
    bool ok = true;
    const uint32_t full0 = smem_u32(c.full), dst0 = smem_u32(smem);
    // A pair's second CTA signals the first one's barriers.
    const uint32_t sig0 = V::kPair ? mapa_shared(full0, 0) : full0;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kCols>(t, f_tiles, g.n_experts, off, first);
      const int part = m.n / S::kCtas;  // rows of x this CTA brings
      const int boxes = (part + V::kBoxRows - 1) / V::kBoxRows;
      const uint32_t bytes = S::kCtas * (kABytes + boxes * V::kBoxRows * 128);
      const int f = m.f0 + kCols * (int)rank, row = (int)((uint32_t)m.row + part * rank);
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
            const bool second = Op::kPasses > 1 && kb + j >= pass_blocks;
            const int k0 = (kb + j - (second ? pass_blocks : 0)) * kBK;
            const uint32_t aj = a + j * S::kBlock;
            const CUtensorMap *x = Op::x_map(p, second), *w = Op::w_map(p, second);
            if constexpr (Op::kGated) {
              // 64 columns of each weight: both majors are boxes of 64 lines.
              const int across = g.trans ? k0 : f, down = g.trans ? f : k0;
              load_3d<V::kPair>(aj, w, across, down, m.expert, sig);
              load_3d<V::kPair>(aj + kBox, Op::w_map(p, true), across, down, m.expert, sig);
            } else if (g.trans) {
              load_3d<V::kPair>(aj, w, k0, f, m.expert, sig);
            } else {
              load_3d<V::kPair>(aj, w, f, k0, m.expert, sig);
              load_3d<V::kPair>(aj + kBox, w, f + 64, k0, m.expert, sig);
            }
#pragma unroll
            for (int b = 0; b < V::kMaxN / S::kCtas / V::kBoxRows; ++b)
              if (b < boxes)
                load_2d<V::kPair>(aj + kABytes + b * V::kBoxRows * 128, x, k0,
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
      const MmTile m = mm_tile<V, kCols>(t, f_tiles, g.n_experts, off, first);
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
    // A quarter of the lanes, every kGroups-th block of 32 columns.
    constexpr int kGroups = Op::kWarps / 4, kBlocks = (V::kMaxN / 32 + kGroups - 1) / kGroups;
    const int q = warp & 3, group = (warp - 4) >> 2;
    int use = 0;
    bool ok = true;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kCols>(t, f_tiles, g.n_experts, off, first);
      float sum[kBlocks][32];
      if constexpr (Op::kFromTmem) {  // (or the last tile's would be kept through its epilogue)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int k = 0; k < 32; ++k) sum[i][k] = 0.f;
      }
      for (int kb = kb0; kb < kb1; kb += seg, ++use) {
        ok = wait_acc(c, use, g.err);
        if (!ok) break;
        const bool last = Op::kFromTmem && !V::kSplit && kb + seg >= kb1;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int col = (kGroups * i + group) * 32;
          const bool back = last && (kBlocks == 1 || !Op::kKeep || i < kBlocks - 1);
          // (One segment's sums are in TMEM already.)
          if (col >= m.n || (back && kb == kb0)) continue;
          add_acc<kGroups == 2>(tmem, use & 1, q, col, kb == kb0, sum[i]);
          if (back) {
            const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)((use & 1) * kAccCols + col);
            tmem_st_32x32b_x16(at, sum[i]);
            tmem_st_32x32b_x16(at + 16, sum[i] + 16);
          }
        }
        if (last) tmem_st_wait();
        else release_acc<V::kPair>(c, use & 1, rank, lane);
      }
      ok = Op::agree(q, group, ok);
      if (!ok) break;
      if constexpr (V::kSplit) {
        // The operand stages are free: this tile's MMAs were the last.
        if (group * 32 < m.n)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            reinterpret_cast<float*>(smem)[(q * V::kMaxN + group * 32 + k) * 32 + lane] = sum[0][k];
      } else if constexpr (Op::kFromTmem) {
        const int ab = (use - 1) & 1;
        bool held = true;
        Op::template finish<V, kBlocks>(
            p, m, m.f0 + kCols * (int)rank, q, group, lane,
            tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kAccCols), sum[kBlocks - 1],
            [&] {
              release_acc<V::kPair>(c, ab, rank, lane);
              held = false;
            },
            smem + V::kStages * S::kStage);
        if (held) release_acc<V::kPair>(c, ab, rank, lane);
      } else {
        Op::template finish<V>(p, m, m.f0 + kCols * (int)rank, q, group, lane, sum,
                               smem + V::kStages * S::kStage);
      }
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x) {
      Op::zero_row(p, z < head ? z : off[g.n_experts] + z - head, (int)threadIdx.x - 128);
    }
  }
  if constexpr (V::kSplit) {
    // The parts of the tile are in the CTAs' shared memory, as [quarter][row of y][column]:
    // every CTA adds and stores a share, the parts in order.
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && unit < tiles) {
      const MmTile m = mm_tile<V, kCols>(unit, f_tiles, g.n_experts, off, first);
      Op::template join<V>(p, m, part_k, smem);
    }
    __syncwarp();
  }
  teardown<V>(c, warp);
}

// The sums of 8 neighbouring lanes (columns `col` .. + 7 of a tile's 128) for its row r, over the parts
// of a tile that a cluster shares, in order.
template <typename V>
__device__ __forceinline__ void join_parts(uint8_t* smem, int parts, int r, int col, float (&sum)[8]) {
  const uint32_t at = smem_u32(smem) + ((col / 32 * V::kMaxN + r) * 32 + col % 32) * 4;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = 0.f;
  for (int q = 0; q < parts; ++q) {
    float v[8];
    const uint32_t from = mapa_shared(at, q);
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(from) : "memory");
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(from + 16) : "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += v[k];
  }
}

// Stores 8 values to dst on, `left` of them inside the row.
template <typename O>
__device__ __forceinline__ void store_8(O* dst, int left, const float (&v)[8]) {
  if (left >= 8 && reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
    if constexpr (sizeof(O) == 4) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_2<O>(v[0], v[1]), pack_2<O>(v[2], v[3]),
                                                  pack_2<O>(v[4], v[5]), pack_2<O>(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) put(&dst[k], v[k]);
  }
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

// A warp's accumulators turned around, kLines (8 or 16) rows of its 32 columns at a time: in the
// accumulators a lane has one column, behind `stage` (kLines x 32 floats) eight columns of a row, so that
// results and what is read beside them move in 16-byte units.  16-byte chunk c of line r stands in slot
// c ^ (r & 7), free of bank conflicts both ways.  The loop over the chunks is not unrolled, only the
// choice of the registers to store.
__device__ __forceinline__ void put_line(float* stage, int lane, int k, float v) {
  stage[32 * k + (lane ^ (k & 7) << 2)] = v;  // chunk lane / 4, element lane % 4
}
// Columns 8 (lane % 4) .. + 7 of a line.
__device__ __forceinline__ void get_line(const float* stage, int lane, int line, float (&v)[8]) {
  const float4* at = reinterpret_cast<const float4*>(stage + 32 * line);
  const float4 a = at[(lane % 4 * 2) ^ (line & 7)], b = at[(lane % 4 * 2 + 1) ^ (line & 7)];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// Stores chunk `c` of the accumulators (value(i, k): row k of block i) to the stage.
template <int kBlocks, int kLines, typename F>
__device__ __forceinline__ void put_chunk(float* stage, int lane, int c, const F& value) {
#pragma unroll
  for (int cc = 0; cc < kBlocks * 32 / kLines; ++cc)
    if (cc == c)
#pragma unroll
      for (int k = 0; k < kLines; ++k) put_line(stage, lane, k, value(cc * kLines / 32, cc * kLines % 32 + k));
}
// The same of 16, or 8, accumulator columns in TMEM.
__device__ __forceinline__ void put_tmem_16(float* stage, int lane, uint32_t taddr) {
  uint32_t v[16];
  tmem_ld_32x32b_x16(taddr, v);
  tmem_ld_wait();
#pragma unroll
  for (int k = 0; k < 16; ++k) put_line(stage, lane, k, __uint_as_float(v[k]));
}
__device__ __forceinline__ void put_tmem_8(float* stage, int lane, uint32_t taddr) {
  uint32_t v[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr)
      : "memory");
  tmem_ld_wait();
#pragma unroll
  for (int k = 0; k < 8; ++k) put_line(stage, lane, k, __uint_as_float(v[k]));
}
// First row of chunk c of a warp that has every kGroups-th block of 32 rows.
template <int kLines, int kGroups>
__device__ __forceinline__ int chunk_row(int c, int group) {
  return (kGroups * (c * kLines / 32) + group) * 32 + c * kLines % 32;
}
// f(row, eight values) for the lane's part of each of the tile's rows.
template <int kBlocks, int kLines, int kGroups, typename G, typename F>
__device__ __forceinline__ void by_rows(float* stage, int lane, int rows, int group, const G& value, const F& f) {
#pragma unroll 1
  for (int c = 0; c < kBlocks * 32 / kLines; ++c) {
    const int r0 = chunk_row<kLines, kGroups>(c, group);
    if (r0 >= rows) break;
    __syncwarp();
    put_chunk<kBlocks, kLines>(stage, lane, c, value);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kLines; j += 8) {
      const int line = j + lane / 4;
      float v[8];
      get_line(stage, lane, line, v);
      if (r0 + line < rows) f(r0 + line, v);
    }
  }
}

// What products do whose result is stored as it is, in type O.
template <typename O>
struct Store {
  static constexpr bool kGated = false;
  static constexpr int kCols = kBM, kStaging = 0, kWarps = kEpiWarps;
  static constexpr bool kFromTmem = false, kKeep = false;
  static __device__ __forceinline__ bool agree(int, int, bool ok) { return ok; }
  template <typename P>
  static __device__ __forceinline__ bool fine(const P&) { return sizeof(O) == 4; }

  template <typename V, typename P>
  static __device__ __forceinline__ void finish(const P& p, const MmTile& m, int f, int q, int half,
                                                int lane, const float (&sum)[Shape<V>::kBlocks][32],
                                                uint8_t*) {
#pragma unroll
    for (int i = 0; i < Shape<V>::kBlocks; ++i)
      if ((2 * i + half) * 32 < m.n) mm_store<O>(p.g, m, 2 * i + half, f + 32 * q, lane, sum[i]);
  }

  template <typename V, int kWarps = kEpiWarps, typename P>
  static __device__ __forceinline__ void join(const P& p, const MmTile& m, const Part& part,
                                              uint8_t* smem) {
    const int cols = p.g.n - m.f0;
    for (int i = threadIdx.x - 128 + part.index * kWarps * 32; i < m.rows * 16;
         i += part.parts * kWarps * 32) {
      const int r = i / 16, col = i % 16 * 8;
      float sum[8];
      join_parts<V>(smem, part.parts, r, col, sum);
      store_8(static_cast<O*>(p.g.y) + (int64_t)(m.row + r) * p.g.ldy + m.f0 + col, cols - col, sum);
    }
  }

  template <int kWarps = kEpiWarps, typename P>
  static __device__ __forceinline__ void zero_row(const P& p, int64_t row, int thread) {
    O* at = static_cast<O*>(p.g.y) + row * p.g.ldy;
    for (int64_t f = thread; f < p.g.n; f += kWarps * 32) put(&at[f], 0.f);
  }
};

struct MmParams {
  CUtensorMap x;   // (k, rows): boxes of 64 x kBoxRows
  CUtensorMap w;   // (inner, outer, expert): boxes of 64 x 128 (trans) or 64 x 64
  GroupedMm g;
};

// y = x W_e.
template <typename O>
struct Plain : Store<O> {
  using Params = MmParams;
  static constexpr int kPasses = 1;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool) { return &p.x; }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool) { return &p.w; }
};

// ---------------------------------------------------------------------------- launches
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
struct MmChoice {
  int parts;
  bool narrow, pair;
  uint32_t box_rows() const { return parts > 1 || narrow ? Narrow::kBoxRows : Wide::kBoxRows; }
};
template <typename Op>
MmChoice choose_tiles(const GroupedMm& g, bool fine, int sms) {
  MmChoice c{1, false, false};
  while (c.parts < kMostParts && mm_tiles<Split>(g, Op::kCols) * c.parts * 2 <= sms &&
         (int64_t)Op::kPasses * g.k >= 4 * kBK * c.parts * 2)
    c.parts *= 2;
  c.narrow = g.rows <= Narrow::kMaxN * (int64_t)g.n_experts || mm_tiles<Narrow>(g, Op::kCols) <= sms;
  c.pair = !c.narrow && !fine && g.n > Op::kCols && mm_tiles<Pair>(g, Op::kCols) >= sms;
  return c;
}

template <typename W, typename Op>
cudaError_t launch_op(const typename Op::Params& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  constexpr int kStaging = W::kSplit ? 0 : Op::kStaging;
  using V = Fit<W, kStaging>;
  return launch(grouped_mm_kernel<V, Op>, p, mm_tiles<V>(p.g, Op::kCols), Shape<V>::kCtas * parts, sms,
                V::kStages * Shape<V>::kStage + kStaging + 1024, &ready, st, 128 + 32 * Op::kWarps);
}

// kPairs: whether results of this type ever run on pairs.
template <typename Op, bool kPairs>
cudaError_t launch_tiles(const typename Op::Params& p, const MmChoice& c, int sms, cudaStream_t st) {
  if (c.parts > 1) return launch_op<Split, Op>(p, c.parts, sms, st);
  if (c.narrow) return launch_op<Narrow, Op>(p, 1, sms, st);
  if constexpr (kPairs)
    if (c.pair) return launch_op<Pair, Op>(p, 1, sms, st);
  return launch_op<Wide, Op>(p, 1, sms, st);
}

}  // namespace muon
