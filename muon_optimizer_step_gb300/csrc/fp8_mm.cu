// Products of 8-bit operands (e4m3) grouped by expert, with a scale for each 128 columns of a row of x and
// for each block of 128 x 128 of a weight.
//
//   y[r, c] = sum over the blocks b of 128 along k of
//             x_scale[b][r] w_scale[e][c / 128][b] (sum over b's k of x[r, k] w_e[c, k])
//
// Tiles of y^T as in the grouped products of 16-bit operands (see grouped_mm.cu): 128 columns of y (the
// weight, operand A) by up to kMaxN rows of one expert, on single CTAs or pairs.  A k-block is 128 bytes
// of a row, that is one block of the scales: each is an accumulator of its own, and the epilogue warps add
// it to the sums in registers, times the scale of its row of y (an accumulator column) and the weight's (the
// same for the whole tile).  So every 128 terms are summed in the tensor core, the blocks in fp32 with
// rounding to nearest.
//
// Warp 3 brings the scales: a ring of slots in shared memory, each with a k-block's scales of the tile's
// rows, loaded several k-blocks ahead (cp.async) and multiplied by the weight's when they are there.
#include "grouped_kernel.cuh"

namespace muon {

namespace {

constexpr int kBK8 = 128;   // elements of a k-block: 128 bytes
constexpr int kSlots = 8;   // of scales
constexpr int kAhead = 6;   // k-blocks that scales are asked for ahead
constexpr int kWarps8 = 16;              // of the epilogue
constexpr int kThreads8 = 128 + 32 * kWarps8;
constexpr int kStaging8 = 1024;          // bytes of each epilogue warp: 8 rows of its 32 columns

struct Fp8Params {
  CUtensorMap x, w;  // (k, rows): boxes of 128 x kBoxRows; (k, columns of y, expert): 128 x 128
  Fp8Mm g;
};

// Tile variants as for 16-bit operands (see grouped_tiles.cuh), with a k-block per stage.
struct Pair8 {
  static constexpr bool kPair = true, kSplit = false;
  static constexpr int kMaxN = 256, kBoxRows = 64, kStages = 5, kSub = 1;
};
struct Wide8 {
  static constexpr bool kPair = false, kSplit = false;
  static constexpr int kMaxN = 256, kBoxRows = 64, kStages = 4, kSub = 1;
};
struct Narrow8 {
  static constexpr bool kPair = false, kSplit = false;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 6, kSub = 1;
};
struct Split8 {
  static constexpr bool kPair = false, kSplit = true;
  static constexpr int kMaxN = 64, kBoxRows = 16, kStages = 6, kSub = 1;
};

struct Scales {
  float slot[kSlots][256];
  float weight[kSlots][32];  // the weight's scale, a copy for each lane of warp 3
  uint64_t full[kSlots], empty[kSlots];
};

__device__ __forceinline__ void copy_4(void* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// v times the scales s, two at a time, added to the sums.
__device__ __forceinline__ void add_scaled(uint64_t& sum, uint32_t v0, uint32_t v1, uint64_t s) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(sum)
      : "r"(v0), "r"(v1), "l"(s));
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// sum += 16 accumulator columns in v, times their scales from s on (16-byte aligned).
__device__ __forceinline__ void add_block(uint64_t (&sum)[16], int at, const uint32_t (&v)[16], const float* s) {
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    uint64_t x, y;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(smem_u32(s + k)));
    add_scaled(sum[at + k / 2], v[k], v[k + 1], x);
    add_scaled(sum[at + k / 2 + 1], v[k + 2], v[k + 3], y);
  }
}

template <typename V, typename O>
__global__ void __launch_bounds__(kThreads8, 1) fp8_mm_kernel(const __grid_constant__ Fp8Params p) {
  using S = Shape<V>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control c;
  __shared__ Scales sc;
  __shared__ int32_t off[kMaxExperts + 1], first[kMaxExperts + 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Fp8Mm& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = V::kPair ? cluster_ctarank() : 0u;
  const Part part_k = split_part<V>();
  if (threadIdx.x == 96) {
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.x);
  }
  if (threadIdx.x == 0)
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sc.full[s], 1);
      mbar_init(&sc.empty[s], kWarps8);
    }
  setup<V::kPair, kWarps8>(c, warp);
  load_offsets(g.offsets, g.n_experts, g.rows, off, g.err);
  if (warp == 3) count_tiles(off, g.n_experts, V::kMaxN, lane, first);
  __syncthreads();
  sync_ctas<V::kPair>();
  const uint32_t tmem = c.tmem;
  const uint32_t f_tiles = (uint32_t)(g.n - 1) / S::kM + 1, tiles = (uint32_t)first[g.n_experts] * f_tiles;
  const int blocks = (g.k - 1) / kBK8 + 1;
  int kb0 = 0, kb1 = blocks;  // this CTA's k-blocks
  uint32_t unit = blockIdx.x / S::kCtas, units = gridDim.x / S::kCtas;
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
    const uint32_t sig0 = V::kPair ? mapa_shared(full0, 0) : full0;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const int part = m.n / S::kCtas;  // rows of x this CTA brings
      const int boxes = (part + V::kBoxRows - 1) / V::kBoxRows;
      const uint32_t bytes = S::kCtas * (kABytes + boxes * V::kBoxRows * 128);
      const int f = m.f0 + kBM * (int)rank, row = (int)((uint32_t)m.row + part * rank);
      for (int kb = kb0; kb < kb1; ++kb, ++fills) {
        ok = wait_warp(&c.empty[ring.stage], ring.phase ^ 1u, g.err, &c.abort);
        if (!ok) break;
        const uint32_t sig = sig0 + 8 * ring.stage, a = dst0 + ring.stage * S::kStage;
        if (elect_one()) {
          if (rank == 0) expect(full0 + 8 * ring.stage, bytes);
          load_3d<V::kPair>(a, &p.w, kb * kBK8, f, m.expert, sig);
#pragma unroll
          for (int b = 0; b < V::kMaxN / S::kCtas / V::kBoxRows; ++b)
            if (b < boxes)
              load_2d<V::kPair>(a + kABytes + b * V::kBoxRows * 128, &p.x, kb * kBK8,
                                (int)((uint32_t)row + b * V::kBoxRows), sig);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) drain_ring<V>(c, fills, rank, g.err);
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    Ring<V::kStages> ring;
    int use = 0;
    bool ok = true;
    const uint32_t a0 = desc_lo(smem_u32(smem), 16), b0 = desc_lo(smem_u32(smem) + kABytes, 16);
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const uint32_t idesc = idesc_16(false, S::kM, m.n, 0, 0);  // e4m3 has the same code as fp16
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        ok = wait_warp(&c.acc_empty[use & 1], ((use >> 1) & 1) ^ 1u, g.err, &c.abort) &&
             wait_warp(&c.full[ring.stage], ring.phase, g.err, &c.abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (use & 1) * kAccCols;
        const uint32_t a = a0 + ring.stage * (S::kStage / 16), b = b0 + ring.stage * (S::kStage / 16);
        if (elect_one()) {
          // K = 32 each; columns past k are zeros in both operands.
          mma<V::kPair, true>(d, a, b, idesc, 0);
          mma<V::kPair, true>(d, a + 2, b + 2, idesc, 1);
          mma<V::kPair, true>(d, a + 4, b + 4, idesc, 1);
          mma<V::kPair, true>(d, a + 6, b + 6, idesc, 1);
          commit<V::kPair>(&c.empty[ring.stage]);
          commit<V::kPair>(&c.acc_full[use & 1]);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elect_one()) {
      if constexpr (V::kPair) tc_commit_pair(&c.mma_done, (uint16_t)0x1);
      else tc_commit(&c.mma_done);
      drain(&c.mma_done, 0, g.err);
    }
    __syncwarp();
  } else if (warp == 3) {
    // Scales: k-block number `use` goes to slot use % kSlots.
    int64_t use = 0;
    bool ok = true;
    const auto ready = [&](int64_t u) {  // multiplies what this lane has brought, and hands the slot over
      const int s = (int)(u % kSlots);
      const float w = sc.weight[s][lane];
#pragma unroll
      for (int k = 0; k < 256; k += 32) sc.slot[s][k + lane] *= w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.full[s]);
    };
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const int f = m.f0 + kBM * (int)rank;
      const int64_t n_blocks = (g.n - 1) / 128 + 1;
      // (A pair's second CTA may have no columns: any scale will do.)
      const float* ws = g.w_scale + ((int64_t)m.expert * n_blocks + (f < g.n ? f / 128 : 0)) * blocks;
      const float* xs = g.x_scale + m.row;
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        const int s = (int)(use % kSlots);
        ok = wait_warp(&sc.empty[s], (uint32_t)((use / kSlots) & 1) ^ 1u, g.err, &c.abort);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 256; k += 32)
          if (k + lane < m.rows) copy_4(&sc.slot[s][k + lane], xs + (int64_t)kb * g.ld_x_scale + k + lane);
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
    // A quarter of the lanes, and every fourth block of 32 columns.
    const int q = warp & 3, group = (warp - 4) >> 2;
    constexpr int kBlocks8 = (V::kMaxN + 127) / 128;
    int use = 0;
    bool ok = true;
    for (uint32_t t = unit; t < tiles && ok; t += units) {
      const MmTile m = mm_tile<V, kBM>(t, f_tiles, g.n_experts, off, first);
      const int f = m.f0 + kBM * (int)rank + 32 * q;
      uint64_t sum[kBlocks8][16];  // pairs
#pragma unroll
      for (int i = 0; i < kBlocks8; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[i][k] = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++use) {
        const int s = use % kSlots;
        ok = wait_warp(&sc.full[s], (uint32_t)(use / kSlots) & 1u, g.err, &c.abort) && wait_acc(c, use, g.err);
        if (!ok) break;
        const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)((use & 1) * kAccCols + 32 * group);
        const float* scales = &sc.slot[s][32 * group];
#pragma unroll
        for (int i = 0; i < kBlocks8; ++i) {
          if ((4 * i + group) * 32 >= m.n) continue;
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(at + 128 * i + h, v);
            tmem_ld_wait();
            add_block(sum[i], h / 2, v, scales + 128 * i + h);
          }
        }
        release_acc<V::kPair>(c, use & 1, rank, lane);
        if (lane == 0) mbar_arrive(&sc.empty[s]);
      }
      if (!ok) break;
      if constexpr (V::kSplit) {
        // The operand stages are free: this tile's MMAs were the last.
        if (group * 32 < m.n)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            reinterpret_cast<float*>(smem)[(q * V::kMaxN + group * 32 + k) * 32 + lane] =
                k & 1 ? high(sum[0][k / 2]) : low(sum[0][k / 2]);
      } else {
        const int col = f + lane % 4 * 8, inside = g.n - col;
        O* y = static_cast<O*>(g.y) + (int64_t)m.row * g.ldy + col;
        by_rows<kBlocks8, 8, 4>(
            reinterpret_cast<float*>(smem + V::kStages * S::kStage + (warp - 4) * kStaging8), lane, m.rows, group,
            [&](int i, int k) { return k & 1 ? high(sum[i][k / 2]) : low(sum[i][k / 2]); },
            [&](int r, const float (&v)[8]) { store_8(y + r * g.ldy, inside, v); });
      }
    }
    // Rows of no expert.
    const int64_t head = off[0], none = head + g.rows - off[g.n_experts];
    for (int64_t z = blockIdx.x; z < none; z += gridDim.x)
      Store<O>::template zero_row<kWarps8>(p, z < head ? z : off[g.n_experts] + z - head, (int)threadIdx.x - 128);
  }
  if constexpr (V::kSplit) {
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && unit < tiles)
      Store<O>::template join<V, kWarps8>(p, mm_tile<V, kBM>(unit, f_tiles, g.n_experts, off, first), part_k, smem);
    __syncwarp();
  }
  teardown<V>(c, warp);
}

template <typename V, typename O>
cudaError_t launch_as(const Fp8Params& p, int parts, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  return launch(fp8_mm_kernel<V, O>, p, mm_tiles<V>(p.g), Shape<V>::kCtas * parts, sms,
                V::kStages * Shape<V>::kStage + (V::kSplit ? 0 : kWarps8 * kStaging8) + 1024, &ready, st,
                kThreads8);
}

template <typename O>
cudaError_t launch_type(const Fp8Params& p, const MmChoice& c, int sms, cudaStream_t st) {
  return c.parts > 1 ? launch_as<Split8, O>(p, c.parts, sms, st)
         : c.narrow  ? launch_as<Narrow8, O>(p, 1, sms, st)
         : c.pair    ? launch_as<Pair8, O>(p, 1, sms, st) : launch_as<Wide8, O>(p, 1, sms, st);
}

}  // namespace

cudaError_t launch_fp8_mm(const Fp8Mm& g, int sms, cudaStream_t st) {
  Fp8Params p;
  p.g = g;
  // (The pitch of a single row means nothing: one that TMA takes.)
  const int64_t line = ((int64_t)g.k + 15) / 16 * 16;
  const Operand x{g.x, g.rows, g.k, g.rows == 1 ? line : g.ldx, 1, 0};
  const Operand w{g.w, g.n, g.k, g.n == 1 ? line : g.ldw, g.n_experts, g.w_stride};
  MmChoice c{1, false, false};
  while (c.parts < kMostParts && mm_tiles<Split8>(g) * c.parts * 2 <= sms && g.k >= 4 * kBK8 * c.parts * 2)
    c.parts *= 2;
  c.narrow = g.rows <= Narrow8::kMaxN * (int64_t)g.n_experts || mm_tiles<Narrow8>(g) <= sms;
  c.pair = !c.narrow && g.n > kBM && mm_tiles<Pair8>(g) >= sms;
  cudaError_t e = encode(&p.x, x, kE4m3, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w, w, kE4m3, true, kBM);
  if (e != cudaSuccess) return e;
  return g.out_dtype == kF32 ? launch_type<float>(p, c, sms, st)
         : g.out_dtype == kBf16 ? launch_type<__nv_bfloat16>(p, c, sms, st)
                                : launch_type<__half>(p, c, sms, st);
}

}  // namespace muon
