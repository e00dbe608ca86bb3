// The gated feed-forward block's products, forward and backward, with the activation in their epilogues.
//
//   gated:  g = x Wg_e, u = x Wu_e, out = p_r silu(g) u                      (silu(g) = g / (1 + exp(-g)))
//   grad:   dh = dy Wd_e, out = p_r silu(g) u, dup = dh p_r silu(g),
//           dgate = dh p_r u s (1 + g (1 - s)), dp_r = sum over the row of dh silu(g) u
//   sum:    y = x1 W1_e + x2 W2_e, in one accumulator                        (dx = dgate Wg^T + dup Wu^T)
//
// The tiles, loads and MMAs are the grouped products' (see grouped_mm.cu).
//
// gated: a tile's 128 accumulator lanes are 64 columns of g and the same 64 columns of u, so a k-block
// brings as many bytes into an SM as a plain product's of the same work.  The epilogue warp that holds 32
// columns of g and the one that holds them of u put 16 rows at a time into shared memory; each then takes
// g and u of 8 of them.  g and u go to memory only where the caller keeps them.  Bound by the tensor cores:
//   4096 rows, 4096 -> 14336, both kept   541-575 us  1.67-1.78 PFLOP/s (power)
//   192 rows, 2048 -> 1408, 64 experts    105 us  6.7 TB/s (the weights, HBM)
// (Passes in a graph, here and below.)
//
// grad: dh stays in the accumulators.  The epilogue reads g and u of its tile and writes three results.  dp_r is
// summed over 32 columns in a warp; a second kernel adds those sums in order, so equal inputs give equal bits.
// The epilogue bounds it: its loads, exponentials and stores of a 256 x 256 tile take 18000 cycles, in which
// the MMAs, 16400, get one accumulator ahead (98304 rows, 2048 -> 1408: 638 us, 0.89 PFLOP/s and 2.8 TB/s, of which
// the fine sigmoid is 9; without dp 555-585; the plain product, muon_swiglu_grad and the activation again 713).  With
// the plain sigmoid it took 633, tiles of half as many rows with four accumulators 677 (an MMA warp needs 450 cycles
// to issue a k-block), single CTAs 639, eight warps of the epilogue 755.
//
// sum: the k-blocks of the second product follow those of the first (24570 rows, 1408 -> 2048: 208 us, 1.36
// PFLOP/s).
#include "activation.cuh"
#include "grouped_kernel.cuh"

namespace muon {

namespace {

// The two warps that hold the same 32 columns of g and of u.
__device__ __forceinline__ int gate_pair(int q, int group) { return (q & 1) + 2 * group; }
__device__ __forceinline__ void sync_pair(int pair) {
  asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
}

struct GatedParams {
  CUtensorMap x, w, w2;  // the weights': boxes of 64 x 64
  GatedMm g;
};

template <typename T>
struct Gated {
  using Params = GatedParams;
  static constexpr bool kGated = true;
  static constexpr int kCols = 64, kPasses = 1, kWarps = 16;
  static constexpr bool kFromTmem = true, kKeep = true;
  static constexpr int kSlot = 16 * 32;                  // floats: 16 rows of a warp's 32 columns
  static constexpr int kStaging = kWarps * kSlot * 4;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool) { return &p.x; }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool second) {
    return second ? &p.w2 : &p.w;
  }
  static __device__ __forceinline__ bool fine(const Params&) { return false; }
  // Both warps of a pair give up, or neither: one that finished alone would wait for ever.
  static __device__ __forceinline__ bool agree(int q, int group, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.and.pred b, %2, 64, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(gate_pair(q, group) + 1)
        : "memory");
    return all != 0;
  }

  static __device__ __forceinline__ void values(const float (&g)[8], const float (&u)[8], float w,
                                                float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const f32x2 x = pair(g[k], g[k + 1]);
      const float2 a = parts(mul2(mul2(mul2(x, sigmoid2<false>(x)), pair(u[k], u[k + 1])), pair(w, w)));
      v[k] = a.x, v[k + 1] = a.y;
    }
  }

  template <typename V, int kBlocks, typename F>
  static __device__ __forceinline__ void finish(const Params& p, const MmTile& m, int f, int q, int group,
                                                int lane, uint32_t tmem, const float (&kept)[32],
                                                const F& release, uint8_t* staging) {
    constexpr int kInTmem = kBlocks == 1 ? 2 : (kBlocks - 1) * 2;  // chunks
    const GatedMm& o = p.g;
    const int pair = gate_pair(q, group), mine = q >> 1;  // 0: has g; 1: has u
    float* slots = reinterpret_cast<float*>(staging) + pair * 2 * kSlot;
    const int col = f + 32 * (q & 1) + lane % 4 * 8, line = 8 * mine + lane / 4;
#pragma unroll 1
    for (int c = 0; c < kBlocks * 2; ++c) {
      const int r0 = chunk_row<16, kWarps / 4>(c, group);
      if (r0 >= m.rows) break;
      if (c < kInTmem) put_tmem_16(slots + mine * kSlot, lane, tmem + r0);
      else put_chunk<1, 16>(slots + mine * kSlot, lane, c - kInTmem, [&](int, int k) { return kept[k]; });
      if (c == kInTmem - 1) release();
      sync_pair(pair);
      float g[8], u[8], v[8];
      get_line(slots, lane, line, g);
      get_line(slots + kSlot, lane, line, u);
      sync_pair(pair);  // the slots are read
      if (r0 + line >= m.rows) continue;
      const int64_t row = (int64_t)m.row + r0 + line;
      const float w = o.p != nullptr ? o.p[row] : 1.f;
      values(g, u, w, v);
      store_8(static_cast<T*>(o.y) + row * o.ldy + col, o.n - col, v);
      if (o.gate != nullptr) store_8(static_cast<T*>(o.gate) + row * o.ld_gate + col, o.n - col, g);
      if (o.up != nullptr) store_8(static_cast<T*>(o.up) + row * o.ld_up + col, o.n - col, u);
    }
  }

  template <typename V>
  static __device__ __forceinline__ void join(const Params& p, const MmTile& m, const Part& part,
                                              uint8_t* smem) {
    const GatedMm& o = p.g;
    for (int i = threadIdx.x - 128 + part.index * kWarps * 32; i < m.rows * 8;
         i += part.parts * kWarps * 32) {
      const int r = i / 8, col = i % 8 * 8, f = m.f0 + col;
      float g[8], u[8], v[8];
      join_parts<V>(smem, part.parts, r, col, g);
      join_parts<V>(smem, part.parts, r, 64 + col, u);
      const int64_t row = (int64_t)m.row + r;
      const float w = o.p != nullptr ? o.p[row] : 1.f;
      values(g, u, w, v);
      store_8(static_cast<T*>(o.y) + row * o.ldy + f, o.n - f, v);
      if (o.gate != nullptr) store_8(static_cast<T*>(o.gate) + row * o.ld_gate + f, o.n - f, g);
      if (o.up != nullptr) store_8(static_cast<T*>(o.up) + row * o.ld_up + f, o.n - f, u);
    }
  }

  static __device__ __forceinline__ void zero_row(const Params& p, int64_t row, int thread) {
    const GatedMm& o = p.g;
    for (int64_t f = thread; f < o.n; f += kWarps * 32) {
      put(static_cast<T*>(o.y) + row * o.ldy + f, 0.f);
      if (o.gate != nullptr) put(static_cast<T*>(o.gate) + row * o.ld_gate + f, 0.f);
      if (o.up != nullptr) put(static_cast<T*>(o.up) + row * o.ld_up + f, 0.f);
    }
  }
};

struct GradParams {
  CUtensorMap x, w;  // as MmParams
  GatedGrad g;
  bool wide;         // every row of gate, up and the results starts on 16 bytes
};

template <typename T>
struct Grad {
  using Params = GradParams;
  static constexpr bool kGated = false;
  static constexpr int kCols = kBM, kPasses = 1, kWarps = 16;
  static constexpr bool kFromTmem = true, kKeep = false;
  static constexpr int kSlot = 8 * 32;                  // floats: 8 rows of a warp's 32 columns
  static constexpr int kStaging = kWarps * kSlot * 4;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool) { return &p.x; }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool) { return &p.w; }
  // dp, an fp32 result, is made of whole sums.
  static __device__ __forceinline__ bool fine(const Params& p) { return p.g.dp != nullptr; }
  static __device__ __forceinline__ bool agree(int, int, bool ok) { return ok; }

  // From dh, g, u and the row's weight (twice), two at a time: dgate, dup and the activation; adds dp's terms.
  // silu'(g) = s + silu(g) (1 - s).
  static __device__ __forceinline__ void values(f32x2 dh, f32x2 g, f32x2 u, f32x2 w, float* dgate, float* dup,
                                                float* out, f32x2& dp) {
    const f32x2 s = sigmoid2<true>(g), silu = mul2(g, s);
    const f32x2 slope = fma2(silu, fma2(s, pair(-1.f, -1.f), pair(1.f, 1.f)), s);
    const f32x2 d = mul2(dh, w), t = mul2(silu, u);
    const float2 a = parts(mul2(d, mul2(u, slope))), b = parts(mul2(d, silu)), c = parts(mul2(t, w));
    dgate[0] = a.x, dgate[1] = a.y, dup[0] = b.x, dup[1] = b.y, out[0] = c.x, out[1] = c.y;
    dp = fma2(dh, t, dp);
  }

  // Eight values of a row, `left` of them inside it, as they are stored.  (Both ways end in the same words:
  // nothing waits for the load here.)
  static __device__ __forceinline__ uint4 load_row(const T* at, int left, bool wide) {
    if (wide && left >= 8) return *reinterpret_cast<const uint4*>(at);
    const uint16_t* p = reinterpret_cast<const uint16_t*>(at);
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = k < left ? p[k] : 0;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
  static __device__ __forceinline__ void store_row(T* at, int left, bool wide, const float (&v)[8]) {
    if (wide && left >= 8) {
      *reinterpret_cast<uint4*>(at) = make_uint4(pack_2<T>(v[0], v[1]), pack_2<T>(v[2], v[3]),
                                                 pack_2<T>(v[4], v[5]), pack_2<T>(v[6], v[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) put(&at[k], v[k]);
    }
  }

  // 8 rows of the warp's 32 columns at a time: dh goes through shared memory (see put_line), so that a lane
  // then has eight columns of a row, the width of its loads and stores.
  template <typename V, int kBlocks, typename F>
  static __device__ __forceinline__ void finish(const Params& p, const MmTile& m, int f, int q, int group,
                                                int lane, uint32_t tmem, const float (&)[32], const F&,
                                                uint8_t* staging) {
    const GatedGrad& o = p.g;
    if (f + 32 * q >= o.n) return;
    float* stage = reinterpret_cast<float*>(staging) + (q + 4 * group) * kSlot;
    const int col = f + 32 * q + lane % 4 * 8, inside = o.n - col;
    const bool wide = p.wide;
    // g, u and the row's weight of the next chunk arrive while this one is computed.
    const T* gate = static_cast<const T*>(o.gate) + (int64_t)m.row * o.ld_gate + col;
    const T* up = static_cast<const T*>(o.up) + (int64_t)m.row * o.ld_up + col;
    T* dgate = static_cast<T*>(o.dgate) + (int64_t)m.row * o.ld_dgate + col;
    T* dup = static_cast<T*>(o.dup) + (int64_t)m.row * o.ld_dup + col;
    T* act = static_cast<T*>(o.y) + (int64_t)m.row * o.ldy + col;
    uint4 g, u;
    float w = 1.f;
    const auto load = [&](int c) {
      const int r = chunk_row<8, kWarps / 4>(c, group) + lane / 4, left = r < m.rows ? inside : 0;
      g = load_row(gate + r * o.ld_gate, left, wide);
      u = load_row(up + r * o.ld_up, left, wide);
      if (o.p != nullptr && left > 0) w = o.p[m.row + r];
    };
    load(0);
#pragma unroll 1
    for (int c = 0; c < kBlocks * 4; ++c) {
      const int r0 = chunk_row<8, kWarps / 4>(c, group), r = r0 + lane / 4, left = r < m.rows ? inside : 0;
      if (r0 >= m.rows) break;
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
      const float weight = w;
      if (c + 1 < kBlocks * 4) load(c + 1);
      __syncwarp();
      put_tmem_8(stage, lane, tmem + r0);
      __syncwarp();
      float dh[8], dg[8], du[8], out[8];
      f32x2 terms = 0;
      get_line(stage, lane, lane / 4, dh);
      if (left < 8)  // columns outside: nothing that dp adds
#pragma unroll
        for (int k = 0; k < 8; ++k) dh[k] = k < left ? dh[k] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 a = unpack_2<T>(gw[k / 2]), b = unpack_2<T>(uw[k / 2]);
        values(pair(dh[k], dh[k + 1]), pair(a.x, a.y), pair(b.x, b.y), pair(weight, weight), &dg[k], &du[k],
               &out[k], terms);
      }
      store_row(dgate + r * o.ld_dgate, left, wide, dg);
      store_row(dup + r * o.ld_dup, left, wide, du);
      if (o.y != nullptr) store_row(act + r * o.ldy, left, wide, out);
      if (o.dp != nullptr) {
        // Four neighbouring lanes have the row's 32 columns.
        float term = parts(terms).x + parts(terms).y;
        term += __shfl_xor_sync(0xffffffffu, term, 1);
        term += __shfl_xor_sync(0xffffffffu, term, 2);
        if (lane % 4 == 0 && left > 0) o.part[(int64_t)((f + 32 * q) / 32) * o.rows + m.row + r] = term;
      }
    }
  }

  template <typename V>
  static __device__ __forceinline__ void join(const Params& p, const MmTile& m, const Part& part,
                                              uint8_t* smem) {
    const GatedGrad& o = p.g;
    for (int i = threadIdx.x - 128 + part.index * kWarps * 32; i < m.rows * 16;
         i += part.parts * kWarps * 32) {
      const int r = i / 16, col = i % 16 * 8, f = m.f0 + col, left = o.n - f;
      float dh[8], g[8], u[8], dg[8], du[8], out[8];
      f32x2 terms = 0;
      join_parts<V>(smem, part.parts, r, col, dh);
      const int64_t row = (int64_t)m.row + r;
      const float w = o.p != nullptr ? o.p[row] : 1.f;
      const T* gate = static_cast<const T*>(o.gate) + row * o.ld_gate + f;
      const T* up = static_cast<const T*>(o.up) + row * o.ld_up + f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dh[k] = k < left ? dh[k] : 0.f;
        g[k] = k < left ? cvt(gate[k]) : 0.f;
        u[k] = k < left ? cvt(up[k]) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        values(pair(dh[k], dh[k + 1]), pair(g[k], g[k + 1]), pair(u[k], u[k + 1]), pair(w, w), &dg[k], &du[k],
               &out[k], terms);
      store_8(static_cast<T*>(o.dgate) + row * o.ld_dgate + f, left, dg);
      store_8(static_cast<T*>(o.dup) + row * o.ld_dup + f, left, du);
      if (o.y != nullptr) store_8(static_cast<T*>(o.y) + row * o.ldy + f, left, out);
      if (o.dp != nullptr) {
        // Four neighbouring threads have 32 columns (a row's 16 are all here).
        float term = parts(terms).x + parts(terms).y;
        const uint32_t four = 0xfu << (threadIdx.x & 28);
        term += __shfl_xor_sync(four, term, 1);
        term += __shfl_xor_sync(four, term, 2);
        if (threadIdx.x % 4 == 0 && f < o.n) o.part[(int64_t)(f / 32) * o.rows + row] = term;
      }
    }
  }

  static __device__ __forceinline__ void zero_row(const Params& p, int64_t row, int thread) {
    const GatedGrad& o = p.g;
    for (int64_t f = thread; f < o.n; f += kWarps * 32) {
      put(static_cast<T*>(o.dgate) + row * o.ld_dgate + f, 0.f);
      put(static_cast<T*>(o.dup) + row * o.ld_dup + f, 0.f);
      if (o.y != nullptr) put(static_cast<T*>(o.y) + row * o.ldy + f, 0.f);
      if (o.dp != nullptr && f % 32 == 0) o.part[f / 32 * o.rows + row] = 0.f;
    }
  }
};

// dp from its sums over 32 columns, in order.
__global__ void __launch_bounds__(256)
row_sums_kernel(const float* __restrict__ part, int64_t rows, int32_t parts, float* __restrict__ dp) {
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows; r += (int64_t)gridDim.x * 256) {
    float s = 0.f;
#pragma unroll 8
    for (int32_t t = 0; t < parts; ++t) s += part[t * rows + r];
    dp[r] = s;
  }
}

struct SumParams {
  CUtensorMap x, w, x2, w2;  // as MmParams
  MmSum g;
};

template <typename O>
struct Sum : Store<O> {
  using Params = SumParams;
  static constexpr int kPasses = 2;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool second) {
    return second ? &p.x2 : &p.x;
  }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool second) {
    return second ? &p.w2 : &p.w;
  }
  static constexpr int kSlot = 16 * 32, kStaging = kEpiWarps * kSlot * 4;
  template <typename V>
  static __device__ __forceinline__ void finish(const Params& p, const MmTile& m, int f, int q, int half,
                                                int lane, const float (&sum)[Shape<V>::kBlocks][32],
                                                uint8_t* staging) {
    const int col = f + 32 * q + lane % 4 * 8, inside = p.g.n - col;
    O* y = static_cast<O*>(p.g.y) + (int64_t)m.row * p.g.ldy + col;
    by_rows<Shape<V>::kBlocks, 16, 2>(
        reinterpret_cast<float*>(staging) + (q + 4 * half) * kSlot, lane, m.rows, half,
        [&](int i, int k) { return sum[i][k]; },
        [&](int r, const float (&v)[8]) { store_8(y + r * p.g.ldy, inside, v); });
  }
};

Operand x_of(const GroupedMm& g, const void* x, int64_t ldx) { return operand(x, g.rows, g.k, ldx, 1, 0); }
Operand w_of(const GroupedMm& g, const void* w, int64_t ldw, int64_t stride) {
  return operand(w, g.trans ? g.n : g.k, g.trans ? g.k : g.n, ldw, g.n_experts, stride);
}

int64_t row_parts(const GroupedMm& g) { return ((int64_t)g.n + 31) / 32; }

}  // namespace

// The device counts tiles in 32 bits (of 64 columns, at least as many as any of these products has).
bool gated_mm_fits(const GroupedMm& g) {
  return (g.rows / Narrow::kMaxN + g.n_experts) * (int64_t)((g.n - 1) / 64 + 1) <= INT32_MAX;
}

size_t gated_mm_workspace(const GatedMm& g) {
  return g.rows == 0 ? 0 : copy_bytes(x_of(g, g.x, g.ldx)) + copy_bytes(w_of(g, g.w, g.ldw, g.w_stride)) +
                               copy_bytes(w_of(g, g.w2, g.ldw2, g.w2_stride));
}

size_t gated_grad_workspace(const GatedGrad& g, bool row_weight_grad) {
  return g.rows == 0 ? 0 : copy_bytes(x_of(g, g.x, g.ldx)) + copy_bytes(w_of(g, g.w, g.ldw, g.w_stride)) +
                               (row_weight_grad ? (size_t)(row_parts(g) * g.rows * 4) : 0);
}

size_t mm_sum_workspace(const MmSum& g) {
  return g.rows == 0 ? 0 : copy_bytes(x_of(g, g.x, g.ldx)) + copy_bytes(w_of(g, g.w, g.ldw, g.w_stride)) +
                               copy_bytes(x_of(g, g.x2, g.ldx2)) +
                               copy_bytes(w_of(g, g.w2, g.ldw2, g.w2_stride));
}

cudaError_t launch_gated_mm(const GatedMm& g, void* workspace, int sms, cudaStream_t st) {
  GatedParams p;
  p.g = g;
  Operand x = x_of(g, g.x, g.ldx), w = w_of(g, g.w, g.ldw, g.w_stride),
          w2 = w_of(g, g.w2, g.ldw2, g.w2_stride);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = align_operands(&x, &w, g.offsets, &at, sms, st);
  if (e == cudaSuccess) e = align_operands(nullptr, &w2, g.offsets, &at, sms, st);
  const MmChoice c = choose_tiles<Gated<__half>>(g, false, sms);
  if (e == cudaSuccess) e = encode(&p.x, x, g.dtype, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, 64);
  if (e == cudaSuccess) e = encode(&p.w2, w2, g.dtype, true, 64);
  if (e != cudaSuccess) return e;
  return g.dtype == kBf16 ? launch_tiles<Gated<__nv_bfloat16>, true>(p, c, sms, st)
                          : launch_tiles<Gated<__half>, true>(p, c, sms, st);
}

cudaError_t launch_gated_grad(const GatedGrad& g, void* workspace, int sms, cudaStream_t st) {
  GradParams p;
  p.g = g;
  Operand x = x_of(g, g.x, g.ldx), w = w_of(g, g.w, g.ldw, g.w_stride);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = align_operands(&x, &w, g.offsets, &at, sms, st);
  p.g.part = reinterpret_cast<float*>(at);
  p.wide = true;
  const void* const matrices[] = {g.gate, g.up, g.dgate, g.dup, g.y};
  const int64_t pitches[] = {g.ld_gate, g.ld_up, g.ld_dgate, g.ld_dup, g.y != nullptr ? g.ldy : 0};
  for (int i = 0; i < 5; ++i)
    p.wide = p.wide && reinterpret_cast<uintptr_t>(matrices[i]) % 16 == 0 && pitches[i] % 8 == 0;
  const MmChoice c = choose_tiles<Grad<__half>>(g, false, sms);
  if (e == cudaSuccess) e = encode(&p.x, x, g.dtype, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, g.trans ? kBM : 64);
  if (e == cudaSuccess)
    e = g.dtype == kBf16 ? launch_tiles<Grad<__nv_bfloat16>, true>(p, c, sms, st)
                         : launch_tiles<Grad<__half>, true>(p, c, sms, st);
  if (e != cudaSuccess || g.dp == nullptr) return e;
  const int64_t blocks = (g.rows + 255) / 256, cap = (int64_t)sms * 8;
  row_sums_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, st>>>(p.g.part, g.rows,
                                                                         (int32_t)row_parts(g), g.dp);
  return cudaGetLastError();
}

cudaError_t launch_mm_sum(const MmSum& g, void* workspace, int sms, cudaStream_t st) {
  SumParams p;
  p.g = g;
  Operand x = x_of(g, g.x, g.ldx), w = w_of(g, g.w, g.ldw, g.w_stride), x2 = x_of(g, g.x2, g.ldx2),
          w2 = w_of(g, g.w2, g.ldw2, g.w2_stride);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  cudaError_t e = align_operands(&x, &w, g.offsets, &at, sms, st);
  if (e == cudaSuccess) e = align_operands(&x2, &w2, g.offsets, &at, sms, st);
  const MmChoice c = choose_tiles<Sum<float>>(g, g.out_dtype == kF32, sms);
  const uint32_t lines = g.trans ? kBM : 64;
  if (e == cudaSuccess) e = encode(&p.x, x, g.dtype, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w, w, g.dtype, true, lines);
  if (e == cudaSuccess) e = encode(&p.x2, x2, g.dtype, false, c.box_rows());
  if (e == cudaSuccess) e = encode(&p.w2, w2, g.dtype, true, lines);
  if (e != cudaSuccess) return e;
  return g.out_dtype == kF32 ? launch_tiles<Sum<float>, false>(p, c, sms, st)
         : g.out_dtype == kBf16 ? launch_tiles<Sum<__nv_bfloat16>, true>(p, c, sms, st)
                                : launch_tiles<Sum<__half>, true>(p, c, sms, st);
}

}  // namespace muon
