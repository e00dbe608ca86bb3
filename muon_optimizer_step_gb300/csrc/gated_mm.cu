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
// g and u of 8 of them.  g and u go to memory only where the caller keeps them.
//
// grad: dh stays in the accumulators.  The epilogue reads g and u of its tile (asked into L2 when the
// tile begins) and writes three results.  dp_r is summed over 32 columns in a warp; a second kernel adds
// those sums in order, so equal inputs give equal bits.
//
// sum: the k-blocks of the second product follow those of the first.
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
  static constexpr bool kFromTmem = true;
  static constexpr int kSlot = 16 * 32;                  // floats: 16 rows of a warp's 32 columns
  static constexpr int kStaging = kWarps * kSlot * 4;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool) { return &p.x; }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool second) {
    return second ? &p.w2 : &p.w;
  }
  static __device__ __forceinline__ bool fine(const Params&) { return false; }
  template <typename V>
  static __device__ __forceinline__ void ahead(const Params&, const MmTile&, int, int, int, int) {}

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

  static __device__ __forceinline__ float value(float g, float u, float w) {
    return g * sigmoid<T, true>(g) * u * w;
  }

  template <typename V, int kBlocks>
  static __device__ __forceinline__ void finish(const Params& p, const MmTile& m, int f, int q, int group,
                                                int lane, uint32_t tmem, uint8_t* staging) {
    const GatedMm& o = p.g;
    const int pair = gate_pair(q, group), mine = q >> 1;  // 0: has g; 1: has u
    float* slots = reinterpret_cast<float*>(staging) + pair * 2 * kSlot;
    const int col = f + 32 * (q & 1) + lane % 4 * 8, line = 8 * mine + lane / 4;
#pragma unroll 1
    for (int c = 0; c < kBlocks * 2; ++c) {
      const int r0 = chunk_row<16, kWarps / 4>(c, group);
      if (r0 >= m.rows) break;
      put_tmem_16(slots + mine * kSlot, lane, tmem + r0);
      sync_pair(pair);
      float g[8], u[8], v[8];
      get_line(slots, lane, line, g);
      get_line(slots + kSlot, lane, line, u);
      sync_pair(pair);  // the slots are read
      if (r0 + line >= m.rows) continue;
      const int64_t row = (int64_t)m.row + r0 + line;
      const float w = o.p != nullptr ? o.p[row] : 1.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = value(g[k], u[k], w);
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
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = value(g[k], u[k], w);
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
  bool wide;         // every row of gate and up starts on 16 bytes
};

template <typename T>
struct Grad {
  using Params = GradParams;
  static constexpr bool kGated = false;
  static constexpr int kCols = kBM, kPasses = 1, kWarps = 16;
  static constexpr bool kFromTmem = true;
  static constexpr int kSlot = 8 * 32;                  // floats: 8 rows of a warp's 32 columns
  static constexpr int kStaging = kWarps * kSlot * 4;
  static __device__ __forceinline__ const CUtensorMap* x_map(const Params& p, bool) { return &p.x; }
  static __device__ __forceinline__ const CUtensorMap* w_map(const Params& p, bool) { return &p.w; }
  // dp, an fp32 result, is made of whole sums.
  static __device__ __forceinline__ bool fine(const Params& p) { return p.g.dp != nullptr; }
  static __device__ __forceinline__ bool agree(int, int, bool ok) { return ok; }

  // Asks for the tile's g and u: a row per lane, the lines of its columns.
  template <typename V>
  static __device__ __forceinline__ void ahead(const Params& p, const MmTile& m, int f, int q, int group,
                                               int lane) {
    const GatedGrad& o = p.g;
    const int r = 16 * (q + 4 * group) + lane % 16, cols = min(kBM, o.n - f);
    if (r >= m.rows || cols <= 0 || lane >= 16) return;
    const int64_t row = (int64_t)m.row + r;
    const char* g = reinterpret_cast<const char*>(static_cast<const T*>(o.gate) + row * o.ld_gate + f);
    const char* u = reinterpret_cast<const char*>(static_cast<const T*>(o.up) + row * o.ld_up + f);
    const int last = 2 * cols - 2;
#pragma unroll
    for (int b = 0; b <= 256; b += 128) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(g + min(b, last)));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(u + min(b, last)));
    }
  }

  // From dh, g, u and the row's weight: dgate, dup and the activation; returns dp's term.  silu'(g) = s +
  // silu(g) (1 - s), with s and 1 - s both from exp(-|g|): neither overflows nor cancels.
  static __device__ __forceinline__ float values(float dh, float g, float u, float w, float* dgate,
                                                 float* dup, float* out) {
    const float e = __expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), er = e * r;
    const float s = g < 0.f ? er : r, silu = g * s, slope = fmaf(silu, g < 0.f ? r : er, s);
    const float d = dh * w, t = silu * u;
    *dup = d * silu;
    *dgate = d * (u * slope);
    *out = t * w;
    return dh * t;
  }

  // Eight values of a row from base + at on, `left` of them inside it, as they are stored; wide: on 16
  // bytes.  (Both ways end in the same words: nothing waits for the load here.)
  static __device__ __forceinline__ uint4 load_row(const void* base, int64_t at, int left, bool wide) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (wide && left >= 8) return *reinterpret_cast<const uint4*>(p);
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = k < left ? p[k] : 0;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }

  template <typename V, int kBlocks>
  static __device__ __forceinline__ void finish(const Params& p, const MmTile& m, int f, int q, int group,
                                                int lane, uint32_t tmem, uint8_t* staging) {
    const GatedGrad& o = p.g;
    if (f + 32 * q >= o.n) return;
    float* stage = reinterpret_cast<float*>(staging) + (q + 4 * group) * kSlot;
    const int col = f + 32 * q + lane % 4 * 8;
    // g, u and the row's weight of the next chunk arrive while this one is computed.
    uint4 g, u;
    float w = 1.f;
    const auto load = [&](int c) {
      const int r = chunk_row<8, kWarps / 4>(c, group) + lane / 4, left = r < m.rows ? o.n - col : 0;
      const int64_t row = (int64_t)m.row + r;
      g = load_row(o.gate, row * o.ld_gate + col, left, p.wide);
      u = load_row(o.up, row * o.ld_up + col, left, p.wide);
      if (o.p != nullptr && left > 0) w = o.p[row];
    };
    load(0);
#pragma unroll 1
    for (int c = 0; c < kBlocks * 4; ++c) {
      const int r0 = chunk_row<8, kWarps / 4>(c, group), r = r0 + lane / 4, left = r < m.rows ? o.n - col : 0;
      if (r0 >= m.rows) break;
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
      const float weight = w;
      if (c + 1 < kBlocks * 4) load(c + 1);
      __syncwarp();
      put_tmem_8(stage, lane, tmem + r0);
      __syncwarp();
      float dh[8], dg[8], du[8], out[8], term = 0.f;
      get_line(stage, lane, lane / 4, dh);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 a = unpack_2<T>(gw[k / 2]), b = unpack_2<T>(uw[k / 2]);
        const float t0 = values(dh[k], a.x, b.x, weight, &dg[k], &du[k], &out[k]);
        const float t1 = values(dh[k + 1], a.y, b.y, weight, &dg[k + 1], &du[k + 1], &out[k + 1]);
        if (k < left) term += t0;
        if (k + 1 < left) term += t1;
      }
      const int64_t row = (int64_t)m.row + r;
      store_8(static_cast<T*>(o.dgate) + row * o.ld_dgate + col, left, dg);
      store_8(static_cast<T*>(o.dup) + row * o.ld_dup + col, left, du);
      if (o.y != nullptr) store_8(static_cast<T*>(o.y) + row * o.ldy + col, left, out);
      if (o.dp != nullptr) {
        // Four neighbouring lanes have the row's 32 columns.
        term += __shfl_xor_sync(0xffffffffu, term, 1);
        term += __shfl_xor_sync(0xffffffffu, term, 2);
        if (lane % 4 == 0 && left > 0) o.part[(int64_t)((f + 32 * q) / 32) * o.rows + row] = term;
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
      float dh[8], dg[8], du[8], out[8], term = 0.f;
      join_parts<V>(smem, part.parts, r, col, dh);
      const int64_t row = (int64_t)m.row + r;
      const float w = o.p != nullptr ? o.p[row] : 1.f;
      const T* gate = static_cast<const T*>(o.gate) + row * o.ld_gate + f;
      const T* up = static_cast<const T*>(o.up) + row * o.ld_up + f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float g = k < left ? cvt(gate[k]) : 0.f, u = k < left ? cvt(up[k]) : 0.f;
        const float t = values(dh[k], g, u, w, &dg[k], &du[k], &out[k]);
        if (k < left) term += t;
      }
      store_8(static_cast<T*>(o.dgate) + row * o.ld_dgate + f, left, dg);
      store_8(static_cast<T*>(o.dup) + row * o.ld_dup + f, left, du);
      if (o.y != nullptr) store_8(static_cast<T*>(o.y) + row * o.ldy + f, left, out);
      if (o.dp != nullptr) {
        // Four neighbouring threads have 32 columns (a row's 16 are all here).
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

size_t gated_grad_workspace(const GatedGrad& g) {
  return g.rows == 0 ? 0 : copy_bytes(x_of(g, g.x, g.ldx)) + copy_bytes(w_of(g, g.w, g.ldw, g.w_stride)) +
                               (g.dp != nullptr ? (size_t)(row_parts(g) * g.rows * 4) : 0);
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
  p.wide = reinterpret_cast<uintptr_t>(g.gate) % 16 == 0 && reinterpret_cast<uintptr_t>(g.up) % 16 == 0 &&
           g.ld_gate % 8 == 0 && g.ld_up % 8 == 0;
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
