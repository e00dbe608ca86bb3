// Layer norm of rows and its gradient.
//
//   y  = (x - mean) * rstd * w + b,  mean = sum x / cols,  rstd = (sum (x - mean)^2 / cols + eps)^-1/2
//   xh = (x - mean) * rstd,  t = dy * w
//   dx = rstd * (t - sum t / cols - xh * sum(t * xh) / cols)
//   dw (+)= sum over the rows of dy * xh,  db (+)= sum over the rows of dy
//
// Sums in fp32, one rounding at each store.  The variance is that of the deviations from the mean,
// which rows with a large mean need; the row stays in registers between the two sums, so HBM sees
// each value once: 2 values move per element, 3 in the gradient.
//
// Short rows, rows of 32 bits and few rows: kTpr threads share a row (8 or 32 lanes of a warp, or a block), kN
// vectors each, and ask for the next row's values before they sum this one's.  In the gradient a thread keeps
// its columns over all the rows of its block and sums dw and db in registers; the blocks' sums go to
// the workspace, and a second kernel adds them in a fixed order, so equal inputs give equal bits.  Longer rows
// of 16-bit values go by slabs (below).  Rows too long for registers are read again for each sum, and their
// columns summed by blocks of columns in a pass of their own.
//
// Bound by HBM as far as the arithmetic, two values to an instruction, and the sums' latency leave room:
//   16384 x 4096 bf16  57 us forward (4.7 TB/s), 102 us backward (3.9 TB/s)
//   16384 x 4096 fp32  88 us (6.1 TB/s), 151 us (5.3 TB/s)
//   65536 x 768 bf16   54 us (3.7 TB/s), 88 us (3.4 TB/s)
//   32 x 4096 bf16     2.9 us, 9 us (launches and the latency of one row)
// (Passes in a graph; a slab's two parts wait for each other, which is what keeps the 16-bit rows from HBM's rate.)
#include <atomic>
#include <type_traits>

#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

template <typename T, int V>
struct Vec {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  Vec<T, V> r;
  if constexpr (V == 1) {
    r.v[0] = *p;
  } else {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    memcpy(r.v, &q, 16);
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& r) {
  if constexpr (V == 1) {
    *p = r.v[0];
  } else {
    uint4 q;
    memcpy(&q, r.v, 16);
    *reinterpret_cast<uint4*>(p) = q;
  }
}

// The arithmetic of V values: on pairs, two to an instruction, or (V = 1) on single ones.
template <int V>
using Wide = typename std::conditional<V == 1, float, f32x2>::type;
template <int V>
constexpr int kWide = V == 1 ? 1 : V / 2;

template <typename W>
__device__ __forceinline__ W both(float v) {
  if constexpr (sizeof(W) == 4) return v;
  else return pair(v, v);
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& v, Wide<V> (&w)[kWide<V>]) {
  if constexpr (V == 1) {
    w[0] = cvt(v.v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V; k += 2) w[k / 2] = pair(v.v[k], v.v[k + 1]);
  } else {
    uint32_t q[V / 2];
    memcpy(q, v.v, sizeof(q));
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const float2 f = unpack_2<T>(q[k]);
      w[k] = pair(f.x, f.y);
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_wide(T* p, const Wide<V> (&w)[kWide<V>]) {
  Vec<T, V> v;
  if constexpr (V == 1) {
    put(&v.v[0], w[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      v.v[k] = parts(w[k / 2]).x;
      v.v[k + 1] = parts(w[k / 2]).y;
    }
  } else {
    uint32_t q[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) q[k] = pack_2<T>(parts(w[k]).x, parts(w[k]).y);
    memcpy(v.v, q, sizeof(q));
  }
  store_vec<T, V>(p, v);
}

// V weights from p on (`value` where there are none); wide: they start on 16 bytes.
template <int V>
__device__ __forceinline__ void load_weights(const float* p, bool wide, float value, Wide<V> (&w)[kWide<V>]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < kWide<V>; ++k) w[k] = both<Wide<V>>(value);
  } else if constexpr (V == 1) {
    w[0] = __ldg(p);
  } else if (wide) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p + k));
      w[k / 2] = pair(q.x, q.y);
      w[k / 2 + 1] = pair(q.z, q.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 2) w[k / 2] = pair(__ldg(p + k), __ldg(p + k + 1));
  }
}

// The sum over a group of kTpr threads, in every one of them, in a fixed order.  Blocks: `turn`
// changes with each call, so that one barrier per call is enough.
template <int kTpr>
__device__ __forceinline__ float2 group_sum(float2 v, float2 (*red)[32], int turn) {
#pragma unroll
  for (int o = (kTpr < 32 ? kTpr : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (kTpr > 32) {
    if (threadIdx.x % 32 == 0) red[turn & 1][threadIdx.x / 32] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kTpr / 32; ++k) {
      const float2 u = red[turn & 1][k];
      v.x += u.x;
      v.y += u.y;
    }
  }
  return v;
}

struct Aligned {
  bool w, b;  // the weights (biases) start on 16 bytes
};

template <int kTpr>
constexpr int kBlockThreads = kTpr > 32 ? kTpr : 256;

// (Threads without a row stay for the shuffles.)
template <typename T, int V, int kTpr, int kN>
__global__ void __launch_bounds__(kBlockThreads<kTpr>)
norm_kernel(const NormArgs a, const Aligned aligned) {
  constexpr int kRows = kBlockThreads<kTpr> / kTpr;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % kTpr, g = threadIdx.x / kTpr;
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  int turn = 0;
  using W = Wide<V>;
  // A thread with one vector of a row keeps its weights.
  W hw[kWide<V>], hb[kWide<V>];
  if (kN == 1 && (uint32_t)t * V < cols) {
    load_weights<V>(a.w == nullptr ? nullptr : a.w + t * V, aligned.w, 1.f, hw);
    load_weights<V>(a.b == nullptr ? nullptr : a.b + t * V, aligned.b, 0.f, hb);
  }
  Vec<T, V> next[kN];
  // A row's values, asked for while the row before is at work.
  const auto load = [&](int64_t r) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (r < a.rows && c < cols) next[i] = load_vec<T, V>(x + c);
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  load((int64_t)blockIdx.x * kRows + g);
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += step) {
    const int64_t r = r0 + g;
    const bool on = r < a.rows;
    float2 s = make_float2(0.f, 0.f);
    W x[kN][kWide<V>], sum[kWide<V>];
#pragma unroll
    for (int k = 0; k < kWide<V>; ++k) sum[k] = both<W>(0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (on && (uint32_t)(t + i * kTpr) * V < cols) {
        widen<T, V>(next[i], x[i]);
#pragma unroll
        for (int k = 0; k < kWide<V>; ++k) sum[k] = add2(sum[k], x[i][k]);
      }
    load(r + step);
#pragma unroll
    for (int k = 0; k < kWide<V>; ++k) s.x += total(sum[k]);
    const float mean = group_sum<kTpr>(s, red, turn++).x * over;
#pragma unroll
    for (int k = 0; k < kWide<V>; ++k) sum[k] = both<W>(0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (on && (uint32_t)(t + i * kTpr) * V < cols)
#pragma unroll
        for (int k = 0; k < kWide<V>; ++k) {
          x[i][k] = add2(x[i][k], both<W>(-mean));
          sum[k] = fma2(x[i][k], x[i][k], sum[k]);
        }
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWide<V>; ++k) s.x += total(sum[k]);
    const float rstd = rsqrtf(group_sum<kTpr>(s, red, turn++).x * over + a.eps);
    if (on) {
      T* y = static_cast<T*>(a.out) + r * a.ldo;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t c = (uint32_t)(t + i * kTpr) * V;
        if (c >= cols) continue;
        W w[kWide<V>], b[kWide<V>];
        if constexpr (kN > 1) {
          load_weights<V>(a.w == nullptr ? nullptr : a.w + c, aligned.w, 1.f, w);
          load_weights<V>(a.b == nullptr ? nullptr : a.b + c, aligned.b, 0.f, b);
        }
#pragma unroll
        for (int k = 0; k < kWide<V>; ++k)
          b[k] = fma2(mul2(x[i][k], both<W>(rstd)), kN > 1 ? w[k] : hw[k], kN > 1 ? b[k] : hb[k]);
        store_wide<T, V>(y + c, b);
      }
      if (t == 0) {
        if (a.mean != nullptr) a.mean[r] = mean;
        if (a.rstd != nullptr) a.rstd[r] = rstd;
      }
    }
  }
}

// Rows of any length: three passes.
constexpr int kLong = 1024;
template <typename T>
__global__ void __launch_bounds__(kLong) norm_long_kernel(const NormArgs a) {
  __shared__ float2 red[2][32];
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.out) + r * a.ldo;
    float2 s = make_float2(0.f, 0.f);
    for (uint32_t c = threadIdx.x; c < cols; c += kLong) s.x += cvt(x[c]);
    const float mean = group_sum<kLong>(s, red, turn++).x * over;
    s = make_float2(0.f, 0.f);
    for (uint32_t c = threadIdx.x; c < cols; c += kLong) {
      const float d = cvt(x[c]) - mean;
      s.x = fmaf(d, d, s.x);
    }
    const float rstd = rsqrtf(group_sum<kLong>(s, red, turn++).x * over + a.eps);
    for (uint32_t c = threadIdx.x; c < cols; c += kLong)
      put(&y[c], fmaf((cvt(x[c]) - mean) * rstd, a.w != nullptr ? a.w[c] : 1.f,
                      a.b != nullptr ? a.b[c] : 0.f));
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[r] = mean;
      if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------- gradient
// kSums: the block's column sums of dy * xh and dy are wanted, at part + (2 block) cols and one
// row behind.
template <typename T, int V, int kTpr, int kN, bool kSums>
__global__ void __launch_bounds__(kBlockThreads<kTpr>)
norm_grad_kernel(const NormArgs a, const Aligned aligned) {
  constexpr int kThreads = kBlockThreads<kTpr>, kRows = kThreads / kTpr;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % kTpr, g = threadIdx.x / kTpr;
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  using W = Wide<V>;
  constexpr int H = kWide<V>;
  W dw[kN][H], db[kN][H];
  if constexpr (kSums)
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int k = 0; k < H; ++k) dw[i][k] = db[i][k] = both<W>(0.f);
  W hw[H];  // as in the forward pass
  if (kN == 1 && (uint32_t)t * V < cols)
    load_weights<V>(a.w == nullptr ? nullptr : a.w + t * V, aligned.w, 1.f, hw);
  int turn = 0;
  Vec<T, V> xv[kN], dv[kN], xn[kN], dn[kN];
  float mean, rstd, mean_n = 0.f, rstd_n = 0.f;
  const auto load = [&](int64_t r) {
    if (r >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    mean_n = a.mean_in[r];
    rstd_n = a.rstd_in[r];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (c < cols) {
        xn[i] = load_vec<T, V>(x + c);
        dn[i] = load_vec<T, V>(dy + c);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  load((int64_t)blockIdx.x * kRows + g);
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += step) {
    const int64_t r = r0 + g;
    const bool on = r < a.rows;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      xv[i] = xn[i];
      dv[i] = dn[i];
    }
    mean = mean_n;
    rstd = rstd_n;
    load(r + step);
    W s1[H], s2[H];
#pragma unroll
    for (int k = 0; k < H; ++k) s1[k] = s2[k] = both<W>(0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (!on || c >= cols) continue;
      W w[H], x[H], d[H];
      if constexpr (kN > 1) {
        load_weights<V>(a.w == nullptr ? nullptr : a.w + c, aligned.w, 1.f, w);
      } else {
#pragma unroll
        for (int k = 0; k < H; ++k) w[k] = hw[k];
      }
      widen<T, V>(xv[i], x);
      widen<T, V>(dv[i], d);
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const W xh = mul2(add2(x[k], both<W>(-mean)), both<W>(rstd)), u = mul2(d[k], w[k]);
        s1[k] = add2(s1[k], u);
        s2[k] = fma2(u, xh, s2[k]);
        if constexpr (kSums) {
          dw[i][k] = fma2(d[k], xh, dw[i][k]);
          db[i][k] = add2(db[i][k], d[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < H; ++k) {
      s.x += total(s1[k]);
      s.y += total(s2[k]);
    }
    s = group_sum<kTpr>(s, red, turn++);
    if (!on) continue;
    // dx = dy (w rstd) - rstd m1 - xh (rstd m2): rstd^2 is beyond fp32 where rows have a tiny spread.
    const W c1 = both<W>(-rstd * (s.x * over)), c2 = both<W>(-rstd * (s.y * over));
    T* dx = static_cast<T*>(a.out) + r * a.ldo;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (c >= cols) continue;
      W w[H], x[H], d[H];
      if constexpr (kN > 1) {
        load_weights<V>(a.w == nullptr ? nullptr : a.w + c, aligned.w, 1.f, w);
      } else {
#pragma unroll
        for (int k = 0; k < H; ++k) w[k] = hw[k];
      }
      widen<T, V>(xv[i], x);
      widen<T, V>(dv[i], d);
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const W xh = mul2(add2(x[k], both<W>(-mean)), both<W>(rstd));
        d[k] = fma2(xh, c2, fma2(d[k], mul2(w[k], both<W>(rstd)), c1));
      }
      store_wide<T, V>(dx + c, d);
    }
  }
  if constexpr (kSums) {
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    const auto value = [](W v, int k) {
      if constexpr (V == 1) return v;
      else return k == 0 ? parts(v).x : parts(v).y;
    };
    constexpr int E = V / H;  // values of a W
    if constexpr (kRows == 1) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t c = (uint32_t)(t + i * kTpr) * V;
        if (c >= cols) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          part[c + k] = value(dw[i][k / E], k % E);
          part[cols + c + k] = value(db[i][k / E], k % E);
        }
      }
    } else {
      // The groups' sums meet in shared memory and are added in order.
      constexpr int kCols = kTpr * kN * V;
      __shared__ float sums[kRows * kCols];
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k)
            sums[g * kCols + (t + i * kTpr) * V + k] = value(which == 0 ? dw[i][k / E] : db[i][k / E], k % E);
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < (uint32_t)kCols && c < cols; c += kThreads) {
          float s = 0.f;
#pragma unroll
          for (int q = 0; q < kRows; ++q) s += sums[q * kCols + c];
          part[which * cols + c] = s;
        }
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLong) norm_grad_long_kernel(const NormArgs a) {
  __shared__ float2 red[2][32];
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dx = static_cast<T*>(a.out) + r * a.ldo;
    const float mean = a.mean_in[r], rstd = a.rstd_in[r];
    float2 s = make_float2(0.f, 0.f);
    for (uint32_t c = threadIdx.x; c < cols; c += kLong) {
      const float u = cvt(dy[c]) * (a.w != nullptr ? a.w[c] : 1.f);
      s.x += u;
      s.y = fmaf(u, (cvt(x[c]) - mean) * rstd, s.y);
    }
    s = group_sum<kLong>(s, red, turn++);
    const float m1 = s.x * over, m2 = s.y * over;
    for (uint32_t c = threadIdx.x; c < cols; c += kLong) {
      const float u = cvt(dy[c]) * (a.w != nullptr ? a.w[c] : 1.f);
      put(&dx[c], rstd * (u - m1 - (cvt(x[c]) - mean) * rstd * m2));
    }
  }
}

// ---------------------------------------------------------------------------- slabs
// Longer rows: a block takes kSlab rows at a time.  First a warp per row sums it, twice for the forward pass
// (the second time out of L1); then every thread has its columns of all the rows, with their weights, and in
// the gradient the sums over the rows, in registers.  So weights are read once per block and the block
// meets twice per kSlab rows, where a group of threads per row reads them, and meets, for every row
// (16384 x 4096 bf16: 101 us forward, 173 backward).  Rows of 32 bits do not stay in L1 (16384 x 4096: 123 us
// against 89).
constexpr int kSlabThreads = 512, kSlab = kSlabThreads / 32;

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> keep_vec(const T* p) {  // as load_vec, to be read again soon
  Vec<T, V> r;
  if constexpr (V == 1) {
    r.v[0] = *p;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    memcpy(r.v, &q, 16);
  }
  return r;
}

// Whether a block asks for its next slab's rows (into L2) before the second part of this one: rows of up to 4 KB
// (65536 x 768 bf16: 66 -> 56 us forward, 96 -> 88 backward; 24570 x 2048: 46 -> 43, 83 -> 76; 8192 x 8192: 93 ->
// 110, 138 -> 163).
template <typename T>
__host__ __device__ __forceinline__ bool slab_ahead(int32_t cols) {
  return cols <= 4096 / (int)sizeof(T);
}

// Asks for a row's lines (a warp).
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int32_t cols, int lane) {
  constexpr int kLine = 128 / sizeof(T);
  for (int32_t c = lane * kLine; c < cols; c += 32 * kLine) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The columns of a thread in a slab's second part: vectors t, t + across, ... of rows g, g + groups, ...
struct SlabShare {
  uint32_t vectors, across;
  int t, g, groups;
};
template <int V, int kThreads = kSlabThreads>
__device__ __forceinline__ SlabShare slab_share(int32_t cols) {
  SlabShare s;
  s.vectors = (uint32_t)cols / V;
  s.across = s.vectors < kThreads ? (s.vectors + 31) / 32 * 32 : kThreads;
  s.groups = kThreads / s.across;
  s.g = threadIdx.x / s.across;
  s.t = threadIdx.x % s.across;
  return s;
}

// kThreads: half as many, and rows, where a row is long, but not the longest (16384 x 4096 bf16: 58 us against 62,
// 8192 x 8192: 79 against 93; 65536 x 768: 73 against 56, 4096 x 16384: 113 against 91).
template <typename T, int V, int kN, int kThreads>
__global__ void __launch_bounds__(kThreads, kN * V <= 16 ? 2 : 1)
norm_slab_kernel(const NormArgs a, const Aligned aligned) {
  constexpr int kRows = kThreads / 32;
  using W = Wide<V>;
  constexpr int H = kWide<V>;
  __shared__ float2 stat[kRows];
  const SlabShare sh = slab_share<V, kThreads>(a.cols);
  const float over = 1.f / (float)a.cols;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  W w[kN][H], b[kN][H];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const uint32_t v = sh.t + i * sh.across;
    if (v < sh.vectors) {
      load_weights<V>(a.w == nullptr ? nullptr : a.w + v * V, aligned.w, 1.f, w[i]);
      load_weights<V>(a.b == nullptr ? nullptr : a.b + v * V, aligned.b, 0.f, b[i]);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t mine = r0 + warp;
    float mean = 0.f, rstd = 0.f;
    if (mine < a.rows) {
      const T* x = static_cast<const T*>(a.x) + mine * a.ldx;
      W sum[H];
#pragma unroll
      for (int k = 0; k < H; ++k) sum[k] = both<W>(0.f);
#pragma unroll 8
      for (uint32_t v = lane; v < sh.vectors; v += 32) {
        W e[H];
        widen<T, V>(keep_vec<T, V>(x + v * V), e);
#pragma unroll
        for (int k = 0; k < H; ++k) sum[k] = add2(sum[k], e[k]);
      }
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < H; ++k) s += total(sum[k]);
      mean = warp_sum(s) * over;
#pragma unroll
      for (int k = 0; k < H; ++k) sum[k] = both<W>(0.f);
#pragma unroll 8
      for (uint32_t v = lane; v < sh.vectors; v += 32) {
        W e[H];
        widen<T, V>(keep_vec<T, V>(x + v * V), e);
#pragma unroll
        for (int k = 0; k < H; ++k) {
          e[k] = add2(e[k], both<W>(-mean));
          sum[k] = fma2(e[k], e[k], sum[k]);
        }
      }
      s = 0.f;
#pragma unroll
      for (int k = 0; k < H; ++k) s += total(sum[k]);
      rstd = rsqrtf(warp_sum(s) * over + a.eps);
      if (lane == 0) {
        stat[warp] = make_float2(mean, rstd);
        if (a.mean != nullptr) a.mean[mine] = mean;
        if (a.rstd != nullptr) a.rstd[mine] = rstd;
      }
    }
    if (slab_ahead<T>(a.cols)) {
      const int64_t next = mine + (int64_t)gridDim.x * kRows;
      prefetch_row(static_cast<const T*>(a.x) + next * a.ldx, next < a.rows ? a.cols : 0, lane);
    }
    __syncthreads();
    const int rows = (int)(a.rows - r0 < kRows ? a.rows - r0 : kRows);
    if (sh.g < sh.groups)
#pragma unroll 4
      for (int q = sh.g; q < rows; q += sh.groups) {
        const T* x = static_cast<const T*>(a.x) + (r0 + q) * a.ldx;
        T* y = static_cast<T*>(a.out) + (r0 + q) * a.ldo;
        const float2 st = stat[q];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint32_t v = sh.t + i * sh.across;
          if (v >= sh.vectors) continue;
          W e[H];
          widen<T, V>(load_vec<T, V>(x + v * V), e);
#pragma unroll
          for (int k = 0; k < H; ++k)
            e[k] = fma2(mul2(add2(e[k], both<W>(-st.x)), both<W>(st.y)), w[i][k], b[i][k]);
          store_wide<T, V>(y + v * V, e);
        }
      }
    __syncthreads();
  }
}

// Vector v of the weights in shared memory, which holds planes of 16 bytes of each vector (V = 1: as they are).
template <int V>
__device__ __forceinline__ void plane_weights(const float4* planes, uint32_t vectors, uint32_t v,
                                              Wide<V> (&w)[kWide<V>]) {
  if constexpr (V == 1) {
    w[0] = reinterpret_cast<const float*>(planes)[v];
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 q = planes[k / 4 * vectors + v];
      w[k / 2] = pair(q.x, q.y);
      w[k / 2 + 1] = pair(q.z, q.w);
    }
  }
}

// kBlocks: on an SM at a time.  kThreads: half as many, and rows, two blocks of them, where a row has up to as many
// vectors (24570 x 2048 bf16: 70 us against 75, 1024 x 2048: 13 against 17).  Of longer rows few or very many would
// gain by it (32768 x 4096 bf16: 184 us against 191), those between lose by the second block's sums (4096 x 4096:
// 44 against 41).
template <typename T, int V, int kN, bool kSums, int kBlocks, int kThreads = kSlabThreads>
__global__ void __launch_bounds__(kThreads, kBlocks)
norm_grad_slab_kernel(const NormArgs a, const Aligned aligned) {
  constexpr int kRows = kThreads / 32;
  using W = Wide<V>;
  constexpr int H = kWide<V>;
  extern __shared__ float4 planes[];
  __shared__ float4 stat[kRows];  // mean, rstd, and what dx takes of the row's sums
  const SlabShare sh = slab_share<V, kThreads>(a.cols);
  const float over = 1.f / (float)a.cols;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  W dw[kN][H], db[kN][H];
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int k = 0; k < H; ++k) dw[i][k] = db[i][k] = both<W>(0.f);
  for (uint32_t v = threadIdx.x; v < sh.vectors; v += kThreads) {
    W w[H];
    load_weights<V>(a.w == nullptr ? nullptr : a.w + v * V, aligned.w, 1.f, w);
    if constexpr (V == 1) {
      reinterpret_cast<float*>(planes)[v] = w[0];
    } else {
#pragma unroll
      for (int k = 0; k < H; k += 2)
        planes[k / 2 * sh.vectors + v] =
            make_float4(parts(w[k]).x, parts(w[k]).y, parts(w[k + 1]).x, parts(w[k + 1]).y);
    }
  }
  __syncthreads();
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t mine = r0 + warp;
    if (mine < a.rows) {
      const T* x = static_cast<const T*>(a.x) + mine * a.ldx;
      const T* dy = static_cast<const T*>(a.dy) + mine * a.lddy;
      const float mean = a.mean_in[mine], rstd = a.rstd_in[mine];
      W s1[H], s2[H];
#pragma unroll
      for (int k = 0; k < H; ++k) s1[k] = s2[k] = both<W>(0.f);
#pragma unroll 4
      for (uint32_t v = lane; v < sh.vectors; v += 32) {
        W e[H], d[H], w[H];
        widen<T, V>(keep_vec<T, V>(x + v * V), e);
        widen<T, V>(keep_vec<T, V>(dy + v * V), d);
        plane_weights<V>(planes, sh.vectors, v, w);
#pragma unroll
        for (int k = 0; k < H; ++k) {
          const W u = mul2(d[k], w[k]);
          s1[k] = add2(s1[k], u);
          s2[k] = fma2(u, mul2(add2(e[k], both<W>(-mean)), both<W>(rstd)), s2[k]);
        }
      }
      float m1 = 0.f, m2 = 0.f;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        m1 += total(s1[k]);
        m2 += total(s2[k]);
      }
      m1 = warp_sum(m1) * over;
      m2 = warp_sum(m2) * over;
      if (lane == 0) stat[warp] = make_float4(mean, rstd, -rstd * m1, -rstd * m2);
    }
    if (slab_ahead<T>(a.cols)) {
      const int64_t next = mine + (int64_t)gridDim.x * kRows;
      prefetch_row(static_cast<const T*>(a.x) + next * a.ldx, next < a.rows ? a.cols : 0, lane);
      prefetch_row(static_cast<const T*>(a.dy) + next * a.lddy, next < a.rows ? a.cols : 0, lane);
    }
    __syncthreads();
    const int rows = (int)(a.rows - r0 < kRows ? a.rows - r0 : kRows);
    if (sh.g < sh.groups)
#pragma unroll 2
      for (int q = sh.g; q < rows; q += sh.groups) {
        const T* x = static_cast<const T*>(a.x) + (r0 + q) * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + (r0 + q) * a.lddy;
        T* dx = static_cast<T*>(a.out) + (r0 + q) * a.ldo;
        const float4 st = stat[q];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint32_t v = sh.t + i * sh.across;
          if (v >= sh.vectors) continue;
          W e[H], d[H], w[H];
          widen<T, V>(load_vec<T, V>(x + v * V), e);
          widen<T, V>(load_vec<T, V>(dy + v * V), d);
          plane_weights<V>(planes, sh.vectors, v, w);
          // dx = dy (w rstd) - rstd m1 - xh rstd m2
#pragma unroll
          for (int k = 0; k < H; ++k) {
            const W xh = mul2(add2(e[k], both<W>(-st.x)), both<W>(st.y));
            if constexpr (kSums) {
              dw[i][k] = fma2(d[k], xh, dw[i][k]);
              db[i][k] = add2(db[i][k], d[k]);
            }
            e[k] = fma2(xh, both<W>(st.w), fma2(d[k], mul2(w[k], both<W>(st.y)), both<W>(st.z)));
          }
          store_wide<T, V>(dx + v * V, e);
        }
      }
    __syncthreads();
  }
  if constexpr (kSums) {
    // The groups add their sums to those of the groups before them, in the workspace.
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    const auto value = [](W v, int k) {
      if constexpr (V == 1) return v;
      else return k == 0 ? parts(v).x : parts(v).y;
    };
    constexpr int E = V / H;  // values of a W
    for (int q = 0; q < sh.groups; ++q) {
      if (q > 0) __syncthreads();
      if (sh.g != q) continue;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t v = sh.t + i * sh.across, c = v * V;
        if (v >= sh.vectors) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float x = value(dw[i][k / E], k % E), y = value(db[i][k / E], k % E);
          part[c + k] = q > 0 ? part[c + k] + x : x;
          part[a.cols + c + k] = q > 0 ? part[a.cols + c + k] + y : y;
        }
      }
    }
  }
}

// Column sums of long rows: a block takes 128 columns (blockIdx.x) of the rows blockIdx.y + i gridDim.y.
constexpr int kColumns = 128;
template <typename T>
__global__ void __launch_bounds__(kColumns) norm_columns_kernel(const NormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kColumns + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float d = cvt(static_cast<const T*>(a.dy)[r * a.lddy + c]);
    dw = fmaf(d, (cvt(static_cast<const T*>(a.x)[r * a.ldx + c]) - a.mean_in[r]) * a.rstd_in[r], dw);
    db += d;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.cols;
  part[c] = dw;
  part[a.cols + c] = db;
}

// dw and db from the blocks' sums: 32 threads share a column, a warp reads 32 columns at a time.
__global__ void __launch_bounds__(1024)
norm_parts_kernel(const float* __restrict__ part, int parts, int32_t cols, float* dw, float* db,
                  int accumulate) {
  __shared__ float red[32][33];
  const int64_t wide = 2 * (int64_t)cols;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < wide; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + threadIdx.x % 32;
    float s = 0.f;
    if (c < wide)
#pragma unroll 4
      for (int p = threadIdx.x / 32; p < parts; p += 32) s += part[p * wide + c];
    __syncthreads();
    red[threadIdx.x % 32][threadIdx.x / 32] = s;
    __syncthreads();
    s = red[threadIdx.x / 32][threadIdx.x % 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t mine = c0 + threadIdx.x / 32;
    if (threadIdx.x % 32 == 0 && mine < wide) {
      float* out = mine < cols ? dw : db;
      const int64_t at = mine < cols ? mine : mine - cols;
      if (out != nullptr) out[at] = accumulate ? out[at] + s : s;
    }
  }
}

// ---------------------------------------------------------------------------- launches
// How a row is shared: its vectors, the threads that take them and how many each.
struct RowPlan {
  int v, tpr, n;   // tpr 0: slabs; n 0: too long for registers
  int blocks;      // of the gradient by slabs on an SM
  bool half;       // slabs of half as many rows and threads
};

constexpr int kMostInRegisters = 16384;  // columns
constexpr int kFewRows = 304;            // two for each of 152 SMs
constexpr int kLongRows = 64;            // rows of long ones whose columns a block sums, at least

bool on_16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

RowPlan plan_row(const NormArgs& a, int dtype, bool grad) {
  const int v = dtype == kF32 ? 4 : 8;
  const bool wide = a.cols % v == 0 && on_16(a.x) && on_16(a.out) && a.ldx % v == 0 && a.ldo % v == 0 &&
                    (!grad || (on_16(a.dy) && a.lddy % v == 0));
  const int64_t n = wide ? a.cols / v : a.cols;
  RowPlan p{wide ? v : 1, 0, 0, 1, false};
  if (n <= 8) p.tpr = 8, p.n = 1;
  else if (n <= 32) p.tpr = 32, p.n = 1;
  else if (n <= 512 && a.rows <= kFewRows) p.tpr = 512, p.n = 1;
  else if (dtype != kF32 && grad && !wide && n > 2048 && n <= 8192)  // (16384 x 4097 bf16: slabs 370 us, this 289)
    p.tpr = 512, p.n = 16;
  else if (dtype != kF32) p.n = n <= 512 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : !wide && n <= 8192 ? 16 : 0;
  else if (n <= 512) p.tpr = 128, p.n = 4;
  else if (n <= 1024) p.tpr = 256, p.n = 4;
  else if (n <= 2048) p.tpr = 512, p.n = 4;
  else if (!wide && n <= 8192) p.tpr = 512, p.n = 16;
  if (p.tpr == 0 && p.n == 1 && n <= 128) p.blocks = 2;
  p.half = p.tpr == 0 && p.n > 0 && wide && (grad ? n > 128 && n <= kSlabThreads / 2 : n >= 256 && n <= 1024);
  return p;
}

int64_t rows_per_block(const RowPlan& p) {
  return p.n == 0 ? kLongRows : p.tpr == 0 ? (p.half ? kSlab / 2 : kSlab) : p.tpr > 32 ? 1 : 256 / p.tpr;
}

// The gradient's blocks, each with sums of its own: two or four per SM of 152.
int64_t grad_blocks(const RowPlan& p, int64_t rows) {
  const int64_t per = rows_per_block(p),
                most = p.n == 0 ? 304 : p.tpr == 0 ? 152 * (p.half ? 2 : p.blocks) : p.tpr <= 128 ? 608 : 304;
  const int64_t blocks = (rows + per - 1) / per;
  return blocks < most ? blocks : most;
}

// Allows a kernel's launches so many bytes of dynamic shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || ready->load(std::memory_order_acquire) >> dev & 1) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready->fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// f(V, kTpr, kN) for the plan, with kTpr 0 for slabs.
template <typename T, int V, bool kGrad, typename F>
cudaError_t by_shape(const RowPlan& p, const F& f) {
  const auto v = std::integral_constant<int, V>();
  const auto go = [&](auto tpr, auto n) { return f(v, tpr, n); };
  const std::integral_constant<int, 0> slab;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 4> four;
  const std::integral_constant<int, 16> many;
  if (p.tpr == 8) return go(std::integral_constant<int, 8>(), one);
  if (p.tpr == 32) return go(std::integral_constant<int, 32>(), one);
  if (p.tpr == 512 && p.n == 1) return go(std::integral_constant<int, 512>(), one);
  if constexpr (sizeof(T) == 4) {
    if (p.tpr == 128) return go(std::integral_constant<int, 128>(), four);
    if (p.tpr == 256) return go(std::integral_constant<int, 256>(), four);
    if (p.n == 4) return go(std::integral_constant<int, 512>(), four);
    if constexpr (V == 1) return go(std::integral_constant<int, 512>(), many);
  } else {
    if (p.n == 1) return go(slab, one);
    if (p.n == 2) return go(slab, std::integral_constant<int, 2>());
    if (p.n == 4) return go(slab, four);
    if constexpr (V == 1 && kGrad) return go(std::integral_constant<int, 512>(), many);
    if constexpr (V == 1 && !kGrad) return go(slab, many);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int dtype = sizeof(T) == 4 ? kF32 : kBf16, v = 16 / sizeof(T);
  const RowPlan p = plan_row(a, dtype, false);
  const Aligned aligned{on_16(a.w), on_16(a.b)};
  if (p.n == 0) {
    norm_long_kernel<T><<<(unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms), kLong, 0, st>>>(a);
    return cudaGetLastError();
  }
  // (Blocks that stay ask for their next slab ahead; the others make way for the next block's.)
  const int64_t per = rows_per_block(p), blocks = (a.rows + per - 1) / per,
                cap = (int64_t)sms * (p.tpr == 0 && slab_ahead<T>(a.cols) ? (p.half ? 4 : 2) : p.half ? 16 : 8);
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  const auto go = [&](auto V, auto tpr, auto n) {
    if constexpr (tpr() == 0 && V() > 1 && n() <= 2)
      if (p.half) {
        norm_slab_kernel<T, V(), 2 * n(), kSlabThreads / 2><<<grid, kSlabThreads / 2, 0, st>>>(a, aligned);
        return cudaGetLastError();
      }
    if constexpr (tpr() == 0 && V() > 1 && n() == 2) return cudaErrorInvalidValue;  // (these are all half)
    else if constexpr (tpr() == 0) norm_slab_kernel<T, V(), n(), kSlabThreads><<<grid, kSlabThreads, 0, st>>>(a, aligned);
    else norm_kernel<T, V(), tpr(), n()><<<grid, kBlockThreads<tpr()>, 0, st>>>(a, aligned);
    return cudaGetLastError();
  };
  return p.v == 1 ? by_shape<T, 1, false>(p, go) : by_shape<T, v, false>(p, go);
}

template <typename T>
cudaError_t launch_norm_grad(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int dtype = sizeof(T) == 4 ? kF32 : kBf16, v = 16 / sizeof(T);
  const RowPlan p = plan_row(a, dtype, true);
  const Aligned aligned{on_16(a.w), false};
  const int64_t parts = grad_blocks(p, a.rows);
  const bool sums = a.dw != nullptr || a.db != nullptr;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0 && p.n == 0) {
    norm_grad_long_kernel<T><<<(unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms), kLong, 0, st>>>(a);
    if (sums)
      norm_columns_kernel<T><<<dim3((unsigned)((a.cols - 1) / kColumns + 1), (unsigned)parts), kColumns, 0,
                               st>>>(a);
    e = cudaGetLastError();
  } else if (a.rows > 0) {
    const auto go = [&](auto V, auto tpr, auto n) {
      if constexpr (tpr() == 0) {
        auto kernel = sums ? norm_grad_slab_kernel<T, V(), n(), true, 1> : norm_grad_slab_kernel<T, V(), n(), false, 1>;
        if constexpr (n() == 1)
          if (p.blocks == 2)
            kernel = sums ? norm_grad_slab_kernel<T, V(), n(), true, 2> : norm_grad_slab_kernel<T, V(), n(), false, 2>;
        if constexpr (V() > 1 && n() == 1)
          if (p.half)
            kernel = sums ? norm_grad_slab_kernel<T, V(), 1, true, 2, kSlabThreads / 2>
                          : norm_grad_slab_kernel<T, V(), 1, false, 2, kSlabThreads / 2>;
        const size_t smem = ((size_t)a.cols * 4 + 15) / 16 * 16;
        // Only the longest rows' weights, with the rows' statistics, come near the 48 KB that a launch has by
        // default.  Their kernels are allowed once what any of them may need: a limit that followed each call's
        // rows would refuse another thread's longer ones between its call and its launch.
        constexpr int kMostSmem = kMostInRegisters * 4;
        if constexpr (V() > 1 && n() == 4) {
          static std::atomic<uint64_t> ready[2];
          const cudaError_t s = allow_smem(kernel, kMostSmem, &ready[sums]);
          if (s != cudaSuccess) return s;
        }
        kernel<<<(unsigned)parts, p.half ? kSlabThreads / 2 : kSlabThreads, smem, st>>>(a, aligned);
      } else {
        (sums ? norm_grad_kernel<T, V(), tpr(), n(), true> : norm_grad_kernel<T, V(), tpr(), n(), false>)
            <<<(unsigned)parts, kBlockThreads<tpr()>, 0, st>>>(a, aligned);
      }
      return cudaGetLastError();
    };
    e = p.v == 1 ? by_shape<T, 1, true>(p, go) : by_shape<T, v, true>(p, go);
  }
  if (e != cudaSuccess || !sums) return e;
  const int64_t tiles = (2 * (int64_t)a.cols + 31) / 32, cap = (int64_t)sms * 16;
  norm_parts_kernel<<<(unsigned)(tiles < cap ? tiles : cap), 1024, 0, st>>>(a.part, (int)parts, a.cols, a.dw,
                                                                          a.db, a.accumulate);
  return cudaGetLastError();
}

}  // namespace

size_t norm_grad_workspace(int64_t rows, int32_t cols) {
  // Enough for every plan of a row of so many columns, by the most blocks that any takes.
  const int64_t most = cols > kMostInRegisters ? 304 : 608,
                blocks = cols > kMostInRegisters ? (rows + kLongRows - 1) / kLongRows : rows;
  return (size_t)(blocks < most ? blocks : most) * 2 * (size_t)cols * sizeof(float);
}

cudaError_t launch_layer_norm(const NormArgs& a, int dtype, int sms, cudaStream_t st) {
  return dtype == kF32 ? launch_norm<float>(a, sms, st)
         : dtype == kBf16 ? launch_norm<__nv_bfloat16>(a, sms, st) : launch_norm<__half>(a, sms, st);
}

cudaError_t launch_layer_norm_grad(const NormArgs& a, int dtype, int sms, cudaStream_t st) {
  return dtype == kF32 ? launch_norm_grad<float>(a, sms, st)
         : dtype == kBf16 ? launch_norm_grad<__nv_bfloat16>(a, sms, st)
                          : launch_norm_grad<__half>(a, sms, st);
}

}  // namespace muon
