// The gated activation between the experts' products, and its gradient.
//
//   a = p_r * silu(g) * u,   silu(g) = g * s,   s = 1 / (1 + exp(-g))
//   du = da * p_r * silu(g)
//   dg = da * p_r * u * s * (1 + g * (1 - s))
//   dp_r = sum over the row of da * silu(g) * u
//
// p_r is the router's weight of row r (1 where there is none).  Elementwise work in fp32,
// one rounding at each store, bound by HBM: 3 (5) values move per element.  For 16-bit tensors
// s takes the fast exponential, whose error of about |g| 2^-24 is far below the store's rounding,
// and the fast division (2 ulp): with expf and an IEEE division the gradient was bound by
// instructions.  Where dp, an fp32 result, is asked for, it takes expf.
// 98304 x 1408 in bf16, gradient: 222 us without dp, 227 with it (6.1 TB/s; 10 us more unrolled by
// two, with fewer loads in flight; other grids and streaming stores made no difference).
//
// kTpr threads share a row: a warp where there are many rows (dp then needs shuffles only), a
// block where there are few, so that a small batch still fills the machine with loads
// (192 x 1408: 1.9 us).
#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;

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

// With e = exp(-|x|), 1 / (1 + e) for x >= 0 and e / (1 + e) below: no power overflows and no
// reciprocal is flushed to 0, as that of 1 + exp(-x) would be from x = -87.3 down.
// kFast: what follows from it is rounded to 16 bits.
template <typename T, bool kFast>
__device__ __forceinline__ float sigmoid(float x) {
  const float e = kFast ? __expf(-fabsf(x)) : expf(-fabsf(x));
  const float r = sizeof(T) == 4 ? 1.f / (1.f + e) : __fdividef(1.f, 1.f + e);
  return x < 0.f ? e * r : r;
}

template <typename T, int V, int kTpr>
__global__ void __launch_bounds__(kThreads, 8)
swiglu_kernel(const T* __restrict__ g, int64_t ldg, const T* __restrict__ u, int64_t ldu,
              T* __restrict__ a, int64_t lda, const float* __restrict__ p, int64_t rows,
              int32_t cols) {
  const int t = threadIdx.x % kTpr;
  const int64_t step = (int64_t)gridDim.x * (kThreads / kTpr);
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr; r < rows;
       r += step) {
    const float w = p != nullptr ? p[r] : 1.f;
#pragma unroll 2
    for (uint32_t c = t * V; c < (uint32_t)cols; c += kTpr * V) {
      const Vec<T, V> gv = load_vec<T, V>(g + r * ldg + c), uv = load_vec<T, V>(u + r * ldu + c);
      Vec<T, V> av;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = cvt(gv.v[e]);
        put(&av.v[e], x * sigmoid<T, sizeof(T) == 2>(x) * cvt(uv.v[e]) * w);
      }
      store_vec<T, V>(a + r * lda + c, av);
    }
  }
}

template <typename T, int V, int kTpr, bool kDp>
__global__ void __launch_bounds__(kThreads)
swiglu_grad_kernel(const T* __restrict__ da, int64_t ldda, const T* __restrict__ g, int64_t ldg,
                   const T* __restrict__ u, int64_t ldu, T* __restrict__ dg, int64_t lddg,
                   T* __restrict__ du, int64_t lddu, const float* __restrict__ p,
                   float* __restrict__ dp, int64_t rows, int32_t cols) {
  __shared__ float red[kThreads / 32];
  const int t = threadIdx.x % kTpr;
  const int64_t step = (int64_t)gridDim.x * (kThreads / kTpr);
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr; r < rows;
       r += step) {
    const float w = p != nullptr ? p[r] : 1.f;
    float sum = 0.f;
#pragma unroll 1
    for (uint32_t c = t * V; c < (uint32_t)cols; c += kTpr * V) {
      const Vec<T, V> dv = load_vec<T, V>(da + r * ldda + c), gv = load_vec<T, V>(g + r * ldg + c),
                      uv = load_vec<T, V>(u + r * ldu + c);
      Vec<T, V> gr, ur;
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = cvt(dv.v[e]), x = cvt(gv.v[e]), y = cvt(uv.v[e]);
        const float s = sigmoid<T, sizeof(T) == 2 && !kDp>(x), silu = x * s;
        part = fmaf(d * silu, y, part);
        put(&ur.v[e], d * w * silu);
        put(&gr.v[e], d * w * y * (s * (1.f + x * (1.f - s))));
      }
      sum += part;
      store_vec<T, V>(dg + r * lddg + c, gr);
      store_vec<T, V>(du + r * lddu + c, ur);
    }
    if constexpr (kDp) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if constexpr (kTpr == 32) {
        if (t == 0) dp[r] = sum;
      } else {
        __syncthreads();  // a block shares the row, so every thread is here
        if (t % 32 == 0) red[t / 32] = sum;
        __syncthreads();
        if (t == 0) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < kThreads / 32; ++k) s += red[k];
          dp[r] = s;
        }
      }
    }
  }
}

// Vectors of 16 bytes where every row of every tensor starts on one and the columns fill
// them; single elements otherwise.
template <typename T>
bool vectors(const SwigluArgs& s, int32_t cols) {
  constexpr int v = 16 / sizeof(T);
  if (cols % v != 0) return false;
  for (int i = 0; i < s.n; ++i)
    if (reinterpret_cast<uintptr_t>(s.ptr[i]) % 16 != 0 || s.ld[i] % v != 0) return false;
  return true;
}

template <typename T, int V, int kTpr>
cudaError_t launch_as(const SwigluArgs& s, const float* p, float* dp, int64_t rows, int32_t cols,
                      int sms, cudaStream_t st) {
  const int64_t per = kThreads / kTpr, blocks = (rows + per - 1) / per, cap = (int64_t)sms * 8;
  const int grid = (int)(blocks < cap ? blocks : cap);
  if (s.n == 3)
    swiglu_kernel<T, V, kTpr><<<grid, kThreads, 0, st>>>(
        static_cast<const T*>(s.ptr[0]), s.ld[0], static_cast<const T*>(s.ptr[1]), s.ld[1],
        static_cast<T*>(s.ptr[2]), s.ld[2], p, rows, cols);
  else
    (dp != nullptr ? swiglu_grad_kernel<T, V, kTpr, true> : swiglu_grad_kernel<T, V, kTpr, false>)
        <<<grid, kThreads, 0, st>>>(
            static_cast<const T*>(s.ptr[0]), s.ld[0], static_cast<const T*>(s.ptr[1]), s.ld[1],
            static_cast<const T*>(s.ptr[2]), s.ld[2], static_cast<T*>(s.ptr[3]), s.ld[3],
            static_cast<T*>(s.ptr[4]), s.ld[4], p, dp, rows, cols);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const SwigluArgs& s, const float* p, float* dp, int64_t rows, int32_t cols,
                        int sms, cudaStream_t st) {
  constexpr int v = 16 / sizeof(T);
  // A warp per row where that gives every SM 32 warps, unless a row is long enough to give each
  // thread of a block four accesses (gradient in bf16, us by warps and by blocks: 2048 x 1408 6.9
  // and 7.3, forward 5.9 and 3.9; 4864 x 1408 12.3 and 17.4, 19456 x 64 8.7 and 25.7, 9728 x 14336
  // 225 and 221).
  const bool many = rows >= (int64_t)sms * 32 && cols < 4 * kThreads * (vectors<T>(s, cols) ? v : 1);
  if (vectors<T>(s, cols))
    return many ? launch_as<T, v, 32>(s, p, dp, rows, cols, sms, st)
                : launch_as<T, v, kThreads>(s, p, dp, rows, cols, sms, st);
  return many ? launch_as<T, 1, 32>(s, p, dp, rows, cols, sms, st)
              : launch_as<T, 1, kThreads>(s, p, dp, rows, cols, sms, st);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& s, int dtype, const float* p, float* dp, int64_t rows,
                          int32_t cols, int sms, cudaStream_t st) {
  return dtype == kF32 ? launch_type<float>(s, p, dp, rows, cols, sms, st)
         : dtype == kBf16 ? launch_type<__nv_bfloat16>(s, p, dp, rows, cols, sms, st)
                          : launch_type<__half>(s, p, dp, rows, cols, sms, st);
}

}  // namespace muon
