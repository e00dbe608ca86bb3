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
// kTpr threads share a row (8 or 32 lanes of a warp, or a block), kN vectors each.  In the gradient a
// thread keeps its columns over all the rows of its block and sums dw and db in registers; the
// blocks' sums go to the workspace, and a second kernel adds them in a fixed order, so equal
// inputs give equal bits.
// Rows too long for registers are read again for each sum, and their columns summed by blocks of
// columns in a pass of their own.
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

// V weights from p on (`value` where there are none).
template <int V>
__device__ __forceinline__ void load_weights(const float* p, bool wide, float value, float (&w)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < V; ++k) w[k] = value;
  } else if (V % 4 == 0 && wide) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p + k));
      w[k] = q.x;
      w[(k + 1) % V] = q.y;
      w[(k + 2) % V] = q.z;
      w[(k + 3) % V] = q.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) w[k] = __ldg(p + k);
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

struct Wide {
  bool w, b;  // the weights (biases) start on 16 bytes
};

template <int kTpr>
constexpr int kBlockThreads = kTpr > 32 ? kTpr : 256;

// (Threads without a row stay for the shuffles.)
template <typename T, int V, int kTpr, int kN>
__global__ void __launch_bounds__(kBlockThreads<kTpr>)
norm_kernel(const NormArgs a, const Wide wide) {
  constexpr int kRows = kBlockThreads<kTpr> / kTpr;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % kTpr, g = threadIdx.x / kTpr;
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + g;
    const bool on = r < a.rows;
    const T* x = static_cast<const T*>(a.x) + (on ? r : 0) * a.ldx;
    Vec<T, V> v[kN];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (on && c < cols) v[i] = load_vec<T, V>(x + c);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (on && (uint32_t)(t + i * kTpr) * V < cols)
#pragma unroll
        for (int k = 0; k < V; ++k) s.x += cvt(v[i].v[k]);
    const float mean = group_sum<kTpr>(s, red, turn++).x * over;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (on && (uint32_t)(t + i * kTpr) * V < cols)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = cvt(v[i].v[k]) - mean;
          s.x = fmaf(d, d, s.x);
        }
    const float rstd = rsqrtf(group_sum<kTpr>(s, red, turn++).x * over + a.eps);
    if (on) {
      T* y = static_cast<T*>(a.out) + r * a.ldo;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t c = (uint32_t)(t + i * kTpr) * V;
        if (c >= cols) continue;
        float w[V], b[V];
        load_weights<V>(a.w == nullptr ? nullptr : a.w + c, wide.w, 1.f, w);
        load_weights<V>(a.b == nullptr ? nullptr : a.b + c, wide.b, 0.f, b);
        Vec<T, V> o;
#pragma unroll
        for (int k = 0; k < V; ++k) put(&o.v[k], fmaf((cvt(v[i].v[k]) - mean) * rstd, w[k], b[k]));
        store_vec<T, V>(y + c, o);
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
norm_grad_kernel(const NormArgs a, const Wide wide) {
  constexpr int kThreads = kBlockThreads<kTpr>, kRows = kThreads / kTpr;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % kTpr, g = threadIdx.x / kTpr;
  const uint32_t cols = (uint32_t)a.cols;
  const float over = 1.f / (float)a.cols;
  float dw[kN][V], db[kN][V];
  if constexpr (kSums)
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.f;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + g;
    const bool on = r < a.rows;
    const T* x = static_cast<const T*>(a.x) + (on ? r : 0) * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + (on ? r : 0) * a.lddy;
    const float mean = on ? a.mean_in[r] : 0.f, rstd = on ? a.rstd_in[r] : 0.f;
    Vec<T, V> xv[kN], dv[kN];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (on && c < cols) {
        xv[i] = load_vec<T, V>(x + c);
        dv[i] = load_vec<T, V>(dy + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (!on || c >= cols) continue;
      float w[V];
      load_weights<V>(a.w == nullptr ? nullptr : a.w + c, wide.w, 1.f, w);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = cvt(dv[i].v[k]), xh = (cvt(xv[i].v[k]) - mean) * rstd, u = d * w[k];
        s.x += u;
        s.y = fmaf(u, xh, s.y);
        if constexpr (kSums) {
          dw[i][k] = fmaf(d, xh, dw[i][k]);
          db[i][k] += d;
        }
      }
    }
    s = group_sum<kTpr>(s, red, turn++);
    const float m1 = s.x * over, m2 = s.y * over;
    if (!on) continue;
    T* dx = static_cast<T*>(a.out) + r * a.ldo;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t c = (uint32_t)(t + i * kTpr) * V;
      if (c >= cols) continue;
      float w[V];
      load_weights<V>(a.w == nullptr ? nullptr : a.w + c, wide.w, 1.f, w);
      Vec<T, V> o;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float xh = (cvt(xv[i].v[k]) - mean) * rstd;
        put(&o.v[k], rstd * (fmaf(cvt(dv[i].v[k]), w[k], -m1) - xh * m2));
      }
      store_vec<T, V>(dx + c, o);
    }
  }
  if constexpr (kSums) {
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (kRows == 1) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t c = (uint32_t)(t + i * kTpr) * V;
        if (c >= cols) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          part[c + k] = dw[i][k];
          part[cols + c + k] = db[i][k];
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
            sums[g * kCols + (t + i * kTpr) * V + k] = which == 0 ? dw[i][k] : db[i][k];
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
  int v, tpr, n;  // tpr 0: too long for registers
};

constexpr int kMostInRegisters = 16384;  // columns
constexpr int kLongRows = 64;            // rows of long ones whose columns a block sums, at least

bool on_16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

RowPlan plan_row(const NormArgs& a, int dtype, bool grad) {
  const int v = dtype == kF32 ? 4 : 8;
  const bool wide = a.cols % v == 0 && on_16(a.x) && on_16(a.out) && a.ldx % v == 0 && a.ldo % v == 0 &&
                    (!grad || (on_16(a.dy) && a.lddy % v == 0));
  const int64_t n = wide ? a.cols / v : a.cols;
  RowPlan p{wide ? v : 1, 0, 0};
  if (n <= 8) p.tpr = 8, p.n = 1;
  else if (n <= 32) p.tpr = 32, p.n = 1;
  else if (n <= 128) p.tpr = 32, p.n = 4;
  else if (n <= 256) p.tpr = 256, p.n = 1;
  else if (n <= 512) p.tpr = 512, p.n = 1;
  else if (n <= 1024) p.tpr = 512, p.n = 2;
  else if (n <= 2048) p.tpr = 512, p.n = 4;
  else if (!wide && n <= 8192) p.tpr = 512, p.n = 16;
  return p;
}

int64_t rows_per_block(const RowPlan& p) { return p.tpr > 32 ? 1 : 256 / p.tpr; }

// The gradient's blocks, each with sums of its own: two or four per SM of 152.
int64_t grad_blocks(const RowPlan& p, int64_t rows) {
  const int64_t per = p.tpr == 0 ? kLongRows : rows_per_block(p), most = p.tpr > 32 || p.tpr == 0 ? 304 : 608;
  const int64_t blocks = (rows + per - 1) / per;
  return blocks < most ? blocks : most;
}

// f(type tag, V, kTpr, kN) for the plan.
template <typename T, int V, typename F>
cudaError_t by_shape(const RowPlan& p, const F& f) {
  using std::integral_constant;
  if (p.tpr == 8) return f(integral_constant<int, V>(), integral_constant<int, 8>(), integral_constant<int, 1>());
  if (p.tpr == 32 && p.n == 1)
    return f(integral_constant<int, V>(), integral_constant<int, 32>(), integral_constant<int, 1>());
  if (p.tpr == 32) return f(integral_constant<int, V>(), integral_constant<int, 32>(), integral_constant<int, 4>());
  if (p.tpr == 256) return f(integral_constant<int, V>(), integral_constant<int, 256>(), integral_constant<int, 1>());
  if (p.n == 1) return f(integral_constant<int, V>(), integral_constant<int, 512>(), integral_constant<int, 1>());
  if (p.n == 2) return f(integral_constant<int, V>(), integral_constant<int, 512>(), integral_constant<int, 2>());
  if (p.n == 4) return f(integral_constant<int, V>(), integral_constant<int, 512>(), integral_constant<int, 4>());
  if constexpr (V == 1)
    return f(integral_constant<int, V>(), integral_constant<int, 512>(), integral_constant<int, 16>());
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int dtype = sizeof(T) == 4 ? kF32 : kBf16, v = 16 / sizeof(T);
  const RowPlan p = plan_row(a, dtype, false);
  const Wide wide{on_16(a.w), on_16(a.b)};
  if (p.tpr == 0) {
    norm_long_kernel<T><<<(unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms), kLong, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int64_t per = rows_per_block(p), blocks = (a.rows + per - 1) / per, cap = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  const auto go = [&](auto V, auto tpr, auto n) {
    norm_kernel<T, V(), tpr(), n()><<<grid, kBlockThreads<tpr()>, 0, st>>>(a, wide);
    return cudaGetLastError();
  };
  return p.v == 1 ? by_shape<T, 1>(p, go) : by_shape<T, v>(p, go);
}

template <typename T>
cudaError_t launch_norm_grad(const NormArgs& a, int sms, cudaStream_t st) {
  constexpr int dtype = sizeof(T) == 4 ? kF32 : kBf16, v = 16 / sizeof(T);
  const RowPlan p = plan_row(a, dtype, true);
  const Wide wide{on_16(a.w), false};
  const int64_t parts = grad_blocks(p, a.rows);
  const bool sums = a.dw != nullptr || a.db != nullptr;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0 && p.tpr == 0) {
    norm_grad_long_kernel<T><<<(unsigned)(a.rows < 2 * sms ? a.rows : 2 * sms), kLong, 0, st>>>(a);
    if (sums)
      norm_columns_kernel<T><<<dim3((unsigned)((a.cols - 1) / kColumns + 1), (unsigned)parts), kColumns, 0,
                               st>>>(a);
    e = cudaGetLastError();
  } else if (a.rows > 0) {
    const auto go = [&](auto V, auto tpr, auto n) {
      (sums ? norm_grad_kernel<T, V(), tpr(), n(), true> : norm_grad_kernel<T, V(), tpr(), n(), false>)
          <<<(unsigned)parts, kBlockThreads<tpr()>, 0, st>>>(a, wide);
      return cudaGetLastError();
    };
    e = p.v == 1 ? by_shape<T, 1>(p, go) : by_shape<T, v>(p, go);
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
