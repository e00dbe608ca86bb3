// 8-bit values (e4m3) with a scale for each block of 128.
//
// A block's scale is the smallest power of two s with max|x| / s <= 448, the largest e4m3 value (1 for
// a block of zeros; at least 2^-126): dividing by it is exact, so the only error is the rounding to e4m3,
// to nearest, and equal inputs give equal bits everywhere.  The largest magnitude is taken over the finite
// elements; the others become NaN.
//
// Rows (activations): blocks of 128 columns of a row, 16 threads each.  Weights: blocks of 128 x 128, a
// CTA each, transposed on request through shared memory.  Both read each value once: 24570 x 2048 bf16 32 us
// (4.7 TB/s), 64 x 2048 x 1408 transposed 109 us (5.1 TB/s).
#include <type_traits>

#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;

// The scale of a block by its largest magnitude, and its reciprocal.
__device__ __forceinline__ float block_scale(float amax, float* inverse) {
  const uint32_t b = __float_as_uint(amax);
  // amax = 1.m 2^e; 448 = 1.75 2^8.
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = amax == 0.f ? 0 : e < -126 ? -126 : e;
  *inverse = __uint_as_float((uint32_t)(127 - e) << 23);
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// Two values as e4m3, the first in the low byte.  (The conversion takes infinities to 448.)
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Eight values as they are stored.  Magnitudes compare as integers; from kInf on they are not finite.
template <typename T>
struct Raw {
  static constexpr uint32_t kInf = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  static constexpr int kWords = 2 * (int)sizeof(T);
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
  }

  // From p on, `left` of them inside the row (zeros behind).
  template <bool kWide>
  __device__ __forceinline__ void load(const T* p, int left) {
    if constexpr (kWide) {
      if (left > 0) {
#pragma unroll
        for (int k = 0; k < kWords; k += 4) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + k / 4);
          w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
        }
      } else {
        zero();
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = k < left ? __float_as_uint(p[k]) : 0;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        w[k / 2] = (k < left ? h[k] : 0u) | (k + 1 < left ? (uint32_t)h[k + 1] << 16 : 0u);
    }
  }

  // The largest magnitude's bits.
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, w[k] & 0x7fffffffu);
      return m;
    } else {
      uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
      for (int k = 1; k < 4; ++k) m = __vmaxu2(m, w[k] & 0x7fff7fffu);
      return max(m & 0xffffu, m >> 16);
    }
  }
  // That of the finite values.
  __device__ __forceinline__ uint32_t most_finite() const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = bits(k) & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fffu);
      if (b < kInf) m = max(m, b);
    }
    return m;
  }
  __device__ __forceinline__ uint32_t bits(int k) const {
    if constexpr (sizeof(T) == 4) return w[k];
    else return w[k / 2] >> (16 * (k & 1)) & 0xffffu;
  }
  static __device__ __forceinline__ float value(uint32_t bits) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
    else return unpack_2<T>(bits).x;
  }

  // As e4m3, times `inverse`; odd: there may be infinities, which become NaN.
  __device__ __forceinline__ uint2 convert(float inverse, bool odd) const {
    return odd ? convert_as<true>(inverse) : convert_as<false>(inverse);
  }
  template <bool kOdd>
  __device__ __forceinline__ uint2 convert_as(float inverse) const {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float2 v;
      if constexpr (sizeof(T) == 4) v = make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1]));
      else v = unpack_2<T>(w[k / 2]);
      if constexpr (kOdd) {
        v.x = isinf(v.x) ? __int_as_float(0x7fc00000) : v.x;
        v.y = isinf(v.y) ? __int_as_float(0x7fc00000) : v.y;
      }
      v = parts(mul2(pair(v.x, v.y), pair(inverse, inverse)));
      q[k / 2] = e4m3x2(v.x, v.y);
    }
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
  }
};

__device__ __forceinline__ void store_8_bytes(uint8_t* p, int left, bool wide, uint2 v) {
  if (wide && left >= 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    const uint64_t w = (uint64_t)v.y << 32 | v.x;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) p[k] = (uint8_t)(w >> (8 * k));
  }
}

// kWide: every row of x starts on 16 bytes and has whole groups of eight; q's likewise on 8.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantizeRows a) {
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x % 16, c0 = lane * 8;
  const uint32_t blocks = ((uint32_t)a.cols + 127) / 128;
  const int64_t total = a.rows * blocks, step = (int64_t)gridDim.x * (kThreads / 16);
  // Item i is block i % blocks of row i / blocks; a step moves on by whole rows and some blocks.
  const int64_t rows_on = step / blocks;
  const uint32_t blocks_on = (uint32_t)(step - rows_on * blocks);
  int64_t i = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16, row = i / blocks;
  uint32_t block = (uint32_t)(i - row * blocks);
  // (A warp's two halves end together.)
  for (int64_t first = i - threadIdx.x / 16; first < total; first += kUnroll * step) {
    Raw<T> v[kUnroll];
    int64_t rows[kUnroll];
    uint32_t at[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      rows[j] = row;
      at[j] = block;
      const int64_t c = (int64_t)block * 128 + c0, left = row < a.rows ? a.cols - c : 0;
      v[j].template load<kWide>(static_cast<const T*>(a.x) + row * a.ldx + c, left < 8 ? (int)left : 8);
      row += rows_on;
      block += blocks_on;
      if (block >= blocks) {
        block -= blocks;
        ++row;
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      uint32_t most = v[j].most();
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      const bool odd = most >= Raw<T>::kInf;
      if (__any_sync(0xffffffffu, odd)) {
        uint32_t m = v[j].most_finite();
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        most = m;
      }
      if (rows[j] >= a.rows) continue;
      float inverse;
      const float scale = block_scale(Raw<T>::value(most), &inverse);
      const int64_t c = (int64_t)at[j] * 128 + c0, left = a.cols - c;
      if (left > 0)
        store_8_bytes(a.q + rows[j] * a.ldq + c, left < 8 ? (int)left : 8, kWide, v[j].convert(inverse, odd));
      if (lane == 0) a.scale[at[j] * a.ld_scale + rows[j]] = scale;
    }
  }
}

// Bytes (r, c) of a 4 x 4 block in words by rows to words by columns.
__device__ __forceinline__ void turn(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
  const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, c, 0x5410);
  w[1] = __byte_perm(a, c, 0x7632);
  w[2] = __byte_perm(b, d, 0x5410);
  w[3] = __byte_perm(b, d, 0x7632);
}

// A CTA per block of 128 x 128 of matrix blockIdx.y; a thread takes 4 rows x 8 columns twice.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) quantize_weights_kernel(const QuantizeWeights a) {
  __shared__ uint32_t red[2][2][kThreads / 32];
  __shared__ uint2 turned[128][16];  // [column][8 rows, at (rows / 8) ^ (column / 8)]
  const int64_t rb = ((int64_t)a.rows + 127) / 128, cb = ((int64_t)a.cols + 127) / 128, per = rb * cb;
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;  // 8 columns; 4 rows, and 64 further on
  // The largest of a value over the CTA (`turn` changes from one block to the next).
  const auto most_of_all = [&](uint32_t m, uint32_t (&to)[kThreads / 32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (threadIdx.x % 32 == 0) to[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) m = max(m, to[k]);
    return m;
  };
  int turn_ = 0;
  const int64_t e = blockIdx.y;
  for (int64_t t = blockIdx.x; t < per; t += gridDim.x, turn_ ^= 1) {
    const int64_t bi = per <= INT32_MAX ? (int64_t)((uint32_t)t / (uint32_t)cb) : t / cb, bj = t - bi * cb;
    const int64_t r0 = bi * 128, c0 = bj * 128 + cg * 8;
    const int64_t across = a.cols - c0;
    const int left = across < 0 ? 0 : across < 8 ? (int)across : 8;
    const T* w = static_cast<const T*>(a.w) + e * a.w_stride + r0 * a.ldw + c0;
    Raw<T> v[2][4];
    uint32_t most = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 64 * h + 4 * rg + k;
        v[h][k].template load<kWide>(w + r * a.ldw, r0 + r < a.rows ? left : 0);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) most = max(most, v[h][k].most());
    most = most_of_all(most, red[turn_][0]);  // (also: the block before has left `turned`)
    const bool odd = most >= Raw<T>::kInf;
    if (odd) {
      most = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, v[h][k].most_finite());
      most = most_of_all(most, red[turn_][1]);
    }
    float inverse;
    const float scale = block_scale(Raw<T>::value(most), &inverse);
    if (threadIdx.x == 0)
      a.scale[e * per + (a.transpose ? bj * rb + bi : bi * cb + bj)] = scale;
    if (!a.transpose) {
      uint8_t* q = a.q + e * a.q_stride + r0 * a.ldq + c0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 64 * h + 4 * rg + k;
          if (r0 + r < a.rows) store_8_bytes(q + r * a.ldq, left, a.wide_q, v[h][k].convert(inverse, odd));
        }
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint2 q = v[h][k].convert(inverse, odd);
        lo[k] = q.x;
        hi[k] = q.y;
      }
      turn(lo);
      turn(hi);
      const int four = 16 * h + rg;  // group of 4 rows
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<uint32_t*>(&turned[cg * 8 + j][(four >> 1) ^ cg])[four & 1] = j < 4 ? lo[j] : hi[j - 4];
    }
    __syncthreads();
    // 16 threads per column, eight rows each.
    const int64_t r = r0 + 8 * cg, down = a.rows - r;
    uint8_t* q = a.q + e * a.q_stride + (bj * 128 + rg) * a.ldq + r;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = 16 * k + rg;
      if (bj * 128 + c < a.cols && down > 0)
        store_8_bytes(q + 16 * k * a.ldq, down < 8 ? (int)down : 8, a.wide_q, turned[c][cg ^ (c >> 3)]);
    }
  }
}

bool on(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
cudaError_t rows_as(const QuantizeRows& a, int sms, cudaStream_t st) {
  constexpr int v = 16 / sizeof(T);
  const int64_t blocks = a.rows * (((int64_t)a.cols + 127) / 128), per = kThreads / 16,
                need = (blocks + 4 * per - 1) / (4 * per), cap = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  const bool wide = a.cols % 8 == 0 && on(a.x, 16) && a.ldx % v == 0 && on(a.q, 8) && a.ldq % 8 == 0;
  (wide ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>)<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t weights_as(QuantizeWeights a, int sms, cudaStream_t st) {
  constexpr int v = 16 / sizeof(T);
  const int64_t blocks = (((int64_t)a.rows + 127) / 128) * (((int64_t)a.cols + 127) / 128), cap = (int64_t)sms * 32;
  const dim3 grid((unsigned)(blocks < cap ? blocks : cap), (unsigned)a.n);
  const bool wide = a.cols % 8 == 0 && on(a.w, 16) && a.ldw % v == 0 && (a.n == 1 || a.w_stride % v == 0);
  a.wide_q = on(a.q, 8) && a.ldq % 8 == 0 && (a.n == 1 || a.q_stride % 8 == 0);
  (wide ? quantize_weights_kernel<T, true> : quantize_weights_kernel<T, false>)<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeRows& a, int dtype, int sms, cudaStream_t st) {
  return dtype == kF32 ? rows_as<float>(a, sms, st)
         : dtype == kBf16 ? rows_as<__nv_bfloat16>(a, sms, st) : rows_as<__half>(a, sms, st);
}

cudaError_t launch_quantize_weights(const QuantizeWeights& a, int dtype, int sms, cudaStream_t st) {
  return dtype == kF32 ? weights_as<float>(a, sms, st)
         : dtype == kBf16 ? weights_as<__nv_bfloat16>(a, sms, st) : weights_as<__half>(a, sms, st);
}

}  // namespace muon
