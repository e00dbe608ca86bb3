// 8-bit values (e4m3) with a scale for each block of 128.
//
// A block's scale is the smallest power of two s with max|x| / s <= 448, the largest e4m3 value (1 for
// a block of zeros; at least 2^-126): dividing by it is exact, so the only error is the rounding to e4m3,
// to nearest, and equal inputs give equal bits everywhere.  The largest magnitude is taken over the finite
// elements; the others become NaN.
//
// Rows (activations): blocks of 128 columns of a row, 16 threads each.  Weights: blocks of 128 x 128, a
// CTA each, transposed on request through shared memory.  Both read each value once and are bound by HBM.
#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float finite_abs(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? __uint_as_float(b) : 0.f;
}

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
__device__ __forceinline__ float or_nan(float v) { return isinf(v) ? __int_as_float(0x7fc00000) : v; }
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float inverse) {
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = or_nan(v[k]) * inverse;
  return make_uint2(e4m3x2(s[0], s[1]) | e4m3x2(s[2], s[3]) << 16, e4m3x2(s[4], s[5]) | e4m3x2(s[6], s[7]) << 16);
}

// Eight values from p on, `left` of them inside the row (zeros behind).
template <typename T, bool kWide>
__device__ __forceinline__ void load_8(const T* p, int left, float (&v)[8]) {
  if constexpr (kWide) {
    if (left > 0) {
      __align__(16) T t[8];
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k)
        reinterpret_cast<uint4*>(t)[k] = __ldcs(reinterpret_cast<const uint4*>(p) + k);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = cvt(t[k]);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < left ? cvt(p[k]) : 0.f;
}

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
  const int lane = threadIdx.x % 16;
  const uint32_t blocks = ((uint32_t)a.cols + 127) / 128;
  const int64_t total = a.rows * blocks, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; i0 - threadIdx.x / 16 < total;
       i0 += kUnroll * step) {
    float v[kUnroll][8];
    int64_t row[kUnroll];
    uint32_t block[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int64_t i = i0 + j * step;
      row[j] = total <= INT32_MAX ? (int64_t)((uint32_t)i / blocks) : i / blocks;
      block[j] = (uint32_t)(i - row[j] * blocks);
      const int64_t c = (int64_t)block[j] * 128 + lane * 8, left = i < total ? a.cols - c : 0;
      load_8<T, kWide>(static_cast<const T*>(a.x) + row[j] * a.ldx + c, left < 8 ? (int)left : 8, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_abs(v[j][k]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (i0 + j * step >= total) continue;
      float inverse;
      const float scale = block_scale(amax, &inverse);
      const int64_t c = (int64_t)block[j] * 128 + lane * 8, left = a.cols - c;
      if (left > 0)
        store_8_bytes(a.q + row[j] * a.ldq + c, left < 8 ? (int)left : 8, kWide, e4m3x8(v[j], inverse));
      if (lane == 0) a.scale[block[j] * a.ld_scale + row[j]] = scale;
    }
  }
}

// A CTA per block of 128 x 128; a thread takes 4 rows x 8 columns twice.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(const QuantizeWeights a) {
  __shared__ float red[2][kThreads / 32];
  __shared__ uint2 turned[128][16];  // [column][8 rows, at (rows / 8) ^ (column / 8)]
  const int64_t rb = ((int64_t)a.rows + 127) / 128, cb = ((int64_t)a.cols + 127) / 128, per = rb * cb;
  const int cg = threadIdx.x % 16, rg = threadIdx.x / 16;  // 8 columns; 4 rows, and 64 further on
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.n * per; t += gridDim.x, ++turn) {
    const int64_t e = t / per, bi = (t - e * per) / cb, bj = t - e * per - bi * cb;
    const int64_t r0 = bi * 128, c0 = bj * 128 + cg * 8;
    const int64_t across = a.cols - c0;
    const int left = across < 0 ? 0 : across < 8 ? (int)across : 8;
    float v[2][4][8], amax = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t r = r0 + 64 * h + 4 * rg + k;
        load_8<T, kWide>(static_cast<const T*>(a.w) + e * a.w_stride + r * a.ldw + c0, r < a.rows ? left : 0,
                         v[h][k]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[h][k][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (threadIdx.x % 32 == 0) red[turn & 1][threadIdx.x / 32] = amax;
    __syncthreads();  // (also: the previous block has left `turned`)
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) amax = fmaxf(amax, red[turn & 1][k]);
    float inverse;
    const float scale = block_scale(amax, &inverse);
    if (threadIdx.x == 0)
      a.scale[e * per + (a.transpose ? bj * rb + bi : bi * cb + bj)] = scale;
    if (!a.transpose) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t r = r0 + 64 * h + 4 * rg + k;
          if (r < a.rows)
            store_8_bytes(a.q + e * a.q_stride + r * a.ldq + c0, left, a.wide_q, e4m3x8(v[h][k], inverse));
        }
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = e4m3x8(v[h][k], inverse);
      const int four = 16 * h + rg;  // group of 4 rows
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) w |= ((j < 4 ? q[k].x : q[k].y) >> (8 * (j & 3)) & 0xffu) << (8 * k);
        reinterpret_cast<uint32_t*>(&turned[cg * 8 + j][(four >> 1) ^ cg])[four & 1] = w;
      }
    }
    __syncthreads();
    // 16 threads per column, eight rows each.
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = 16 * k + rg, eight = cg;
      const int64_t col = bj * 128 + c, r = r0 + 8 * eight, down = a.rows - r;
      if (col < a.cols && down > 0)
        store_8_bytes(a.q + e * a.q_stride + col * a.ldq + r, down < 8 ? (int)down : 8, a.wide_q,
                      turned[c][eight ^ (c >> 3)]);
    }
  }
}

bool on(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
cudaError_t rows_as(const QuantizeRows& a, int sms, cudaStream_t st) {
  constexpr int v = 16 / sizeof(T);
  const int64_t blocks = a.rows * (((int64_t)a.cols + 127) / 128), per = kThreads / 16,
                need = (blocks + 4 * per - 1) / (4 * per), cap = (int64_t)sms * 32;
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  const bool wide = a.cols % 8 == 0 && on(a.x, 16) && a.ldx % v == 0 && on(a.q, 8) && a.ldq % 8 == 0;
  (wide ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>)<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t weights_as(QuantizeWeights a, int sms, cudaStream_t st) {
  constexpr int v = 16 / sizeof(T);
  const int64_t tiles = a.n * (((int64_t)a.rows + 127) / 128) * (((int64_t)a.cols + 127) / 128),
                cap = (int64_t)sms * 32;
  const unsigned grid = (unsigned)(tiles < cap ? tiles : cap);
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
