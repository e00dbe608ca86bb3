// Products grouped by expert over ragged rows.
//
//   mm:    y[r, :] = x[r, :] W_e           (W_e stored k x n)
//          y[r, :] = x[r, :] W_e^T         (W_e stored n x k, trans)
//   wgrad: dW_e (+)= sum over the rows r of expert e of a[r, :]^T b[r, :]
//
// Expert e owns rows offsets[e] .. offsets[e + 1] - 1.  The offsets are on the device, so
// every block reads them, checks them and works out its own tile; rows of no expert (before
// offsets[0], from offsets[n_experts] on) get zeros.
#include "device_common.cuh"
#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kStep = 16;

// Reads the row offsets into shared memory.  If they are not ascending within 0..rows, no
// expert gets a row and kErrRowOffsets is recorded.
__device__ __forceinline__ void load_offsets(const int64_t* offsets, int n_experts, int64_t rows,
                                             int32_t* off, int* err) {
  bool bad = false;
  for (int e = threadIdx.x; e <= n_experts; e += blockDim.x) {
    const int64_t o = offsets[e];
    bad |= o < 0 || o > rows || (e > 0 && offsets[e - 1] > o);
    off[e] = (int32_t)o;
  }
  if (__syncthreads_or(bad)) {
    for (int e = threadIdx.x; e <= n_experts; e += blockDim.x) off[e] = 0;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(err, kErrRowOffsets);
    __syncthreads();
  }
}

// c[4][4] += A-tile x B-tile over `depth`, from shared memory stored depth-major.
__device__ __forceinline__ void fma_tile(const float (&as)[kStep][kTile], const float (&bs)[kStep][kTile],
                                         int ty, int tx, float (&c)[4][4]) {
#pragma unroll
  for (int q = 0; q < kStep; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = fmaf(as[q][ty * 4 + i], bs[q][tx * 4 + j], c[i][j]);
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) mm_kernel(const GroupedMm p) {
  __shared__ int32_t off[kMaxExperts + 1];
  __shared__ float as[kStep][kTile], bs[kStep][kTile];
  load_offsets(p.offsets, p.n_experts, p.rows, off, p.err);
  const T* x = static_cast<const T*>(p.x);
  O* y = static_cast<O*>(p.y);
  // Tiles of expert 0, 1, ... and then of the rows of no expert.
  int tile = blockIdx.x, e = 0;
  for (; e < p.n_experts; ++e) {
    const int tiles = (off[e + 1] - off[e] + kTile - 1) / kTile;
    if (tile < tiles) break;
    tile -= tiles;
  }
  const int j0 = blockIdx.y * kTile, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  if (e == p.n_experts) {
    const int64_t head = off[0], tail = p.rows - off[p.n_experts];
    for (int q = threadIdx.x; q < kTile * kTile; q += kThreads) {
      const int64_t z = (int64_t)tile * kTile + q / kTile;
      const int j = j0 + q % kTile;
      if (z < head + tail && j < p.n)
        put(&y[(z < head ? z : off[p.n_experts] + z - head) * p.ldy + j], 0.f);
    }
    return;
  }
  const int64_t r0 = off[e] + (int64_t)tile * kTile;
  const int rows = min(kTile, (int)(off[e + 1] - r0));
  const T* w = static_cast<const T*>(p.w) + e * p.w_stride;
  float c[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += kStep) {
    for (int q = threadIdx.x; q < kStep * kTile; q += kThreads) {
      const int i = q / kStep, d = q % kStep;
      as[d][i] = (i < rows && k0 + d < p.k) ? cvt(x[(r0 + i) * p.ldx + k0 + d]) : 0.f;
      const int jj = p.trans ? i : q % kTile, dd = p.trans ? d : q / kTile;
      const bool in = j0 + jj < p.n && k0 + dd < p.k;
      bs[dd][jj] = !in ? 0.f
                   : cvt(p.trans ? w[(int64_t)(j0 + jj) * p.ldw + k0 + dd]
                                 : w[(int64_t)(k0 + dd) * p.ldw + j0 + jj]);
    }
    __syncthreads();
    fma_tile(as, bs, ty, tx, c);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (ty * 4 + i < rows && j0 + tx * 4 + j < p.n)
        put(&y[(r0 + ty * 4 + i) * p.ldy + j0 + tx * 4 + j], c[i][j]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(const GroupedWgrad p) {
  __shared__ int32_t off[kMaxExperts + 1];
  __shared__ float as[kStep][kTile], bs[kStep][kTile];
  load_offsets(p.offsets, p.n_experts, p.rows, off, p.err);
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  const int tiles_m = (p.m + kTile - 1) / kTile;
  const int e = blockIdx.x / tiles_m, i0 = blockIdx.x % tiles_m * kTile, j0 = blockIdx.y * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float c[4][4] = {};
  for (int r0 = off[e]; r0 < off[e + 1]; r0 += kStep) {
    for (int q = threadIdx.x; q < kStep * kTile; q += kThreads) {
      const int i = q % kTile, d = q / kTile;
      const bool in = r0 + d < off[e + 1];
      as[d][i] = in && i0 + i < p.m ? cvt(a[(int64_t)(r0 + d) * p.lda + i0 + i]) : 0.f;
      bs[d][i] = in && j0 + i < p.n ? cvt(b[(int64_t)(r0 + d) * p.ldb + j0 + i]) : 0.f;
    }
    __syncthreads();
    fma_tile(as, bs, ty, tx, c);
    __syncthreads();
  }
  float* dw = p.dw + e * p.dw_stride;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (i0 + ty * 4 + i < p.m && j0 + tx * 4 + j < p.n) {
        float* o = dw + (int64_t)(i0 + ty * 4 + i) * p.lddw + j0 + tx * 4 + j;
        *o = p.accumulate ? *o + c[i][j] : c[i][j];
      }
}

template <typename T>
cudaError_t launch_mm(const GroupedMm& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.rows + kTile - 1) / kTile + p.n_experts + 2), (p.n + kTile - 1) / kTile);
  if (p.out_dtype == kF32) mm_kernel<T, float><<<grid, kThreads, 0, st>>>(p);
  else mm_kernel<T, T><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_mm(const GroupedMm& p, cudaStream_t st) {
  return p.dtype == kBf16 ? launch_mm<__nv_bfloat16>(p, st) : launch_mm<__half>(p, st);
}

cudaError_t launch_grouped_wgrad(const GroupedWgrad& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.m + kTile - 1) / kTile) * p.n_experts, (p.n + kTile - 1) / kTile);
  if (p.dtype == kBf16) wgrad_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  else wgrad_kernel<__half><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace muon
