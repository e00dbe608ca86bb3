// Global gradient norm over many tensors, and clipping by it.
//
//   ||g|| = sqrt(sum over tensors and elements of g^2)
//   coef  = min(1, max_norm / (||g|| + 1e-6))
//   out   = coef * g
//
// Two launches: every block sums the squares of its chunks into one double; then every
// block of the second launch adds those sums in the same fixed order (about ten kilobytes
// from L2), so no block waits on another, no atomic decides an order, and the result does
// not depend on timing.  Both are bound by HBM: the gradients are read twice unless L2
// still holds them, which is why the second launch walks each block's chunks backwards.
// 574 M fp32 elements in 196 tensors: 332 us (6.9 TB/s) and 713 us (6.3 TB/s) alone, 1036 us
// together; 8.8 us for ten tensors of 0.36 M.  (Where a Muon step follows, muon_step_scaled
// takes the coefficient, and the second launch is not needed: on the 85 M gradients of 12
// GPT-2-small layers clipping then costs 67 us instead of 175.)
//
// Sums: a thread adds at most 32 squares in fp32 (in four sums), then goes on in double.
// A thread whose fp32 sum overflowed, or is so small that squares may have been flushed,
// takes those elements again in double, so the whole fp32 range is covered.
#include "device_common.cuh"
#include "element.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
// Four resident blocks per SM, 64 bytes in flight per thread, and chunks fine enough for equal
// shares (27 M elements: 58 us; with chunks of 32 KB and 8 blocks, three of them resident, 72).
constexpr int kBlocksPerSm = 4;
constexpr int kChunkBytes = 16384;
constexpr int kIter = kChunkBytes / 16 / kThreads;

// One tensor of a launch.  Chunk j of the tensor covers bytes j * kChunkBytes to
// (j + 1) * kChunkBytes counted from the 16-byte boundary below its start, mis elements before
// it: every chunk's vectors are aligned wherever the tensor starts.
struct TensorRec {
  const void* g;
  void* out;
  int64_t numel;
  int32_t chunk_begin;
  int8_t dtype, out_dtype;
  int8_t mis, pad_;
};

template <int N>
struct TensorArgs {
  TensorRec t[N];
  int32_t n, n_chunks;
};

// Index of the tensor that holds a chunk.
template <int N>
__device__ __forceinline__ int find_tensor(const TensorArgs<N>& a, int chunk) {
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].chunk_begin <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Block b's chunks: an equal share in one run, so that the tensor is looked up once.
template <int N>
__device__ __forceinline__ int2 chunk_range(const TensorArgs<N>& a) {
  return make_int2((int)((int64_t)a.n_chunks * blockIdx.x / gridDim.x),
                   (int)((int64_t)a.n_chunks * (blockIdx.x + 1) / gridDim.x));
}

// This thread's elements of a chunk: kIter vectors of kVec.
template <typename T>
struct ChunkIter {
  static constexpr int kVec = 16 / sizeof(T);
  // First element of vector u (before or behind the tensor's elements, or across its ends, in
  // its first and last chunk).
  __device__ static int64_t first(const TensorRec& t, int64_t j, int u) {
    return j * (kChunkBytes / (int)sizeof(T)) + (threadIdx.x + u * kThreads) * kVec - t.mis;
  }
  // Elements outside the tensor read as zero.
  __device__ static void load(const TensorRec& t, int64_t i, T (&v)[kVec]) {
    const T* g = static_cast<const T*>(t.g);
    if (i >= 0 && i + kVec <= t.numel) {
      const uint4 q = *reinterpret_cast<const uint4*>(g + i);
      memcpy(v, &q, 16);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        v[e] = (i + e >= 0 && i + e < t.numel) ? g[i + e] : static_cast<T>(0.f);
    }
  }
};

template <typename T>
__device__ __forceinline__ double chunk_sum(const TensorRec& t, int64_t j) {
  using C = ChunkIter<T>;
  T v[kIter][C::kVec];
#pragma unroll
  for (int u = 0; u < kIter; ++u) C::load(t, C::first(t, j, u), v[u]);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  bool nonzero = false;
#pragma unroll
  for (int u = 0; u < kIter; ++u)
#pragma unroll
    for (int e = 0; e < C::kVec; ++e) {
      const float f = cvt(v[u][e]);
      s[e & 3] = fmaf(f, f, s[e & 3]);
      nonzero |= f != 0.f;  // true for NaN as well
    }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  if (nonzero && !(sum >= 0x1p-100f && sum <= 0x1p126f)) {
    double d = 0.0;
#pragma unroll 1
    for (int u = 0; u < kIter; ++u) {  // read again: rare
      T w[C::kVec];
      C::load(t, C::first(t, j, u), w);
#pragma unroll
      for (int e = 0; e < C::kVec; ++e) d = fma((double)cvt(w[e]), (double)cvt(w[e]), d);
    }
    return d;
  }
  return (double)sum;
}
static_assert(kIter == 4, "chunk_sum and the bound on a thread's squares");

// The same order every run; the result is valid in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
sum_squares_kernel(const __grid_constant__ TensorArgs<N> a, double* __restrict__ partials) {
  __shared__ double red[kThreads / 32];
  double s = 0.0;
  const int2 r = chunk_range(a);
  int i = r.x < r.y ? find_tensor(a, r.x) : 0;
  for (int c = r.x; c < r.y; ++c) {
    while (i + 1 < a.n && a.t[i + 1].chunk_begin <= c) ++i;
    const TensorRec& t = a.t[i];
    const int64_t j = c - t.chunk_begin;
    s += t.dtype == kF32 ? chunk_sum<float>(t, j)
         : t.dtype == kBf16 ? chunk_sum<__nv_bfloat16>(t, j) : chunk_sum<__half>(t, j);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// Norm and coefficient from the partial sums (every thread of the block gets both).
__device__ __forceinline__ float2 norm_and_coef(const double* partials, int n, float max_norm,
                                                double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partials[i];
  const double norm = sqrt(block_sum(s, red));
  double c = (double)max_norm / (norm + 1e-6);
  if (c > 1.0) c = 1.0;  // a NaN norm keeps a NaN coefficient
  return make_float2((float)norm, (float)c);
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(const double* __restrict__ partials, int n, float max_norm, float* __restrict__ norm) {
  __shared__ double red[kThreads / 32];
  const float2 nc = norm_and_coef(partials, n, max_norm, red);
  if (threadIdx.x == 0) {
    norm[0] = nc.x;
    norm[1] = nc.y;
  }
}

template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const TensorRec& t, int64_t j, float c) {
  using C = ChunkIter<T>;
  constexpr int kVec = C::kVec, kPieces = kVec * sizeof(O) / 16;  // 16-byte pieces out
  T v[kIter][kVec];
#pragma unroll
  for (int u = 0; u < kIter; ++u) C::load(t, C::first(t, j, u), v[u]);
  O* out = static_cast<O*>(t.out);
#pragma unroll
  for (int u = 0; u < kIter; ++u) {
    const int64_t i = C::first(t, j, u);
    O r[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) put(&r[e], cvt(v[u][e]) * c);
    if (i >= 0 && i + kVec <= t.numel && reinterpret_cast<uintptr_t>(out + i) % 16 == 0) {
#pragma unroll
      for (int b = 0; b < kPieces; ++b) {
        uint4 q;
        memcpy(&q, r + b * (kVec / kPieces), 16);
        reinterpret_cast<uint4*>(out + i)[b] = q;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (i + e >= 0 && i + e < t.numel) out[i + e] = r[e];
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
clip_kernel(const __grid_constant__ TensorArgs<N> a, const double* __restrict__ partials,
            int n_partials, float max_norm, float* __restrict__ norm) {
  __shared__ double red[kThreads / 32];
  const int2 r = chunk_range(a);
  int i = r.x < r.y ? find_tensor(a, r.y - 1) : 0;
  const float2 nc = norm_and_coef(partials, n_partials, max_norm, red);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = nc.x;
    norm[1] = nc.y;
  }
  for (int c = r.y - 1; c >= r.x; --c) {
    while (a.t[i].chunk_begin > c) --i;
    const TensorRec& t = a.t[i];
    if (nc.y == 1.f && t.out == t.g) continue;  // in place and not clipped: already there
    const int64_t j = c - t.chunk_begin;
    if (t.dtype == kF32) scale_chunk<float, float>(t, j, nc.y);
    else if (t.dtype == kBf16 && t.out_dtype == kF32) scale_chunk<__nv_bfloat16, float>(t, j, nc.y);
    else if (t.dtype == kBf16) scale_chunk<__nv_bfloat16, __nv_bfloat16>(t, j, nc.y);
    else if (t.out_dtype == kF32) scale_chunk<__half, float>(t, j, nc.y);
    else scale_chunk<__half, __half>(t, j, nc.y);
  }
}

// Kernel arguments hold up to kMany records by value (they must stay below 32,764 bytes);
// calls with fewer tensors take smaller forms, whose launches copy less.
constexpr int kFew = 32, kSome = 256, kMany = 960;
static_assert(sizeof(TensorArgs<kMany>) + 64 < 32764, "kernel arguments too large");

int esize(int dtype) { return dtype == kF32 ? 4 : 2; }

int64_t misalign(const TensorSpec& g) {
  return (int64_t)(reinterpret_cast<uintptr_t>(g.data) % 16) / esize(g.dtype);
}

int64_t chunks_of(const TensorSpec& g) {
  const int64_t chunk = kChunkBytes / esize(g.dtype);
  return g.numel == 0 ? 0 : (g.numel + misalign(g) + chunk - 1) / chunk;
}

// The tensors from *at on that one launch takes; outs may be null (norm only).
template <int N>
void fill(const TensorSpec* grads, const TensorSpec* outs, int n, int* at, TensorArgs<N>* a) {
  a->n = 0;
  int64_t chunks = 0;
  for (; *at < n && a->n < N; ++*at) {
    const TensorSpec& g = grads[*at];
    const int64_t c = chunks_of(g);
    if (c == 0) continue;
    TensorRec& r = a->t[a->n++];
    r.g = g.data;
    r.out = outs != nullptr ? outs[*at].data : nullptr;
    r.numel = g.numel;
    r.chunk_begin = (int32_t)chunks;
    r.dtype = (int8_t)g.dtype;
    r.out_dtype = (int8_t)(outs != nullptr ? outs[*at].dtype : g.dtype);
    r.mis = (int8_t)misalign(g);
    r.pad_ = 0;
    chunks += c;
  }
  a->n_chunks = (int32_t)chunks;
}

int grid_of(int64_t chunks, int sms) {
  const int64_t cap = (int64_t)sms * kBlocksPerSm;
  return (int)(chunks < cap ? chunks : cap);
}

template <int N>
cudaError_t run_clip(const TensorSpec* grads, const TensorSpec* outs, int n, float max_norm,
                     float* norm, double* partials, int sms, cudaStream_t st) {
  int n_partials = 0;
  for (int at = 0; at < n;) {
    TensorArgs<N> a;
    fill(grads, nullptr, n, &at, &a);
    if (a.n == 0) break;
    const int grid = grid_of(a.n_chunks, sms);
    sum_squares_kernel<N><<<grid, kThreads, 0, st>>>(a, partials + n_partials);
    n_partials += grid;
  }
  bool wrote = false;
  if (outs != nullptr)
    for (int at = 0; at < n;) {
      TensorArgs<N> a;
      fill(grads, outs, n, &at, &a);
      if (a.n == 0) break;
      clip_kernel<N><<<grid_of(a.n_chunks, sms), kThreads, 0, st>>>(a, partials, n_partials,
                                                                    max_norm, norm);
      wrote = true;
    }
  if (!wrote) norm_kernel<<<1, kThreads, 0, st>>>(partials, n_partials, max_norm, norm);
  return cudaGetLastError();
}

}  // namespace

int64_t clip_chunks(const TensorSpec* grads, int n) {
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) chunks += chunks_of(grads[i]);
  return chunks;
}

size_t clip_workspace_bytes(const TensorSpec* grads, int n, int sms) {
  // One double per block of the summing launches (kMany tensors each, or all in one); a
  // bound that holds wherever the tensors start.
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) chunks += grads[i].numel > 0 ? grads[i].numel * 4 / kChunkBytes + 2 : 0;
  const int64_t slots = (int64_t)((n + kMany - 1) / kMany) * sms * kBlocksPerSm;
  return (size_t)(chunks < slots ? chunks : slots) * sizeof(double);
}

cudaError_t launch_clip(const TensorSpec* grads, const TensorSpec* outs, int n, float max_norm,
                        float* norm, void* ws, int sms, cudaStream_t st) {
  double* partials = static_cast<double*>(ws);
  return n <= kFew ? run_clip<kFew>(grads, outs, n, max_norm, norm, partials, sms, st)
         : n <= kSome ? run_clip<kSome>(grads, outs, n, max_norm, norm, partials, sms, st)
                      : run_clip<kMany>(grads, outs, n, max_norm, norm, partials, sms, st);
}

}  // namespace muon
