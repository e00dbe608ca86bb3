// Blocks of rows that a sum over an expert's rows goes through, in arithmetic that holds for every
// row count from 0 to 2^31 - 1 (on the host too, where it is tested).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MUON_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MUON_HOST_DEVICE inline
#endif

namespace muon {

constexpr int kBK = 64;  // k-block: 128 bytes of a 16-bit row

MUON_HOST_DEVICE int32_t row_blocks(int32_t rows) { return rows / kBK + (rows % kBK != 0); }

// The share of `index` among 2^shift CTAs that sum the rows together: whole blocks.
struct RowShare {
  int32_t first, rows;
};
MUON_HOST_DEVICE RowShare row_share(int32_t rows, int index, int shift) {
  const int64_t blocks = row_blocks(rows);
  const int64_t begin = (blocks * index >> shift) * kBK, end = (blocks * (index + 1) >> shift) * kBK;
  return {(int32_t)begin, (int32_t)((end < rows ? end : rows) - begin)};
}

// k-blocks of each of a sum's segments (at most `most`, a multiple of sub), whole stages of `sub`
// and of equal number up to the last segment.
MUON_HOST_DEVICE int32_t segment_blocks(int32_t k_blocks, int most, int sub) {
  const int32_t n = k_blocks / most + (k_blocks % most != 0);
  const int32_t len = n > 1 ? k_blocks / n + (k_blocks % n != 0) : k_blocks;
  return (len + sub - 1) / sub * sub;
}

}  // namespace muon
