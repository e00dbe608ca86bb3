// The sigmoid of the gated activation.
#pragma once

#include <cuda_runtime.h>

namespace muon {

// With e = exp(-|x|), 1 / (1 + e) for x >= 0 and e / (1 + e) below: no power overflows and no
// reciprocal is flushed to 0, as that of 1 + exp(-x) would be from x = -87.3 down.
// kFast: what follows from it is rounded to 16 bits.
template <typename T, bool kFast>
__device__ __forceinline__ float sigmoid(float x) {
  const float e = kFast ? __expf(-fabsf(x)) : expf(-fabsf(x));
  const float r = sizeof(T) == 4 ? 1.f / (1.f + e) : __fdividef(1.f, 1.f + e);
  return x < 0.f ? e * r : r;
}

}  // namespace muon
