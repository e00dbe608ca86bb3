// The sigmoid of the gated activation, one by one and two at a time.
#pragma once

#include <cuda_runtime.h>

#include "element.cuh"

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

// The same of two values.  exp(-|x|) is the square of 2^(-|x| log2(e) / 2), which stays normal wherever exp(-|x|) is
// not zero in fp32, so that the fast power, which flushes subnormals, does for all x; 1 + e lies in 1 .. 2, where the
// fast reciprocal is within an ulp.  The rounded argument puts exp(-|x|) off by up to |x| 2^-24.  kFine, for results
// of 32 bits, makes up for that: what the rounding left of the argument, times ln 2, is the power's relative error.
template <bool kFine>
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  const float2 v = parts(x);
  float2 h, r;
  const float half_log2e = 0.72134752f;
  f32x2 hh;
  if constexpr (kFine) {
    // (From 104 on e is zero, and an infinite x would leave NaN.)
    const f32x2 size = pair(fminf(fabsf(v.x), 128.f), fminf(fabsf(v.y), 128.f));
    const f32x2 arg = mul2(size, pair(-half_log2e, -half_log2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h.x) : "f"(parts(arg).x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h.y) : "f"(parts(arg).y));
    // (A product and what its rounding left, by two fused multiply-adds; log2(e) / 2 is half_log2e + 9.63e-9.)
    const f32x2 left = fma2(size, pair(9.6298e-9f, 9.6298e-9f), fma2(size, pair(half_log2e, half_log2e), arg));
    hh = pair(h.x, h.y);
    hh = fma2(hh, mul2(left, pair(-0.69314718f, -0.69314718f)), hh);
  } else {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h.x) : "f"(-fabsf(v.x) * half_log2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h.y) : "f"(-fabsf(v.y) * half_log2e));
    hh = pair(h.x, h.y);
  }
  const f32x2 e = mul2(hh, hh);
  const float2 one = parts(add2(e, pair(1.f, 1.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(one.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(one.y));
  const float2 er = parts(mul2(e, pair(r.x, r.y)));
  return pair(v.x < 0.f ? er.x : r.x, v.y < 0.f ? er.y : r.y);
}

}  // namespace muon
