// What the kernels of products with block scales share (linear_fp8.cu; linear_fp8_few.cu: a few rows).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace f8 {

// Scale of a group of h whose largest magnitude is `amax`, and the factor that codes take: the
// reciprocal where it is a normal number (a code can then differ from the quotient's where h
// lies within an fp32 rounding of a midpoint between codes, less than h's own error).
__device__ __forceinline__ float group_scale(float amax, float& inv) {
  const float s = amax / 448.0f;
  if (!(s > 0.0f)) {
    inv = 1.0f;
    return 1.0f;
  }
  inv = s >= 1.17549435e-38f ? 1.0f / s : 0.0f;
  return s;
}
// The code of h; inv == 0 next to the smallest scales (and for an infinite one).
__device__ __forceinline__ float scaled(float h, float s, float inv) { return inv > 0.0f ? h * inv : h / s; }

// Up to 16 rows (linear_fp8_few.cu).
bool takes_few(const Fp8Args& a);
cudaError_t launch_few(const Fp8Args& a, cudaStream_t s);

}  // namespace f8
}  // namespace moe
