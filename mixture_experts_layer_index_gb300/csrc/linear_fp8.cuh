// What the kernels of products with block scales share (linear_fp8.cu; linear_fp8_few.cu: a few rows).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace f8 {

// Scale s of a group of h from its largest magnitude, and what makes a code's argument of h: (h lift)
// inv, inv = 1 / (s lift).  lift keeps the reciprocal of the smallest scales finite; it is a power of two,
// so that the argument differs from the quotient h / s by at most an fp32 rounding (and a code where h
// lies that near a midpoint between codes, less than h's own error).  An infinite scale gives 0 and NaN.
struct GroupScale {
  float s, lift, inv;
  __device__ __forceinline__ explicit GroupScale(float amax) {
    s = amax / 448.0f;
    if (!(s > 0.0f)) s = 1.0f;
    lift = s < 1e-30f ? 18446744073709551616.0f : 1.0f;
    inv = 1.0f / (s * lift);
  }
  __device__ __forceinline__ float scaled(float h) const { return h * lift * inv; }
};

// Up to 16 rows, 8 gated (linear_fp8_few.cu).
bool takes_few(const Fp8Args& a);
cudaError_t launch_few(const Fp8Args& a, cudaStream_t s);

}  // namespace f8
}  // namespace moe
