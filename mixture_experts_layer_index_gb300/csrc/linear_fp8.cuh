// What the kernels of products with block scales share (linear_fp8.cu; linear_fp8_few.cu: a few rows).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace f8 {

// Scale s of a group of h from its largest magnitude and the codes' arguments, which are the quantiser's
// (quantise.cu): the correctly rounded quotients h / s, by Markstein's correction of the product with the
// reciprocal's negative, which gives -h / s with a zero's sign; the codes' sign bits are turned over at the end.
// Group and scale are lifted by a power of two where the scale has no normal reciprocal or a remainder could
// leave the normal range, which changes no quotient; most groups are not (lift is 1).  An infinite scale leaves
// zeros and NaN.
struct GroupScale {
  float s, lift, lifted, ninv;
  __device__ __forceinline__ explicit GroupScale(float amax) {
    s = amax / 448.0f;
    if (!(s > 0.0f)) s = 1.0f;
    lift = amax >= 1e25f ? 0x1p-64f : amax > 0.0f && amax <= 1e-20f ? 0x1p100f : 1.0f;
    lifted = s * lift;
    ninv = -1.0f / lifted;
    if (amax == __int_as_float(0x7f800000)) lifted = 0.0f;  // no remainder: infinity times 0
  }
  // -h / s for h times lift
  __device__ __forceinline__ float negative(float h) const {
    const float q = h * ninv;
    return fmaf(fmaf(q, lifted, h), ninv, q);
  }
};
__device__ __forceinline__ uint32_t codes4(const float* h, const GroupScale& g) {
  return (static_cast<uint32_t>(cvt_e4m3x2(g.negative(h[0]), g.negative(h[1]))) |
          static_cast<uint32_t>(cvt_e4m3x2(g.negative(h[2]), g.negative(h[3]))) << 16) ^ 0x80808080u;
}

// Up to 16 rows, 8 gated (linear_fp8_few.cu).
bool takes_few(const Fp8Args& a);
cudaError_t launch_few(const Fp8Args& a, cudaStream_t s);

}  // namespace f8
}  // namespace moe
