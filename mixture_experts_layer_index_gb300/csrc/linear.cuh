// Parts shared by the kernels of the linear layer (linear.cu: any shape; linear_pair.cu:
// large ones; linear_few.cu: a few rows).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace lin {

constexpr int BK = 64;  // values of the sum per stage: 128 bytes

// Shared-memory descriptor of an operand in TMA boxes of 128-byte rows with the
// 128-byte swizzle, and how it moves along the sum.  K-major: as sw128_kmajor_desc, 16
// values of the sum are 32 bytes on.  MN-major: boxes of 64 values along MN x 64 along
// the sum; 8-row groups along the sum 1024 bytes apart (stride byte offset), the next
// 64 along MN one box = 8192 bytes on (leading byte offset); 16 values of the sum are
// 2048 bytes on.  Only the address field changes, and it never carries out of its bits.
struct OperandWalk {
  uint64_t fixed;
  uint32_t step;
  __device__ __forceinline__ explicit OperandWalk(bool mn)
      : fixed((static_cast<uint64_t>(mn ? 8192u >> 4 : 1u) << 16) | (static_cast<uint64_t>(1024u >> 4) << 32) |
              (1ull << 46) | (2ull << 61)),
        step((mn ? 2048u : 32u) >> 4) {}
  // kk-th run of 16 values of the stage at smem_addr
  __device__ __forceinline__ uint64_t at(uint32_t smem_addr, int kk) const {
    return fixed | (((smem_addr & 0x3FFFFu) >> 4) + kk * step);
  }
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// ------------------------------------------------------------------ activations
// An epilogue has about as many instructions per output value as the tensor cores leave
// time for, so the activations use the hardware's exponential and reciprocal
// (__expf, __fdividef: relative errors of a few 2^-23 over the range that matters) and,
// for erf, the rational approximation 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions: absolute error at most 1.5e-7.

// 1 / (1 + e^-z)
__device__ __forceinline__ float fast_sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// The upper tail of the normal distribution, (1 - erf(x / sqrt 2)) / 2 for x >= 0, and e = e^(-x^2 / 2).
__device__ __forceinline__ float normal_tail(float x, float& e) {
  const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678f, x, 1.0f));
  e = __expf(-0.5f * x * x);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  return 0.5f * p * t * e;
}
// 2 u of the tanh form: (1 + tanh u) / 2 = sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh_2u(float z) { return 1.59576912f * z * fmaf(0.044715f * z, z, 1.0f); }

// max(z, 0) that keeps a NaN, which fmaxf drops.
__device__ __forceinline__ float relu(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return relu(z);
    case MOE_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
    case MOE_ACT_GELU: {
      float e;
      const float tail = normal_tail(fabsf(z), e);
      return z * (z > 0.0f ? 1.0f - tail : tail);  // z - z tail would be infinity - NaN at z = infinity
    }
    case MOE_ACT_GELU_TANH: return z * fast_sigmoid(gelu_tanh_2u(z));
    default: return z;
  }
}
// All values of a thread at once: one branch for all of them.
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MOE_ACT_RELU);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MOE_ACT_SILU);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MOE_ACT_GELU);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MOE_ACT_GELU_TANH);
      break;
    default: break;
  }
}
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
      const float s = fast_sigmoid(z);
      return s * fmaf(z, 1.0f - s, 1.0f);
    }
    case MOE_ACT_GELU: {
      float e;
      const float tail = normal_tail(fabsf(z), e);
      return fmaf(0.39894228f * z, e, z > 0.0f ? 1.0f - tail : tail);
    }
    case MOE_ACT_GELU_TANH: {
      // s + s (1 - s) z 2u'(z), the vanishing factor first: z^2 alone passes fp32's range
      const float s = fast_sigmoid(gelu_tanh_2u(z)), d = z * (s * (1.0f - s));
      return fmaf(1.59576912f, fmaf(0.134145f * z, z * d, d), s);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float load_as_f32(const void* p, int dtype, size_t i) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T as_type(float v);
template <>
__device__ __forceinline__ float as_type<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 as_type<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half as_type<__half>(float v) { return __float2half_rn(v); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

struct Operand {
  const void* base;
  long long ld;
  int inner, outer;  // inner: contiguous extent
};

// The epilogue of a product: out = alpha act(sum + bias) + residual, z = sum + bias.
struct Epilogue {
  int act, bias_dtype, out_dtype, z_dtype;
  float alpha;
  long long ld_y, ld_z;
  const void* bias;
  const void* residual;
  void* y;
  void* z;
};

// A 16-bit matrix of `outer` rows of `inner` values, ld values apart, in boxes.
inline bool encode(CUtensorMap* map, const void* base, int type, uint64_t inner, uint64_t outer, long long ld,
            uint32_t box_inner, uint32_t box_outer) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, type ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out[r][c] = epilogue(sum_k rows[r][k] cols[c][k]); ROWS_MN / COLS_MN: the operand lies
// contiguous along r / c instead of along the sum.
struct Product {
  int R, C, K;
  int type;  // 0 = f16, 1 = bf16 operands
  Operand rows, cols;
  bool rows_mn, cols_mn;
  Epilogue ep;
  int reset_status;
  DeviceHeader* hdr;
};

// linear_pair.cu: about how long a launch takes (us); the product, or two of a gradient
// (the same type and row length, no bias, activation, residual or z).
float pair_estimate(const Product& p);
cudaError_t launch_pair(const Product& first, const Product* second, cudaStream_t s);
// A few rows (linear_few.cu).
bool takes_few(const LinearArgs& a);
cudaError_t launch_few(const LinearArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace moe
