// Parts shared by the two kernels of the linear layer (linear.cu: any shape;
// linear_pair.cu: large ones).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace lin {

constexpr int BK = 64;  // values of the sum per stage: 128 bytes

// Descriptor of an MN-major operand in the layout of TMA boxes of 64 values along MN
// (128 bytes, 128-byte swizzle) x 64 along the sum: 8-row groups along the sum 1024
// bytes apart (stride byte offset), the next 64 along MN one box = 8192 bytes on
// (leading byte offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

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
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return fmaxf(z, 0.0f);
    case MOE_ACT_SILU: return z / (1.0f + expf(-z));
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case MOE_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU: return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
    case MOE_ACT_GELU_TANH: {
      const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
      return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * 0.79788456f * (1.0f + 0.134145f * z * z);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float load_as_f32(const void* p, int dtype, size_t i) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

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

// Whether launch_pair takes the product: outputs that TMA can store, enough work.
bool pair_takes(const Product& p);
cudaError_t launch_pair(const Product& p, cudaStream_t s);

}  // namespace lin
}  // namespace moe
