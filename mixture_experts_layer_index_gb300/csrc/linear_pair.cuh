// What the kernels that work in pairs of SMs share (linear_pair.cu, linear_fp8.cu): the two-SM
// forms of loads, MMAs and barriers, and epilogue warps' boxes of 32 rows on their way to memory.
#pragma once

#include "linear.cuh"

namespace moe {
namespace lin {

constexpr int BOX_BYTES = 32 * 128;  // 32 rows of 128 bytes

// Barriers of the four epilogue warps that share 32 lanes (quadrant q).  They have no time limit, so all
// four come to one or none: quad_all, met once per tile by each of them whatever its waits said, gives
// all the same answer.
__device__ __forceinline__ void quad_barrier(int q) { asm volatile("bar.sync %0, 128;" ::"r"(2 + q) : "memory"); }
__device__ __forceinline__ bool quad_all(int q, bool good) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, r;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred r, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(good)), "r"(2 + q)
      : "memory");
  return all != 0;
}

// ------------------------------------------------------------------ two-SM forms
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// A load into this block's shared memory that counts on a barrier of the pair's even block.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both blocks once the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// The same after reads of tensor memory that are complete (in registers, behind tc_fence_before): nothing
// else of this thread has to be seen first.  The release above waits for every load and store of the
// thread that is on its way, too much for a loop.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t remote) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// 16 values (columns c.. of one row) into row `lane` of a swizzled box: 16-byte chunk j of a
// row sits at chunk j ^ (lane & 7).  `part`: which 16 of the box's columns.
__device__ __forceinline__ void put_box(uint8_t* box, int lane, int part, int dtype, const float (&v)[16]) {
  uint8_t* row = box + lane * 128;
  if (dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(row + (((part * 4 + j) ^ (lane & 7)) << 4)) =
          make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
      if (dtype == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 b = __floats2half2_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      *reinterpret_cast<uint4*>(row + (((part * 2 + j) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Columns c.. c + 31 of a box of fp32 values (32 rows from r0) to an array whose rows TMA
// cannot store: a row at a time, one lane per column, plus the residual's values.  Not
// inlined: its registers would be spilled from the paths that TMA stores.
template <typename T>
__device__ __forceinline__ void flush_box_as(const uint8_t* box, int lane, T* out, long long ld, const T* residual,
                                             int r0, int R, int c, int C) {
  const int rows = c + lane < C ? min(32, R - r0) : 0;
  const size_t at = static_cast<size_t>(r0) * ld + c + lane;
  out += at;
  if (residual) residual += at;
#pragma unroll 1
  for (int r = 0; r < rows; r += 16) {
    T u[16] = {};
    if (residual) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (r + i < rows) u[i] = residual[i * ld];
      residual += 16 * ld;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (r + i < rows) {
        float v = *reinterpret_cast<const float*>(box + (r + i) * 128 + (((lane >> 2) ^ ((r + i) & 7)) << 4) + (lane & 3) * 4);
        if (residual) v += as_float(u[i]);
        out[i * ld] = as_type<T>(v);
      }
    out += 16 * ld;
  }
  __syncwarp();  // the box may be written again
}
static __device__ __noinline__ void flush_box(const uint8_t* box, int lane, void* out, int dtype, long long ld,
                                          const void* residual, int r0, int R, int c, int C) {
  if (dtype == MOE_DTYPE_F32)
    flush_box_as(box, lane, static_cast<float*>(out), ld, static_cast<const float*>(residual), r0, R, c, C);
  else if (dtype == MOE_DTYPE_BF16)
    flush_box_as(box, lane, static_cast<__nv_bfloat16*>(out), ld, static_cast<const __nv_bfloat16*>(residual), r0, R, c, C);
  else
    flush_box_as(box, lane, static_cast<__half*>(out), ld, static_cast<const __half*>(residual), r0, R, c, C);
}

// v[i] += p[at + i], 16 values of which `n` exist; `wide`: p + at is 16-byte aligned.
__device__ __forceinline__ void add16(float (&v)[16], const void* p, int dtype, size_t at, int n, bool wide) {
  if (n < 16 || !wide) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i] += load_as_f32(p, dtype, at + i);
  } else if (dtype == MOE_DTYPE_F32) {
    float4 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[4 * j] += f[j].x; v[4 * j + 1] += f[j].y; v[4 * j + 2] += f[j].z; v[4 * j + 3] += f[j].w;
    }
  } else {
    uint4 raw[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) raw[j] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at)[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = dtype == MOE_DTYPE_BF16
                             ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]))
                             : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[8 * j + 2 * i] += f.x;
        v[8 * j + 2 * i + 1] += f.y;
      }
    }
  }
}

// 16 values into row `lane` of a box of 32 rows of 64 bytes (16-bit values; the 64-byte swizzle
// has chunk j of a row at chunk j ^ (row / 2 & 3)).  `part`: which 16 of the box's 32 columns.
__device__ __forceinline__ void put_half_box(uint8_t* box, int lane, int part, int dtype, const float* v) {
  uint8_t* row = box + lane * 64;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t w[4];
    if (dtype == MOE_DTYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    *reinterpret_cast<uint4*>(row + (((part * 2 + j) ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A store map: boxes of 32 rows of 128 bytes, or of 64.
inline bool encode_store(CUtensorMap* map, void* base, int dtype, int cols, int rows, long long ld, uint32_t row_bytes = 128) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const uint32_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  const cuuint32_t box[2] = {row_bytes / es, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = dtype == MOE_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, type, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA can store `cols` values per row: rows at 16-byte boundaries that end at one, because
// what TMA clips at a row's end it clips in whole 16 bytes.
inline bool storable(const void* base, int dtype, int cols, long long ld) {
  const int es = dtype == MOE_DTYPE_F32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld * es % 16 == 0 && static_cast<long long>(cols) * es % 16 == 0;
}

}  // namespace lin
}  // namespace moe
