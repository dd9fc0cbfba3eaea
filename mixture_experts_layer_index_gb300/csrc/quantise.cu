// Quantisation in blocks of 128 (moe_quantise): s = amax / 448 over 128 columns of a row or over
// 128 x 128 values (1 where that is 0), q = e4m3(v / s), to nearest even.  One pass: a block's
// values stay in registers between its maximum and its codes.  Bound by memory.
//
// The quotient is the correctly rounded one, by Markstein's correction of the product with the
// reciprocal (P. Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990): q' = q + (v - q s) / s with the remainder exact in one fused operation, four
// instructions instead of a division.  The reciprocal itself is a division, once per block; where
// the scale is so small or large that a remainder could leave the normal range, every quotient is.
#include "linear.cuh"

namespace moe {
namespace {

using lin::as_float;

struct Scale {
  float s, inv;
  bool plain;  // quotients by division
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale r;
  r.s = amax / 448.0f;
  if (!(r.s > 0.0f)) r.s = 1.0f;
  r.plain = !(r.s > 1e-25f && r.s < 1e25f);
  r.inv = 1.0f / r.s;
  return r;
}
__device__ __forceinline__ float quotient(float v, const Scale& c) {
  if (c.plain) return v / c.s;
  const float q = v * c.inv;
  return copysignf(fmaf(fmaf(-q, c.s, v), c.inv, q), v);  // of a negative zero the remainder is a positive one
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Scale& c) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(cvt_e4m3x2(quotient(v[4 * i], c), quotient(v[4 * i + 1], c))) |
           static_cast<uint32_t>(cvt_e4m3x2(quotient(v[4 * i + 2], c), quotient(v[4 * i + 3], c))) << 16;
  return make_uint2(w[0], w[1]);
}

// This thread's eight values of a group of 128 columns from k0: VEC 8 l .. 8 l + 7, else l + 16 i
// (l = its place among 16 threads), zeros past K.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(T (&v)[8], const T* row, int k0, int l, int K) {
  if (VEC) {
    const int k = k0 + 8 * l;
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      reinterpret_cast<uint4*>(v)[j] = k < K ? __ldg(reinterpret_cast<const uint4*>(row + k) + j) : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + l + 16 * i < K ? row[k0 + l + 16 * i] : T(0.0f);
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* row, int k0, int l, int K, uint2 w) {
  if (VEC) {
    if (k0 + 8 * l < K) *reinterpret_cast<uint2*>(row + k0 + 8 * l) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + l + 16 * i < K) row[k0 + l + 16 * i] = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}
template <typename T>
__device__ __forceinline__ float amax8(const T (&v)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(as_float(v[i])));  // without a NaN's part
  return m;
}

// Groups of 16 threads take (row, 128 columns); a block of 16 groups lies `across` groups wide
// and takes AHEAD of its heights, all of them loaded before the first is used.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantise_rows_kernel(QuantiseArgs a, int nk, int across) {
  constexpr int AHEAD = sizeof(T) == 4 ? 2 : 4;
  dep_wait();
  dep_launch();
  const int l = threadIdx.x & 15, group = threadIdx.x >> 4, high = 16 / across;
  const int kb = blockIdx.x * across + group % across;
  const T* x = static_cast<const T*>(a.x);
  for (long long m0 = static_cast<long long>(blockIdx.y) * high * AHEAD; m0 < a.M; m0 += static_cast<long long>(gridDim.y) * high * AHEAD) {
    alignas(16) T v[AHEAD][8];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long long m = m0 + i * high + group / across;
      if (kb < nk && m < a.M) load8<T, VEC>(v[i], x + m * a.ld_x, kb * 128, l, a.K);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long long m = m0 + i * high + group / across;
      const bool in = kb < nk && m < a.M;
      float amax = in ? amax8(v[i], 0.0f) : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (!in) continue;
      const Scale c = scale_of(amax);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = as_float(v[i][j]);
      store8<VEC>(a.q + m * a.ld_q, kb * 128, l, a.K, codes8(f, c));
      if (l == 0) a.scale[m * nk + kb] = c.s;
    }
  }
}

// A block of threads takes 128 x 128 values: 16 threads across, every 16th row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantise_block_kernel(QuantiseArgs a, int nk) {
  __shared__ float s_max[8];
  dep_wait();
  dep_launch();
  const int l = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int kb = blockIdx.x % nk;
  const long long m0 = static_cast<long long>(blockIdx.x / nk) * 128 + r;
  const T* x = static_cast<const T*>(a.x);
  alignas(16) T v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (m0 + 16 * i < a.M) load8<T, VEC>(v[i], x + (m0 + 16 * i) * a.ld_x, kb * 128, l, a.K);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (m0 + 16 * i < a.M) amax = amax8(v[i], amax);
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, s_max[i]);
  const Scale c = scale_of(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (m0 + 16 * i >= a.M) break;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = as_float(v[i][j]);
    store8<VEC>(a.q + (m0 + 16 * i) * a.ld_q, kb * 128, l, a.K, codes8(f, c));
  }
  if (threadIdx.x == 0) a.scale[blockIdx.x] = c.s;
}

template <typename T, bool VEC>
cudaError_t launch(const QuantiseArgs& a, cudaStream_t s) {
  const int nk = (a.K + 127) / 128;
  if (a.block_rows == 128)
    return launch_dependent(quantise_block_kernel<T, VEC>, dim3(static_cast<unsigned>((a.M + 127) / 128) * nk), dim3(256), 0, s, a, nk);
  int across = 1;
  while (across < 16 && across < nk) across *= 2;
  const int rows = 16 / across * (sizeof(T) == 4 ? 2 : 4);
  const long long high = (a.M + static_cast<long long>(rows) - 1) / rows;
  const dim3 grid((nk + across - 1) / across, static_cast<unsigned>(high < 65535 ? high : 65535));
  return launch_dependent(quantise_rows_kernel<T, VEC>, grid, dim3(256), 0, s, a, nk, across);
}
template <typename T>
cudaError_t launch(const QuantiseArgs& a, cudaStream_t s) {
  const bool vec = a.K % 8 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ld_x * sizeof(T) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && a.ld_q % 8 == 0;
  return vec ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

cudaError_t launch_quantise(const QuantiseArgs& a, cudaStream_t s) {
  stage_begin("quantise", s);
  const cudaError_t err = a.dtype == MOE_DTYPE_F32    ? launch<float>(a, s)
                          : a.dtype == MOE_DTYPE_BF16 ? launch<__nv_bfloat16>(a, s)
                                                      : launch<__half>(a, s);
  stage_end(s);
  return err;
}

}  // namespace moe
