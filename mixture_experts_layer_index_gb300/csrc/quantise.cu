// Quantisation in blocks of 128 (moe_quantise): s = amax / 448 over 128 columns of a row or over
// 128 x 128 values (1 where that is 0), q = e4m3(v / s), to nearest even.  One pass: a block's
// values stay in registers between its maximum and its codes.  Bound by memory and, for 16-bit rows, by
// instructions; threads walk over their blocks with the next values on their way while they work on the
// last.  16384 x 2048 bf16 rows 18.3 us (5.5 TB/s), fp32 rows 26 (6.4), 8192 x 4096 fp32 blocks 29.6 (5.7);
// rows of 2047 bf16 values, 2 bytes a load, 36.4 (2.8; blocks of such rows spill 150 bytes too).  Packed pairs of fp32 and two buffers used in turn
// were slower (28.9).
//
// Quotients are the correctly rounded ones, by Markstein's correction of the product with the
// reciprocal (P. Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990): q' = q + (v - q s) / s with the remainder exact in one fused operation, three
// instructions instead of a division.  All of it with the reciprocal's
// negative, which gives -q' and keeps the sign of a zero; the codes' sign bits are turned over at the
// end.  The reciprocal itself is a division, once per block; where the scale is so small or large
// that a remainder could leave the normal range, every quotient is.
#include "linear.cuh"

namespace moe {
namespace {

using lin::as_float;

struct Scale {
  float s, ninv;
  bool plain;  // quotients by division
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale r;
  r.plain = !(amax > 1e-20f && amax < 1e25f);
  const float q = amax * (1.0f / 448.0f);
  r.s = r.plain ? amax / 448.0f : fmaf(fmaf(-q, 448.0f, amax), 1.0f / 448.0f, q);
  if (!(r.s > 0.0f)) r.s = 1.0f;
  r.ninv = -__frcp_rn(r.s);
  return r;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Scale& c) {
  float q[8];  // negative quotients
  if (c.plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = -(v[i] / c.s);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float nq = v[i] * c.ninv;
      q[i] = fmaf(fmaf(nq, c.s, v[i]), c.ninv, nq);
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (static_cast<uint32_t>(cvt_e4m3x2(q[4 * i], q[4 * i + 1])) |
            static_cast<uint32_t>(cvt_e4m3x2(q[4 * i + 2], q[4 * i + 3])) << 16) ^ 0x80808080u;
  return make_uint2(w[0], w[1]);
}

// Eight values of a row from column k0 on for thread l of L that share the columns: VEC 8 l .. 8 l + 7,
// else l + L i; zeros past K.
template <typename T, bool VEC, int L>
__device__ __forceinline__ void load8(T (&v)[8], const T* row, int k0, int l, int K) {
  if (VEC) {
    const int k = k0 + 8 * l;
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      reinterpret_cast<uint4*>(v)[j] = k < K ? __ldg(reinterpret_cast<const uint4*>(row + k) + j) : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + l + L * i < K ? row[k0 + l + L * i] : T(0.0f);
  }
}
template <bool VEC, int L>
__device__ __forceinline__ void store8(uint8_t* row, int k0, int l, int K, uint2 w) {
  if (VEC) {
    if (k0 + 8 * l < K) *reinterpret_cast<uint2*>(row + k0 + 8 * l) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + l + L * i < K) row[k0 + l + L * i] = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}
// The largest magnitude, without a NaN's part.
__device__ __forceinline__ float amax8(const float (&v)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
template <typename T2, typename T>
__device__ __forceinline__ float amax8_pairs(const T (&v)[8], float m) {
  const T2* p = reinterpret_cast<const T2*>(v);
  const T2 a = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
  return fmaxf(m, fmaxf(as_float(a.x), as_float(a.y)));
}
__device__ __forceinline__ float amax8(const __nv_bfloat16 (&v)[8], float m) { return amax8_pairs<__nv_bfloat162>(v, m); }
__device__ __forceinline__ float amax8(const __half (&v)[8], float m) { return amax8_pairs<__half2>(v, m); }
template <bool VEC, int L, typename T>
__device__ __forceinline__ void put8(uint8_t* row, int k0, int l, int K, const T (&v)[8], const Scale& c) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = as_float(v[j]);
  store8<VEC, L>(row, k0, l, K, codes8(f, c));
}

// Groups of 8 threads take (row, 128 columns), 64 columns at a time; a block of 32 groups lies
// `across` groups wide and takes AHEAD of its heights at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantise_rows_kernel(QuantiseArgs a, int nk, int across) {
  constexpr int AHEAD = sizeof(T) == 4 ? 1 : 2;
  dep_wait();
  dep_launch();
  const int l = threadIdx.x & 7, group = threadIdx.x >> 3, high = 32 / across;
  const int kb = blockIdx.x * across + group % across, k0 = kb * 128;
  const T* x = static_cast<const T*>(a.x);
  alignas(16) T buffer[2][AHEAD][2][8];
  auto load = [&](T (&v)[AHEAD][2][8], long long m0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long long m = m0 + i * high + group / across;
      if (kb < nk && m < a.M) {
        load8<T, VEC, 8>(v[i][0], x + m * a.ld_x, k0, l, a.K);
        load8<T, VEC, 8>(v[i][1], x + m * a.ld_x, k0 + 64, l, a.K);
      }
    }
  };
  auto finish = [&](const T (&v)[AHEAD][2][8], long long m0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long long m = m0 + i * high + group / across;
      const bool in = kb < nk && m < a.M;
      float amax = in ? amax8(v[i][1], amax8(v[i][0], 0.0f)) : 0.0f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (!in) continue;
      const Scale c = scale_of(amax);
      uint8_t* q = a.q + m * a.ld_q;
      put8<VEC, 8>(q, k0, l, a.K, v[i][0], c);
      put8<VEC, 8>(q, k0 + 64, l, a.K, v[i][1], c);
      if (l == 0) a.scale[m * nk + kb] = c.s;
    }
  };
  const long long step = static_cast<long long>(gridDim.y) * high * AHEAD;
  long long m0 = static_cast<long long>(blockIdx.y) * high * AHEAD;
  load(buffer[0], m0);
  for (; m0 < a.M; m0 += step) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) buffer[1][i][j][e] = buffer[0][i][j][e];
    load(buffer[0], m0 + step);
    finish(buffer[1], m0);
  }
}

// A block of threads takes 128 x 128 values at a time: 16 threads across, every 32nd row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, 2) quantise_block_kernel(QuantiseArgs a, int nk, int blocks) {
  __shared__ float s_max[2][16];
  dep_wait();
  dep_launch();
  const int l = threadIdx.x & 15, r = threadIdx.x >> 4;
  const T* x = static_cast<const T*>(a.x);
  alignas(16) T buffer[2][4][8];
  auto load = [&](T (&v)[4][8], int b) {
    if (b >= blocks) return;
    const int kb = b % nk;
    const long long m0 = static_cast<long long>(b / nk) * 128 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + 32 * i < a.M) load8<T, VEC, 16>(v[i], x + (m0 + 32 * i) * a.ld_x, kb * 128, l, a.K);
  };
  auto finish = [&](const T (&v)[4][8], float* maxima, int b) {
    const int kb = b % nk;
    const long long m0 = static_cast<long long>(b / nk) * 128 + r;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + 32 * i < a.M) amax = amax8(v[i], amax);
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) maxima[threadIdx.x >> 5] = amax;
    __syncthreads();  // the other set of maxima is written next: one barrier per block of values
    amax = warp_max(maxima[threadIdx.x & 15]);
    const Scale c = scale_of(amax);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + 32 * i < a.M) put8<VEC, 16>(a.q + (m0 + 32 * i) * a.ld_q, kb * 128, l, a.K, v[i], c);
    if (threadIdx.x == 0) a.scale[b] = c.s;
  };
  // 16-bit values: the next on their way meanwhile; fp32: the registers go to a second block on the SM
  constexpr bool EARLY = sizeof(T) == 2;
  const int step = static_cast<int>(gridDim.x);
  load(buffer[0], blockIdx.x);
  int turn = 0;
  for (long long b = blockIdx.x; b < blocks; b += step) {
    const int next = static_cast<int>(min(b + step, static_cast<long long>(blocks)));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) buffer[1][i][e] = buffer[0][i][e];
    if (EARLY) load(buffer[0], next);
    finish(buffer[1], s_max[turn], static_cast<int>(b));
    if (!EARLY) load(buffer[0], next);
    turn ^= 1;
  }
}

template <typename T, bool VEC>
cudaError_t launch(const QuantiseArgs& a, cudaStream_t s) {
  const int nk = (a.K + 127) / 128, sms = num_sms();
  if (sms < 1) return cudaErrorNoDevice;
  if (a.block_rows == 128) {
    const int blocks = (a.M + 127) / 128 * nk, grid = sms * 2;
    return launch_dependent(quantise_block_kernel<T, VEC>, dim3(blocks < grid ? blocks : grid), dim3(512), 0, s, a, nk, blocks);
  }
  int across = 1;
  while (across < 32 && across < nk) across *= 2;
  const int wide = (nk + across - 1) / across, rows = 32 / across * (sizeof(T) == 4 ? 1 : 2);
  const int high = static_cast<int>((a.M + static_cast<long long>(rows) - 1) / rows), full = (sms * 4 + wide - 1) / wide;
  return launch_dependent(quantise_rows_kernel<T, VEC>, dim3(wide, high < full ? high : full < 65535 ? full : 65535), dim3(256), 0, s, a, nk, across);
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
