// Gated linear layer (moe_gated) and its gradient (moe_gated_backward): the first half of a
// gated feed-forward block, both projections, the activation and the product in one kernel:
//   z = [g, u] = x W^T + b   (W holds N gate rows, then N up rows),   h = act(g) u
//   dg = dh u act'(g),  du = dh act(g),  db = sum_m [dg, du],  dx = [dg, du] W,  dW = [dg, du]^T x
//
// The products are the linear layer's (linear.cu, linear_pair.cu, linear_few.cu) with a
// column operand whose tiles hold as many gate rows as up rows, so that a tile's epilogue
// has both of every h it writes: g and u never reach memory unless z is wanted.
//
// The gradient's [dg, du] takes one pass over dh and z (bound by memory) and is rounded to the
// operands' type for the two products, which are the linear layer's with 2 N columns.
#include "linear.cuh"

namespace moe {
namespace lin {
namespace {

// dz = [dh u act'(g), dh act(g)] in the operands' type, and per chunk of rows the fp32 sums of
// its unrounded columns.  Thread (x, y): eight columns of every 8th row of dh and the 2 x 8
// of z beside them, two rows' loads issued before the first is used.  VEC: rows that 16-byte
// accesses fit, columns 8 x .. 8 x + 7; otherwise columns x + 32 i, so that a warp's accesses
// are neighbours.
struct GatedDzArgs {
  int M, N, rows;  // rows per chunk
  int act;
  long long ld_dh, ld_dz;
  const void* dh;
  const void* z;
  void* dz;
  float* partials;  // [chunks][2 N], null: not wanted
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_columns(T (&v)[8], const T* q, int n) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      reinterpret_cast<uint4*>(v)[j] = __ldg(reinterpret_cast<const uint4*>(q) + j);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) v[i] = q[32 * i];
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_columns(T* to, const float (&v)[8], int n) {
  if (VEC) {
    alignas(16) T out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = as_type<T>(v[i]);
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(out);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) to[32 * i] = as_type<T>(v[i]);
  }
}

template <typename DT, typename T, bool VEC>
__global__ void __launch_bounds__(256) gated_dz_kernel(GatedDzArgs a) {
  __shared__ float s_sum[8][256 + 8];
  constexpr int AHEAD = 2;
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 256 + threadIdx.x * (VEC ? 8 : 1);  // first column
  const int n = a.N - c;                                         // columns from there on
  const int m0 = blockIdx.y * a.rows, m1 = min(a.M, m0 + a.rows);
  const long long ld_z = 2ll * a.N;
  float sum_g[8] = {}, sum_u[8] = {};
  if (n > 0) {
    for (int mb = m0 + threadIdx.y; mb < m1; mb += 8 * AHEAD) {
      alignas(16) DT d[AHEAD][8];
      alignas(16) T g[AHEAD][8], u[AHEAD][8];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const int m = mb + 8 * q;
        if (m < m1) {
          const T* z = static_cast<const T*>(a.z) + m * ld_z + c;
          load_columns<DT, VEC>(d[q], static_cast<const DT*>(a.dh) + m * a.ld_dh + c, n);
          load_columns<T, VEC>(g[q], z, n);
          load_columns<T, VEC>(u[q], z + a.N, n);
        }
      }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const int m = mb + 8 * q;
        if (m >= m1) break;
        float dg[8], du[8];
        auto gradient = [&](int act) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dg[i] = du[i] = 0.0f;
            if (VEC || 32 * i < n) {
              const float gv = as_float(g[q][i]), dv = as_float(d[q][i]);
              dg[i] = dv * as_float(u[q][i]) * act_grad(gv, act);
              du[i] = dv * act_value(gv, act);
            }
          }
        };
        switch (a.act) {
          case MOE_ACT_NONE: gradient(MOE_ACT_NONE); break;
          case MOE_ACT_RELU: gradient(MOE_ACT_RELU); break;
          case MOE_ACT_SILU: gradient(MOE_ACT_SILU); break;
          case MOE_ACT_GELU: gradient(MOE_ACT_GELU); break;
          default: gradient(MOE_ACT_GELU_TANH);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum_g[i] += dg[i];
          sum_u[i] += du[i];
        }
        if (a.dz) {
          T* to = static_cast<T*>(a.dz) + m * a.ld_dz + c;
          store_columns<T, VEC>(to, dg, n);
          store_columns<T, VEC>(to + a.N, du, n);
        }
      }
    }
  }
  if (!a.partials) return;
  const int col = threadIdx.y * 32 + threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s_sum[threadIdx.y][VEC ? threadIdx.x * 8 + i : threadIdx.x + 32 * i] = h ? sum_u[i] : sum_g[i];
    __syncthreads();
    if (blockIdx.x * 256 + col < a.N) {
      float v = 0.0f;
#pragma unroll
      for (int y = 0; y < 8; ++y) v += s_sum[y][col];
      a.partials[(static_cast<size_t>(blockIdx.y) * 2 + h) * a.N + blockIdx.x * 256 + col] = v;
    }
    __syncthreads();
  }
}

template <typename DT, typename T>
cudaError_t launch_dz(const GatedDzArgs& d, bool vec, int chunks, cudaStream_t s) {
  const dim3 grid((d.N + 255) / 256, chunks), block(32, 8);
  return vec ? launch_dependent(gated_dz_kernel<DT, T, true>, grid, block, 0, s, d)
             : launch_dependent(gated_dz_kernel<DT, T, false>, grid, block, 0, s, d);
}
template <typename T>
cudaError_t launch_dz(const GatedDzArgs& d, int dh_dtype, bool vec, int chunks, cudaStream_t s) {
  if (dh_dtype == MOE_DTYPE_F32) return launch_dz<float, T>(d, vec, chunks, s);
  if (dh_dtype == MOE_DTYPE_BF16) return launch_dz<__nv_bfloat16, T>(d, vec, chunks, s);
  return launch_dz<__half, T>(d, vec, chunks, s);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace lin

cudaError_t launch_gated(const GatedArgs& a, cudaStream_t s) {
  using namespace lin;
  Product q{};
  q.R = a.M;
  q.C = a.N;
  q.K = a.K;
  q.type = a.dtype == MOE_DTYPE_BF16 ? 1 : 0;
  q.gated = true;
  q.rows = {a.x, a.ld_x, a.K, a.M};
  q.cols = {a.w, a.ld_w, a.K, 2 * a.N};
  q.ep = {a.act, a.bias_dtype, a.out_dtype, a.dtype, 1.0f, a.ld_h, 2ll * a.N, a.bias, nullptr, a.h, a.z};
  q.reset_status = 1;
  q.hdr = a.hdr;
  stage_begin("gated", s);
  const cudaError_t err = takes_few(a) ? launch_few(a, s) : launch_product(q, s);
  stage_end(s);
  return err;
}

cudaError_t launch_gated_backward(const GatedBackwardArgs& a, cudaStream_t s) {
  using namespace lin;
  const bool products = a.dx || a.dw;
  // the first product clears the status word; without one nobody else does
  cudaError_t err = products ? cudaSuccess : launch_reset_header(a.hdr, s);
  if (err != cudaSuccess || (!products && !a.dbias)) return err;
  GatedDzArgs d{};
  d.M = a.M;
  d.N = a.N;
  d.rows = dz_rows(a.M);
  d.act = a.act;
  d.ld_dh = a.ld_h;
  d.ld_dz = dz_ld(2 * a.N);
  d.dh = a.dh;
  d.z = a.z;
  d.dz = products ? a.dz : nullptr;
  const int chunks = (a.M + d.rows - 1) / d.rows;
  d.partials = !a.dbias ? nullptr : chunks == 1 ? a.dbias : a.partials;
  const bool vec = a.N % 8 == 0 && a.ld_h % 8 == 0 && aligned16(a.dh) && aligned16(a.z);
  stage_begin("gated_dz", s);
  err = a.dtype == MOE_DTYPE_BF16 ? launch_dz<__nv_bfloat16>(d, a.dh_dtype, vec, chunks, s)
                                  : launch_dz<__half>(d, a.dh_dtype, vec, chunks, s);
  stage_end(s);
  if (err == cudaSuccess && a.dbias && chunks > 1) err = launch_column_sums(a.partials, chunks, 2 * a.N, a.dbias, s);
  if (err != cudaSuccess || !products) return err;
  const Operand dz{a.dz, d.ld_dz, 2 * a.N, a.M};
  return launch_gradient_products({a.M, 2 * a.N, a.K, a.dtype, a.ld_x, a.ld_w, a.x, a.w, a.dx, a.dw, dz, a.hdr}, s);
}

}  // namespace moe
