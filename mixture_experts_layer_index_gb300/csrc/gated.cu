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
// of z beside them, two rows' loads issued before the first is used.  W: values of an access that
// fit every row: 8 (16 bytes of 16-bit values; columns 8 x .. 8 x + 7), 2 (columns 2 x and 2 x + 1 of
// every 64) or 1 (columns x + 32 i), so that a warp's accesses are neighbours.  Bound by memory:
// 16384 x 4096 bf16 98 us, 6.8 TB/s.
struct GatedDzArgs {
  int M, N, rows;  // rows per chunk
  int act;
  long long ld_dh, ld_dz;
  const void* dh;
  const void* z;
  void* dz;
  float* partials;  // [chunks][2 N], null: not wanted
};

// Distance of a thread's i-th column from its first.
template <int W>
__device__ __forceinline__ int column(int i) {
  return W == 8 ? i : W == 2 ? 64 * (i / 2) + (i & 1) : 32 * i;
}
template <typename T>
struct alignas(2 * sizeof(T)) Two {
  T v[2];
};
template <typename T, int W>
__device__ __forceinline__ void load_columns(T (&v)[8], const T* q, int n) {
  if (W == 8) {
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      reinterpret_cast<uint4*>(v)[j] = __ldg(reinterpret_cast<const uint4*>(q) + j);
  } else if (W == 2) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      if (column<W>(i) < n) *reinterpret_cast<Two<T>*>(&v[i]) = *reinterpret_cast<const Two<T>*>(q + column<W>(i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (column<W>(i) < n) v[i] = q[column<W>(i)];
  }
}
template <typename T, int W>
__device__ __forceinline__ void store_columns(T* to, const float (&v)[8], int n) {
  alignas(16) T out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = as_type<T>(v[i]);
  if (W == 8) {
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(out);
  } else if (W == 2) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      if (column<W>(i) < n) *reinterpret_cast<Two<T>*>(to + column<W>(i)) = *reinterpret_cast<const Two<T>*>(&out[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (column<W>(i) < n) to[column<W>(i)] = out[i];
  }
}

template <typename DT, typename T, int W>
__global__ void __launch_bounds__(256) gated_dz_kernel(GatedDzArgs a) {
  __shared__ float s_sum[8][256 + 8];
  constexpr int AHEAD = 2;
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 256 + threadIdx.x * W;  // first column
  const int n = a.N - c;                             // columns from there on
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
          load_columns<DT, W>(d[q], static_cast<const DT*>(a.dh) + m * a.ld_dh + c, n);
          load_columns<T, W>(g[q], z, n);
          load_columns<T, W>(u[q], z + a.N, n);
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
            if (W == 8 || column<W>(i) < n) {
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
          store_columns<T, W>(to, dg, n);
          store_columns<T, W>(to + a.N, du, n);
        }
      }
    }
  }
  if (!a.partials) return;
  const int col = threadIdx.y * 32 + threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[threadIdx.y][threadIdx.x * W + column<W>(i)] = h ? sum_u[i] : sum_g[i];
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
cudaError_t launch_dz(const GatedDzArgs& d, int width, int chunks, cudaStream_t s) {
  const dim3 grid((d.N + 255) / 256, chunks), block(32, 8);
  return width == 8   ? launch_dependent(gated_dz_kernel<DT, T, 8>, grid, block, 0, s, d)
         : width == 2 ? launch_dependent(gated_dz_kernel<DT, T, 2>, grid, block, 0, s, d)
                      : launch_dependent(gated_dz_kernel<DT, T, 1>, grid, block, 0, s, d);
}
template <typename T>
cudaError_t launch_dz(const GatedDzArgs& d, int dh_dtype, int width, int chunks, cudaStream_t s) {
  if (dh_dtype == MOE_DTYPE_F32) return launch_dz<float, T>(d, width, chunks, s);
  if (dh_dtype == MOE_DTYPE_BF16) return launch_dz<__nv_bfloat16, T>(d, width, chunks, s);
  return launch_dz<__half, T>(d, width, chunks, s);
}

// Whether accesses of `width` values fit every row.
bool fits_rows(const GatedBackwardArgs& a, int width) {
  const size_t es = a.dh_dtype == MOE_DTYPE_F32 ? 4 : 2;
  return a.N % width == 0 && a.ld_h % width == 0 && reinterpret_cast<uintptr_t>(a.dh) % (width == 8 ? 16 : width * es) == 0 &&
         reinterpret_cast<uintptr_t>(a.z) % (2 * width) == 0;
}
// Rows of a chunk: few enough that small problems fill the GPU too, in at most 256 chunks.
int chunk_rows(int M, int N) {
  const long long across = (N + 255) / 256;
  int rows = dz_rows(M);
  while (rows > 16 && (M + rows - 1) / rows * across < 304 && (M + rows / 2 - 1) / (rows / 2) <= 256) rows /= 2;
  return M <= rows ? M : rows;
}

}  // namespace
}  // namespace lin

size_t gated_partials_bytes(int M, int N) {
  const int rows = lin::chunk_rows(M, N);
  return rows ? static_cast<size_t>((M + rows - 1) / rows) * 2 * N * sizeof(float) : 0;
}

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
  d.rows = chunk_rows(a.M, a.N);
  d.act = a.act;
  d.ld_dh = a.ld_h;
  d.ld_dz = dz_ld(2 * a.N);
  d.dh = a.dh;
  d.z = a.z;
  d.dz = products ? a.dz : nullptr;
  const int chunks = (a.M + d.rows - 1) / d.rows;
  d.partials = !a.dbias ? nullptr : chunks == 1 ? a.dbias : a.partials;
  const int width = fits_rows(a, 8) ? 8 : fits_rows(a, 2) ? 2 : 1;
  stage_begin("gated_dz", s);
  err = a.dtype == MOE_DTYPE_BF16 ? launch_dz<__nv_bfloat16>(d, a.dh_dtype, width, chunks, s)
                                  : launch_dz<__half>(d, a.dh_dtype, width, chunks, s);
  stage_end(s);
  if (err == cudaSuccess && a.dbias && chunks > 1) err = launch_column_sums(a.partials, chunks, 2 * a.N, a.dbias, s);
  if (err != cudaSuccess || !products) return err;
  const Operand dz{a.dz, d.ld_dz, 2 * a.N, a.M};
  return launch_gradient_products({a.M, 2 * a.N, a.K, a.dtype, a.ld_x, a.ld_w, a.x, a.w, a.dx, a.dw, dz, true, a.hdr}, s);
}

}  // namespace moe
