// The linear layer for up to eight rows, without tensor cores: y = alpha act(x W^T + b)
// + residual.
//
// A warp takes COLS columns n: its lanes read their rows of W side by side, 16 bytes
// each, and the same parts of every row of x, and add in fp32; a butterfly joins the lanes
// and the first ROWS x COLS of them finish one output each.  No barrier, no tensor memory, no
// shared memory: what is left of a call is the launch, one or a few trips to memory and five
// shuffles (1 x 128 x 2048: 2.0 us, 5.6 on the tensor cores).  Bound by reading W once,
// 1 x 8192 x 4096: 11.6 to 12.1 us, 5.5 to 5.8 TB/s; but each row of x costs two instructions per pair of
// products, so that more rows gain less and only where W is small.
#include "linear.cuh"

namespace moe {
namespace lin {
namespace {

constexpr int FEW_WARPS = 4;

__device__ __forceinline__ float2 pair_of(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <typename T, int ROWS, int COLS>
__global__ void __launch_bounds__(FEW_WARPS * 32) linear_few_kernel(LinearArgs a) {
  constexpr int AHEAD = ROWS < 8 && (COLS == 1 || ROWS == 1) ? 4 : 2;  // 16-byte parts of each row on their way
  dep_wait();
  dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = a.hdr->info = 0u;
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * FEW_WARPS + (threadIdx.x >> 5)) * COLS;
  if (n0 >= a.N) return;
  // columns past the last and rows past M stand in for the last
  const T* w[COLS];
  const T* x[ROWS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) w[c] = static_cast<const T*>(a.w) + static_cast<size_t>(min(n0 + c, a.N - 1)) * a.ld_w;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) x[r] = static_cast<const T*>(a.x) + static_cast<size_t>(min(r, a.M - 1)) * a.ld_x;
  float sum[ROWS][COLS] = {};
  for (int k0 = lane * 8; k0 < a.K; k0 += 256 * AHEAD) {
    uint4 wv[AHEAD][COLS], xv[AHEAD][ROWS];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int k = k0 + 256 * q;
      if (k < a.K) {  // takes_few: K is a multiple of 8
#pragma unroll
        for (int c = 0; c < COLS; ++c) wv[q][c] = __ldg(reinterpret_cast<const uint4*>(w[c] + k));
#pragma unroll
        for (int r = 0; r < ROWS; ++r) xv[q][r] = __ldg(reinterpret_cast<const uint4*>(x[r] + k));
      }
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (k0 + 256 * q >= a.K) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 xf[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) xf[r] = pair_of((&xv[q][r].x)[i], T());
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const float2 wf = pair_of((&wv[q][c].x)[i], T());
#pragma unroll
          for (int r = 0; r < ROWS; ++r) sum[r][c] = fmaf(xf[r].y, wf.y, fmaf(xf[r].x, wf.x, sum[r][c]));
        }
      }
    }
  }
  // lane r * COLS + c finishes output (r, n0 + c)
  float z = 0.0f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      float v = sum[r][c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == r * COLS + c) z = v;
    }
  const int r = lane / COLS, n = n0 + lane % COLS;
  if (lane >= ROWS * COLS || r >= a.M || n >= a.N) return;
  if (a.bias) z += load_as_f32(a.bias, a.bias_dtype, n);
  if (a.z) static_cast<T*>(a.z)[static_cast<size_t>(r) * a.N + n] = as_type<T>(z);
  float y = a.alpha * act_value(z, a.act);
  const size_t at = static_cast<size_t>(r) * a.ld_y + n;
  if (a.residual) y += load_as_f32(a.residual, a.out_dtype, at);
  if (a.out_dtype == MOE_DTYPE_F32) static_cast<float*>(a.y)[at] = y;
  else if (a.out_dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(y);
  else static_cast<__half*>(a.y)[at] = __float2half_rn(y);
}

template <typename T, int ROWS, int COLS>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  const int blocks = (a.N - 1) / (FEW_WARPS * COLS) + 1;
  return launch_dependent(linear_few_kernel<T, ROWS, COLS>, dim3(blocks), dim3(FEW_WARPS * 32), 0, s, a);
}
// Two columns per warp share what reading x costs where there are more columns than warps find a place.
template <typename T, int ROWS>
cudaError_t launch_cols(const LinearArgs& a, cudaStream_t s) {
  return a.N > 152 * 16 ? launch<T, ROWS, 2>(a, s) : launch<T, ROWS, 1>(a, s);
}
template <typename T>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t s) {
  return a.M == 1 ? launch_cols<T, 1>(a, s) : a.M == 2 ? launch_cols<T, 2>(a, s) : a.M <= 4 ? launch_cols<T, 4>(a, s) : launch<T, 8, 1>(a, s);
}

}  // namespace

// Measured in graphs, weights from memory where they pass L2 together (us, here / on the tensor
// cores), for N x K; the rule comes from some 1500 such shapes, N of 8 to 16384 and K of 32 to 8192:
//   1 row   128 x 2048  2.0 / 5.6;  4096 x 4096  7.9 / 10.4;  256 x 8192  7.3 / 8.4;  16384 x 64  3.8 / 3.3
//   2 rows  8192 x 4096  13.4 / 15.6;  3000 x 8192  14.9 / 13.7;  16384 x 128  3.6 / 3.8
//   4 rows  128 x 8192  7.8 / 8.0;  2048 x 4096  7.0 / 8.6;  4096 x 2048  7.2 / 8.2;  3000 x 4096  9.9 / 9.4
//           8192 x 256  3.5 / 4.0;  16384 x 64  5.0 / 3.3;  16384 x 512  6.7 / 5.8
//   8 rows  64 x 4096  5.0 / 6.4;  256 x 3000  4.4 / 6.5;  2048 x 2048  6.3 / 6.9;  4096 x 64  3.3 / 2.6
//           1024 x 4096  8.4 / 7.4;  256 x 8192  13.5 / 8.4
// With a long K a warp walks it alone, where the tensor cores' tiles split the sum; with many
// columns the rows of x are read again by every other one.
// Rows are read in whole parts of eight values, which may not reach into what lies between two
// rows or behind the last: other K go to the tensor cores, whose TMA boxes end at K.
bool takes_few(const LinearArgs& a) {
  if (a.K % 8 != 0) return false;
  const long long weights = static_cast<long long>(a.N) * a.K;
  if (a.M <= 2) return a.N < 1 << 14 || a.K > 128;
  if (a.M <= 4) return a.N <= 8192 && weights <= 1 << 23;
  return a.M <= 8 && a.N <= 152 * 16 && weights <= 1 << 22 && a.K <= (a.N <= 192 ? 4096 : 3000);
}

cudaError_t launch_few(const LinearArgs& a, cudaStream_t s) {
  return a.dtype == MOE_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(a, s) : launch_rows<__half>(a, s);
}

}  // namespace lin
}  // namespace moe
