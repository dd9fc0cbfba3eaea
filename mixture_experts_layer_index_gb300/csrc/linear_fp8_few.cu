// Products of e4m3 operands with block scales for up to 16 rows of x (8 gated): bound by reading w once.
//
// A block takes 16 output columns, eight warps each the groups of 128 of the sum in turn.  All of
// the block's weights are asked for at once, as prefetches into L2 (which may begin before the kernel
// before this one has ended: nothing is read), then come to registers, 16 bytes a lane and row, 64
// consecutive bytes of a row at a time.  mma.sync.m16n8k32 multiplies 16 weight rows (M) with 8 rows
// of x (N); the order of a group's 128 values is permuted, alike on both sides, so that a lane's
// 16 bytes are its fragments.  (The tensor cores' tcgen05 form wants 128 rows and a trip through
// shared memory: 8 x 4096 x 4096 8.8 us in linear_fp8.cu, here 5.1.)  Each group's partial is multiplied by
// its scales and added in fp32; the warps' sums meet in shared memory in a fixed order.
// GATED: the block's 16 columns are two tiles of 8 gate and 8 up rows each, with eight warps per
// tile; a thread's sums hold both of its values of h; with e4m3 output the eight blocks of a group
// of 128 columns are a cluster and share their rows' maxima.
#include "linear_pair.cuh"
#include "linear_fp8.cuh"

namespace moe {
namespace f8 {
namespace {

using namespace lin;

constexpr int WARPS = 8;  // per tile of 16 weight rows

// Codes k .. k + 15 of a row; zeros past K, where nothing is read.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int k, int K) {
  const int rest = K - k;
  if (rest >= 16) return __ldg(reinterpret_cast<const uint4*>(row + k));
  if (rest <= 0) return make_uint4(0, 0, 0, 0);
  // whole words, then the bytes of the last one: all loads at once
  const int words = rest >> 2;
  uint32_t w[4], last = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) w[i] = i < words ? __ldg(reinterpret_cast<const uint32_t*>(row + k) + i) : 0u;
  w[3] = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (4 * words + i < rest) last |= static_cast<uint32_t>(__ldg(row + k + 4 * words + i)) << (8 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i == words) w[i] = last;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void mma_m16n8k32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// XT: tiles of 8 rows of x.
template <int XT, bool GATED>
__global__ void __launch_bounds__(WARPS * 32 * (GATED ? 2 : 1), 2) fp8_few_kernel(Fp8Args a) {
  constexpr int WT = GATED ? 2 : 1;  // tiles of 16 weight rows
  constexpr int AHEAD = GATED || XT > 1 ? 1 : 2;  // groups on their way to registers
  __shared__ float sums[WARPS][WT][16][XT * 8];
  __shared__ float s_max[XT * 8][16], s_block[XT * 8];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warp = threadIdx.x / 32 % WARPS, tile = threadIdx.x / 32 / WARPS;
  const int n0 = blockIdx.x * 16;
  const int nk = (a.K + 127) / 128;
  // weight rows g and g + 8 of the warp's tile: two of a linear layer's, or a gate and its up row;
  // columns past the last and rows past M stand in for the last
  const uint8_t* w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = min(GATED ? n0 + 8 * tile + g : n0 + 8 * h + g, a.N - 1);
    w[h] = static_cast<const uint8_t*>(a.w) + (n + (GATED && h ? static_cast<size_t>(a.N) : 0)) * a.ld_w;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (int kb = warp + WARPS * t; kb < nk; kb += WARPS * 4) prefetch_l2(w[h] + kb * 128);
  dep_wait();
  dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->status = a.hdr->info = 0u;
  const uint8_t* x[XT];
  int sx[XT][2];  // scales of rows 2 t and 2 t + 1
#pragma unroll
  for (int i = 0; i < XT; ++i) {
    x[i] = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(min(8 * i + g, a.M - 1)) * a.ld_x;
#pragma unroll
    for (int j = 0; j < 2; ++j) sx[i][j] = min(8 * i + 2 * t + j, a.M - 1) * nk;
  }
  const int blocks = (a.N + 127) / 128, block = min(n0 / 128, blocks - 1);
  const float* sw = a.w_scale + static_cast<size_t>(block) * nk;
  const float* su = sw + static_cast<size_t>(GATED ? blocks : 0) * nk;

  float acc[XT][4] = {};
  for (int kb0 = warp; kb0 < nk; kb0 += WARPS * AHEAD) {
    uint4 wv[AHEAD][2][2], xv[AHEAD][XT][2];
    float fx[AHEAD][XT][2], fw[AHEAD], fu[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int kb = kb0 + WARPS * q;
      if (kb < nk) {
        const int k = kb * 128 + 16 * t;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) wv[q][h][j] = load16(w[h], k + 64 * j, a.K);
#pragma unroll
          for (int i = 0; i < XT; ++i) xv[q][i][j] = load16(x[i], k + 64 * j, a.K);
        }
        fw[q] = __ldg(sw + kb);
        fu[q] = GATED ? __ldg(su + kb) : fw[q];
#pragma unroll
        for (int i = 0; i < XT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) fx[q][i][j] = __ldg(a.x_scale + sx[i][j] + kb);
      }
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (kb0 + WARPS * q >= nk) break;
#pragma unroll
      for (int i = 0; i < XT; ++i) {
        float d[4] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 lo = wv[q][0][j], hi = wv[q][1][j], b = xv[q][i][j];
          mma_m16n8k32(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
          mma_m16n8k32(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
        }
        // rows g and g + 8 of the weights, columns 2 t and 2 t + 1 of x
        acc[i][0] = fmaf(d[0], fw[q] * fx[q][i][0], acc[i][0]);
        acc[i][1] = fmaf(d[1], fw[q] * fx[q][i][1], acc[i][1]);
        acc[i][2] = fmaf(d[2], fu[q] * fx[q][i][0], acc[i][2]);
        acc[i][3] = fmaf(d[3], fu[q] * fx[q][i][1], acc[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < XT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[warp][tile][g + 8 * (r >> 1)][8 * i + 2 * t + (r & 1)] = acc[i][r];
  __syncthreads();

  // thread: column n of row m (16 columns of a row side by side)
  const int c = threadIdx.x & 15, m = threadIdx.x >> 4, n = n0 + c;
  const bool has = m < XT * 8, in = has && m < a.M && n < a.N;
  float v = 0.0f;
  if (has) {
    auto total = [&](int i, int r) {
      float z = 0.0f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) z += sums[k][i][r][m];
      return z;
    };
    if constexpr (GATED) {
      float gate = total(c >> 3, c & 7), up = total(c >> 3, (c & 7) + 8);
      if (a.bias && in) {
        gate += load_as_f32(a.bias, a.bias_dtype, n);
        up += load_as_f32(a.bias, a.bias_dtype, static_cast<size_t>(a.N) + n);
      }
      v = act_value(gate, a.act) * up;
    } else {
      v = total(0, c);
      if (a.bias && in) v += load_as_f32(a.bias, a.bias_dtype, n);
      v = a.alpha * act_value(v, a.act);
    }
  }
  const size_t at = static_cast<size_t>(m) * a.ld_y + n;
  if (GATED && a.h_scale) {
    if (has) s_max[m][c] = in ? fabsf(v) : 0.0f;
    __syncthreads();
    if (threadIdx.x < XT * 8) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s_max[threadIdx.x][i]);
      s_block[threadIdx.x] = top;
    }
    cluster_sync_all();
    if (has) {
      float top = 0.0f;
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r) {
        float o;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(map_rank(smem_u32(&s_block[m]), r)) : "memory");
        top = fmaxf(top, o);
      }
      const GroupScale g8(top);
      if (in) static_cast<uint8_t*>(a.y)[at] = static_cast<uint8_t>(cvt_e4m3x2(g8.negative(v * g8.lift), 0.0f) ^ 0x80u);
      if (c == 0 && m < a.M && (n0 & 127) == 0) a.h_scale[static_cast<size_t>(m) * blocks + n0 / 128] = g8.s;
    }
    cluster_sync_all();  // no block leaves while another still reads its maxima
    return;
  }
  if (!in) return;
  if (!GATED && a.residual) v += load_as_f32(a.residual, a.out_dtype, at);
  if (a.out_dtype == MOE_DTYPE_F32) static_cast<float*>(a.y)[at] = v;
  else if (a.out_dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.y)[at] = __float2half_rn(v);
}

template <int XT, bool GATED>
cudaError_t launch(const Fp8Args& a, cudaStream_t s) {
  // with e4m3 output a cluster covers a whole group of 128 columns
  const bool cluster = GATED && a.h_scale;
  const unsigned grid = cluster ? static_cast<unsigned>((a.N + 127) / 128) * 8 : static_cast<unsigned>((a.N + 15) / 16);
  cudaLaunchAttribute la[2];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  la[1].id = cudaLaunchAttributeClusterDimension;
  la[1].val.clusterDim.x = 8;
  la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(WARPS * 32 * (GATED ? 2 : 1));
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp8_few_kernel<XT, GATED>, a);
}

}  // namespace

// Measured in graphs, weights from memory (us, here / in linear_fp8.cu, whose time depends on where the operands
// lie, 8 x 8192 x 8192 20.2 to 26.2: means over six places), for M x N x K; the rules come from some 150 of these:
//   8 x 2048 x 768  1.8 / 5.2;  8 x 4096 x 4096  5.1 / 8.8;  8 x 8192 x 8192  19.0 / 21.6;  8 x 16384 x 8192  32.7 / 30.3
//   8 x 4096 x 12288  13.4 / 16.7;  8 x 8192 x 12288  27.1 / 23.9;  8 x 7168 x 18432  37.1 / 28.0
//   16 x 4096 x 4096  6.5 / 8.7;  16 x 14336 x 4096  19.1 / 20.1;  16 x 16384 x 4096  22.4 / 21.4;
//   16 x 8192 x 8192  22.8 / 16.8;  16 x 2048 x 8192  9.8 / 9.3;  12 x 4096 x 8192  11.2 / 12.8
//   gated to bf16, 8 rows   2048 x 768  2.4 / 6.3;  4096 x 4096  8.0 / 13.2;  14336 x 4096  26.9 / 30.9;
//   8192 x 8192  30.5 / 29.9;  8192 x 12288  45.6 / 41.4;  2048 x 18432  25.6 / 17.9
//   gated to e4m3, 8 rows   2048 x 768  3.8 / 7.1;  4096 x 4096  9.9 / 11.8;  4096 x 8192  16.4 / 17.7;
//   6144 x 4096  17.5 / 17.4 (1 row 16.8 / 18.4);  8192 x 4096  20.3 / 18.4;  2048 x 12288  19.4 / 17.5
//   gated, 16 rows (in a trial)  4096 x 4096 to bf16  14.6 / 13.4
// A warp walks its groups of the sum alone, where the tensor cores' tiles split it; with e4m3 output the
// clusters of a wide h come in waves.
bool takes_few(const Fp8Args& a) {
  const long long weights = static_cast<long long>(a.N) * a.K;
  if (a.gated) return a.M <= 8 && a.K <= 8192 && (!a.h_scale || a.N <= 6144);
  if (a.M <= 8) return a.K <= 8192 || weights <= 1 << 26;
  return a.M <= 16 && a.K <= 4096 && weights < 1 << 26;
}

cudaError_t launch_few(const Fp8Args& a, cudaStream_t s) {
  if (a.gated) return launch<1, true>(a, s);
  return a.M <= 8 ? launch<1, false>(a, s) : launch<2, false>(a, s);
}

}  // namespace f8
}  // namespace moe
