// The norms at the two ends of a block, fused with the block's gate and the
// residual sum (moe_norm_forward), and their gradient (moe_norm_backward):
//   h' = beta h + alpha g * N_post(o),   x' = N_pre(h')
// with N(v) = (v - mu) r w + b, r = 1 / sqrt(mean((v - mu)^2) + eps); mu = 0 and
// no b for RMS norms.
//
// Gradient, u = (v - mu) r the normalised value and dn the gradient of N(v):
//   dv = r (dn w - u mean(dn w u) - mean(dn w)),   dw = sum_t dn u,   db = sum_t dn
// (the last mean for layer norms only).  With G = dh' + dv of the pre norm:
//   dh = beta G,   dn_post = alpha g G,   dg = alpha G N_post(o).
//
// Both directions are bound by memory: one pass, every row read once and
// written once.  A block takes whole rows; a thread keeps its eight columns (or
// two runs of eight) of every operand in registers, so a mean and the
// second moment about it are two reductions over registers instead of two
// passes over memory.  All sums are in fp32, each over at most 16 values per
// thread and then a tree over the block, in a fixed order.
// Blocks walk over rows, which keeps the per-column vectors in registers and, in
// the gradient, the column sums in shared memory; each block writes its column
// sums to the workspace once and a second kernel adds them in block order.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int EPT = 8;  // consecutive columns per thread and run

// How a thread's EPT columns lie: VEC, columns [run*8*NT + tid*8, + 8), one or two
// 16-byte accesses; otherwise columns run*8*NT + i*NT + tid, for widths, strides
// or addresses that 16-byte accesses do not fit.
template <bool VEC>
__device__ __forceinline__ int col_of(int run, int i) {
  return VEC ? (run * blockDim.x + threadIdx.x) * EPT + i : (run * EPT + i) * blockDim.x + threadIdx.x;
}

template <typename T>
__device__ __forceinline__ float as_f32(T v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float as_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T as(float v);
template <>
__device__ __forceinline__ float as<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 as<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half as<__half>(float v) { return __float2half_rn(v); }

// A thread's EPT values of one row and run as loaded (converted when used, so that
// a prefetched row costs few registers).  Plain loads: an output may be the input's
// own array.
template <typename T>
struct Raw {
  T v[EPT];
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_raw(Raw<T>& r, const T* row, int run, int H) {
  if (VEC) {
    const int c = col_of<true>(run, 0);
    uint4* dst = reinterpret_cast<uint4*>(r.v);
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q)
      dst[q] = c < H ? *(reinterpret_cast<const uint4*>(row + c) + q) : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<false>(run, i);
      r.v[i] = c < H ? row[c] : as<T>(0.0f);
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row(T* row, int run, int H, const float (&v)[EPT]) {
  if (VEC) {
    const int c = col_of<true>(run, 0);
    if (c >= H) return;
    T t[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) t[i] = as<T>(v[i]);
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q)
      reinterpret_cast<uint4*>(row + c)[q] = reinterpret_cast<const uint4*>(t)[q];
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<false>(run, i);
      if (c < H) row[c] = as<T>(v[i]);
    }
  }
}

// Value c of a per-column vector stored in one of the three types.
__device__ __forceinline__ float column_value(const void* p, int dtype, int c) {
  if (dtype == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(p) + c);
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
  return __half2float(static_cast<const __half*>(p)[c]);
}

// A thread's columns of a per-column vector; `none` where there is no vector or column.
template <bool VEC>
__device__ __forceinline__ void load_columns(float (&v)[EPT], const void* p, int dtype, int run, int H, float none) {
  if (VEC) {
    const int c = col_of<true>(run, 0);
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] = none;
    if (p == nullptr || c >= H) return;
    if (dtype == MOE_DTYPE_F32) {
      const float4 lo = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c));
      const float4 hi = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + 1);
      v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
      v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    } else {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c));
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = dtype == MOE_DTYPE_BF16
                             ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]))
                             : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<false>(run, i);
      v[i] = p != nullptr && c < H ? column_value(p, dtype, c) : none;
    }
  }
}

// Sums of N values over the block, for every thread, in a fixed order.  Two buffers
// taken in turn: a warp can be at most one reduction ahead of the others' reads.
template <int N>
struct BlockSum {
  float (*buf)[32][N];  // [2][32][N] in shared memory
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
    if (nw == 1) return;
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < N; ++j) buf[turn][warp][j] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = lane < nw ? buf[turn][lane][j] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
    turn ^= 1;
  }
};

// 1 / sqrt(sum / H + eps) of the second moment's sum.
__device__ __forceinline__ float inv_std(float sum, float inv_h, float eps) { return 1.0f / sqrtf(sum * inv_h + eps); }

// ------------------------------------------------------------------ forward
// RUNS runs of eight columns per thread.  The next row's loads are issued before
// this row's reductions.
template <typename HT, typename OT, bool VEC, int RUNS, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_forward_kernel(NormArgs a) {
  __shared__ float s_sum[2][32][1];
  BlockSum<1> block_sum{s_sum};
  const int H = a.H;
  const float inv_h = 1.0f / static_cast<float>(H);
  const HT* h = static_cast<const HT*>(a.h);
  const OT* o = static_cast<const OT*>(a.o);
  HT* h_out = static_cast<HT*>(a.h_out);
  OT* x_out = static_cast<OT*>(a.x_out);

  Raw<HT> rh[RUNS], nh[RUNS];
  Raw<OT> ro[RUNS], no[RUNS];
  int t = blockIdx.x;
  if (t < a.T) {
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      load_raw<OT, VEC>(no[r], o + static_cast<size_t>(t) * a.ld_o, r, H);
      load_raw<HT, VEC>(nh[r], h + static_cast<size_t>(t) * a.ld_h, r, H);
    }
  }
  for (; t < a.T; t += gridDim.x) {
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      rh[r] = nh[r];
      ro[r] = no[r];
    }
    const int tn = t + gridDim.x;
    if (tn < a.T) {
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        load_raw<OT, VEC>(no[r], o + static_cast<size_t>(tn) * a.ld_o, r, H);
        load_raw<HT, VEC>(nh[r], h + static_cast<size_t>(tn) * a.ld_h, r, H);
      }
    }
    float v[RUNS][EPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r)
#pragma unroll
      for (int i = 0; i < EPT; ++i) v[r][i] = as_f32(ro[r].v[i]);

    // v = N(v): moments over the block, then the affine part
    auto normalise = [&](int kind, const void* w, const void* b) {
      if (kind == MOE_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
          for (int i = 0; i < EPT; ++i) s[0] += v[r][i];
        block_sum(s);
        const float mu = s[0] * inv_h;
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
          for (int i = 0; i < EPT; ++i) v[r][i] = col_of<VEC>(r, i) < H ? v[r][i] - mu : 0.0f;
      }
      float q[1] = {0.0f};
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) q[0] = fmaf(v[r][i], v[r][i], q[0]);
      block_sum(q);
      const float rs = inv_std(q[0], inv_h, a.eps);
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        float cw[EPT], cb[EPT];
        load_columns<VEC>(cw, w, a.w_dtype, r, H, 1.0f);
        load_columns<VEC>(cb, b, a.w_dtype, r, H, 0.0f);
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[r][i] = fmaf(v[r][i] * rs, cw[i], cb[i]);
      }
    };

    if (a.post != MOE_NORM_NONE) normalise(a.post, a.w_post, a.b_post);
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        float g[EPT];
        load_columns<VEC>(g, a.gate, a.w_dtype, r, H, 0.0f);
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[r][i] *= g[i];
      } else if (a.gate_kind == MOE_GATE_FULL) {
        Raw<OT> g;
        load_raw<OT, VEC>(g, static_cast<const OT*>(a.gate) + static_cast<size_t>(t) * a.ld_o, r, H);
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[r][i] *= as_f32(g.v[i]);
      } else if (a.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) v[r][i] *= gt;
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i)
        v[r][i] = col_of<VEC>(r, i) < H ? fmaf(a.alpha, v[r][i], a.beta * as_f32(rh[r].v[i])) : 0.0f;
      store_row<HT, VEC>(h_out + static_cast<size_t>(t) * a.ld_h, r, H, v[r]);
    }
    // x' is taken from h' before its rounding: one rounding each
    if (a.pre != MOE_NORM_NONE) {
      normalise(a.pre, a.w_pre, a.b_pre);
#pragma unroll
      for (int r = 0; r < RUNS; ++r) store_row<OT, VEC>(x_out + static_cast<size_t>(t) * a.ld_o, r, H, v[r]);
    }
  }
}

// ------------------------------------------------------------------ backward
// acc: this block's column sums, `nacc` vectors of H, in shared memory or (where
// they do not fit) in its part of the workspace; each column belongs to one
// thread, so they need no barrier.
template <bool VEC>
__device__ __forceinline__ void add_columns(float* acc, int run, int H, const float (&v)[EPT]) {
  if (VEC) {
    const int c = col_of<true>(run, 0);
    if (c >= H) return;
    float4* p = reinterpret_cast<float4*>(acc + c);
    float4 x = p[0], y = p[1];
    x.x += v[0]; x.y += v[1]; x.z += v[2]; x.w += v[3];
    y.x += v[4]; y.y += v[5]; y.z += v[6]; y.w += v[7];
    p[0] = x;
    p[1] = y;
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<false>(run, i);
      if (c < H) acc[c] += v[i];
    }
  }
}

template <typename HT, typename OT, bool VEC, int RUNS, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_backward_kernel(NormArgs a) {
  extern __shared__ float4 s_acc4[];
  __shared__ float s_sum[2][32][4];
  BlockSum<4> block_sum{s_sum};
  const int H = a.H;
  const float inv_h = 1.0f / static_cast<float>(H);
  float* part = a.partials + static_cast<size_t>(blockIdx.x) * a.nacc * H;
  float* acc = a.acc_in_smem ? reinterpret_cast<float*>(s_acc4) : part;
  for (int j = 0; j < a.nacc; ++j)
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if (VEC) {
        const int c = col_of<true>(r, 0);
        if (c < H) {
          float4* p = reinterpret_cast<float4*>(acc + static_cast<size_t>(j) * H + c);
          p[0] = p[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int c = col_of<false>(r, i);
          if (c < H) acc[static_cast<size_t>(j) * H + c] = 0.0f;
        }
      }
    }

  const bool pre = a.pre != MOE_NORM_NONE, post = a.post != MOE_NORM_NONE;
  const bool layer_pre = a.pre == MOE_NORM_LAYER, layer_post = a.post == MOE_NORM_LAYER;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
    float G[RUNS][EPT], hc[RUNS][EPT], dx[RUNS][EPT], oc[RUNS][EPT];
    Raw<HT> rg[RUNS], rh[RUNS];
    Raw<OT> rx[RUNS], ro[RUNS];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if (a.dh_out) load_raw<HT, VEC>(rg[r], static_cast<const HT*>(a.dh_out) + at_h, r, H);
      if (pre) {
        load_raw<HT, VEC>(rh[r], static_cast<const HT*>(a.h) + at_h, r, H);
        load_raw<OT, VEC>(rx[r], static_cast<const OT*>(a.dx_out) + at_o, r, H);
      }
      load_raw<OT, VEC>(ro[r], static_cast<const OT*>(a.o) + at_o, r, H);
    }
#pragma unroll
    for (int r = 0; r < RUNS; ++r)
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        G[r][i] = a.dh_out ? as_f32(rg[r].v[i]) : 0.0f;
        hc[r][i] = pre ? as_f32(rh[r].v[i]) : 0.0f;
        dx[r][i] = pre ? as_f32(rx[r].v[i]) : 0.0f;
        oc[r][i] = as_f32(ro[r].v[i]);
      }
    if (layer_pre || layer_post) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          s[0] += hc[r][i];
          s[1] += oc[r][i];
        }
      block_sum(s);
      const float mh = layer_pre ? s[0] * inv_h : 0.0f, mo = layer_post ? s[1] * inv_h : 0.0f;
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const bool in = col_of<VEC>(r, i) < H;
          hc[r][i] = in ? hc[r][i] - mh : 0.0f;
          oc[r][i] = in ? oc[r][i] - mo : 0.0f;
        }
    }
    // second moments, and the two means of the pre norm's gradient
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float dxw[RUNS][EPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      load_columns<VEC>(dxw[r], pre ? a.w_pre : nullptr, a.w_dtype, r, H, 1.0f);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        dxw[r][i] *= dx[r][i];
        s[0] = fmaf(hc[r][i], hc[r][i], s[0]);
        s[1] = fmaf(dxw[r][i], hc[r][i], s[1]);
        s[2] += dxw[r][i];
        s[3] = fmaf(oc[r][i], oc[r][i], s[3]);
      }
    }
    block_sum(s);
    const float ro_std = post ? inv_std(s[3], inv_h, a.eps) : 1.0f;
    if (pre) {
      const float rs = inv_std(s[0], inv_h, a.eps);
      const float m1 = s[1] * rs * inv_h;                     // mean(dx w u)
      const float m0 = layer_pre ? s[2] * inv_h : 0.0f;       // mean(dx w)
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        float du[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const float u = hc[r][i] * rs;
          G[r][i] += rs * (dxw[r][i] - u * m1 - m0);
          du[i] = dx[r][i] * u;
        }
        if (a.acc_dw_pre >= 0) add_columns<VEC>(acc + static_cast<size_t>(a.acc_dw_pre) * H, r, H, du);
        if (a.acc_db_pre >= 0) add_columns<VEC>(acc + static_cast<size_t>(a.acc_db_pre) * H, r, H, dx[r]);
      }
    }
    if (a.dh) {
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        float d[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) d[i] = a.beta * G[r][i];
        store_row<HT, VEC>(static_cast<HT*>(a.dh) + at_h, r, H, d);
      }
    }
    // block side: G <- alpha G (gradient of the gated, normalised o), dn = g G
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float dn[RUNS][EPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      float g[EPT], w[EPT], b[EPT], tg[EPT], du[EPT];
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load_columns<VEC>(g, a.gate, a.w_dtype, r, H, 0.0f);
      } else if (a.gate_kind == MOE_GATE_FULL) {
        Raw<OT> graw;
        load_raw<OT, VEC>(graw, static_cast<const OT*>(a.gate) + at_o, r, H);
#pragma unroll
        for (int i = 0; i < EPT; ++i) g[i] = as_f32(graw.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) g[i] = gt;
      }
      load_columns<VEC>(w, post ? a.w_post : nullptr, a.w_dtype, r, H, 1.0f);
      if (a.dgate) load_columns<VEC>(b, post ? a.b_post : nullptr, a.w_dtype, r, H, 0.0f);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const bool in = col_of<VEC>(r, i) < H;
        const float ag = in ? a.alpha * G[r][i] : 0.0f;
        oc[r][i] *= ro_std;  // u of the post norm, or o itself
        const float dg = ag * g[i];
        du[i] = dg * oc[r][i];
        if (a.dgate) tg[i] = ag * fmaf(oc[r][i], w[i], b[i]);
        dn[r][i] = dg * w[i];
        d[0] = fmaf(dn[r][i], oc[r][i], d[0]);
        d[1] += dn[r][i];
        if (a.dgate) d[2] += tg[i];
        g[i] = dg;
      }
      if (a.acc_dw_post >= 0) add_columns<VEC>(acc + static_cast<size_t>(a.acc_dw_post) * H, r, H, du);
      if (a.acc_db_post >= 0) add_columns<VEC>(acc + static_cast<size_t>(a.acc_db_post) * H, r, H, g);
      if (a.dgate && a.gate_kind == MOE_GATE_CHANNEL)
        add_columns<VEC>(acc + static_cast<size_t>(a.acc_dgate) * H, r, H, tg);
      if (a.dgate && a.gate_kind == MOE_GATE_FULL)
        store_row<OT, VEC>(static_cast<OT*>(a.dgate) + at_o, r, H, tg);
    }
    const bool token_sum = a.dgate && a.gate_kind == MOE_GATE_TOKEN;
    if (post || token_sum) block_sum(d);
    if (token_sum && threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = d[2];
    if (a.d_o) {
      const float m1 = post ? d[0] * inv_h : 0.0f, m0 = layer_post ? d[1] * inv_h : 0.0f;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) dn[r][i] = ro_std * (dn[r][i] - oc[r][i] * m1 - m0);
        store_row<OT, VEC>(static_cast<OT*>(a.d_o) + at_o, r, H, dn[r]);
      }
    }
  }
  if (a.acc_in_smem) {  // each thread hands over the columns that it summed
    for (int j = 0; j < a.nacc; ++j)
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int c = col_of<VEC>(r, i);
          if (c < H) part[static_cast<size_t>(j) * H + c] = acc[static_cast<size_t>(j) * H + c];
        }
  }
}

// out[j][c] = sum over the blocks' partials, 32 columns per block; 32 rows of
// threads add every 32nd partial in ascending order and the 32 sums are added in
// order, so the result does not depend on timing.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ partials, int nparts, size_t stride,
                                                           int n, ColumnOutputs out, int width) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < n) {
#pragma unroll 4
    for (int p = threadIdx.y; p < nparts; p += 32) v += partials[static_cast<size_t>(p) * stride + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    out.p[c / width][c % width] = sum;
  }
}

// Threads of a block for rows of H columns: one run of eight columns each up to
// 8192 columns, two beyond (where the gradient's registers no longer hold a row).
inline int norm_threads(int H) {
  const int t = (H + EPT - 1) / EPT;
  return t >= 1024 ? 1024 : (t + 31) / 32 * 32;
}

// Blocks: as many as are resident at 1024 threads per SM of a 152-SM part (a pure
// function of the problem, because the workspace holds one set of sums for each).
inline int norm_blocks(int T, int H) {
  const int per_sm = 1024 / norm_threads(H);
  const int cap = 152 * (per_sm > 8 ? 8 : per_sm);
  return T < cap ? T : cap;
}

constexpr size_t kNormAccSmemMax = 200 * 1024;

template <typename HT, typename OT, bool VEC, int RUNS, int MAXT>
cudaError_t forward_of(const NormArgs& a, int threads, cudaStream_t s) {
  const int cap = 152 * (1024 / threads);
  norm_forward_kernel<HT, OT, VEC, RUNS, MAXT><<<a.T < cap ? a.T : cap, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename HT, typename OT, bool VEC, int RUNS, int MAXT>
cudaError_t backward_of(const NormArgs& a, int threads, cudaStream_t s) {
  static const cudaError_t attr = cudaFuncSetAttribute(norm_backward_kernel<HT, OT, VEC, RUNS, MAXT>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(kNormAccSmemMax));
  if (attr != cudaSuccess) return attr;
  const size_t smem = a.acc_in_smem ? static_cast<size_t>(a.nacc) * a.H * sizeof(float) : 0;
  norm_backward_kernel<HT, OT, VEC, RUNS, MAXT><<<norm_blocks(a.T, a.H), threads, smem, s>>>(a);
  return cudaGetLastError();
}

// MAXT: registers for up to 4096 columns (512 threads) or for more.
#define MOE_NORM_SHAPES(F)                                                       \
  const int threads = norm_threads(a.H);                                         \
  if (a.H > threads * EPT)                                                       \
    return vec ? F<HT, OT, true, 2, 1024>(a, threads, s) : F<HT, OT, false, 2, 1024>(a, threads, s); \
  if (threads > 512)                                                             \
    return vec ? F<HT, OT, true, 1, 1024>(a, threads, s) : F<HT, OT, false, 1, 1024>(a, threads, s); \
  return vec ? F<HT, OT, true, 1, 512>(a, threads, s) : F<HT, OT, false, 1, 512>(a, threads, s)

template <typename HT, typename OT>
cudaError_t forward_types(const NormArgs& a, bool vec, cudaStream_t s) {
  MOE_NORM_SHAPES(forward_of);
}

template <typename HT, typename OT>
cudaError_t backward_types(const NormArgs& a, bool vec, cudaStream_t s) {
  MOE_NORM_SHAPES(backward_of);
}

#define MOE_NORM_TYPES(F)                                                                              \
  (h_dtype == MOE_DTYPE_F32                                                                            \
       ? (o_dtype == MOE_DTYPE_F32    ? F<float, float>(a, vec, s)                                     \
          : o_dtype == MOE_DTYPE_BF16 ? F<float, __nv_bfloat16>(a, vec, s)                             \
                                      : F<float, __half>(a, vec, s))                                   \
       : (h_dtype == MOE_DTYPE_BF16 ? F<__nv_bfloat16, __nv_bfloat16>(a, vec, s) : F<__half, __half>(a, vec, s)))

}  // namespace

size_t norm_partials_bytes(int T, int H) { return static_cast<size_t>(norm_blocks(T, H)) * 5 * H * sizeof(float); }

cudaError_t launch_norm_forward(const NormArgs& a, int h_dtype, int o_dtype, bool vec, cudaStream_t s) {
  stage_begin("norm_forward", s);
  const cudaError_t err = MOE_NORM_TYPES(forward_types);
  stage_end(s);
  return err;
}

cudaError_t launch_norm_backward(const NormArgs& args, int h_dtype, int o_dtype, bool vec, float* const (&sums)[5],
                                 cudaStream_t s) {
  NormArgs a = args;
  // the sums that are wanted, packed: vector j of a block's partials is out.p[j]
  int* slot[5] = {&a.acc_dw_post, &a.acc_db_post, &a.acc_dw_pre, &a.acc_db_pre, &a.acc_dgate};
  ColumnOutputs out{};
  a.nacc = 0;
  for (int j = 0; j < 5; ++j) {
    *slot[j] = sums[j] ? a.nacc : -1;
    if (sums[j]) out.p[a.nacc++] = sums[j];
  }
  a.acc_in_smem = static_cast<size_t>(a.nacc) * a.H * sizeof(float) <= kNormAccSmemMax;
  stage_begin("norm_backward", s);
  cudaError_t err = MOE_NORM_TYPES(backward_types);
  stage_end(s);
  if (err == cudaSuccess && a.nacc > 0)
    err = launch_column_sums(a.partials, norm_blocks(a.T, a.H), static_cast<size_t>(a.nacc) * a.H, a.nacc * a.H, out,
                             a.H, s);
  return err;
}

cudaError_t launch_column_sums(const float* partials, int nparts, size_t stride, int n, const ColumnOutputs& out,
                               int width, cudaStream_t s) {
  stage_begin("column_sums", s);
  column_sums_kernel<<<(n + 31) / 32, dim3(32, 32), 0, s>>>(partials, nparts, stride, n, out, width);
  const cudaError_t err = cudaGetLastError();
  stage_end(s);
  return err;
}

}  // namespace moe
