// Routing rules beyond top-k of raw scores (moe_route_ex) and the gradient of
// the routing weights into the scores (moe_route_backward).
//
// Forward, per token: p = softmax over the experts or sigmoid of the scores;
// selection key = p + bias (the score itself without a bias: both score
// functions are monotone, so the order needs no rounding); with expert groups
// only the topk_group best groups stay; the k largest keys win, ties to the
// lower expert id; w = p of the selected, optionally divided by their sum, times
// a constant.  Renormalised softmax weights are the softmax over the selected
// scores, computed with the maximum of those, so they never underflow as a whole.
//
// Backward, with r_j the weights before the constant c and g_j = c dw_j:
//   softmax, renormalised   ds_j = r_j (g_j - sum_i r_i g_i)            j selected
//   sigmoid, renormalised   ds_j = r_j (g_j - sum_i r_i g_i) (1 - p_j)  j selected
//   sigmoid                 ds_j = g_j p_j (1 - p_j)                    j selected
//   softmax                 ds_e = p_e (g_e - sum_j p_j g_j)            every e
// Only the last needs the scores of the experts that were not selected.
//
// One warp per token in both directions.  The bytes are one row of E scores in
// and k pairs out (a row of E gradients out); the arithmetic per row (exp, a
// division where p is needed for every expert, k selection rounds) is of the
// same size, which is why rows are spread one per warp with eight warps a block:
// the long selection chains of many warps overlap.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "routing.cuh"

namespace moe {
namespace {

constexpr int kRouterWarps = 8;

template <typename ST>
__device__ __forceinline__ float to_f32(ST v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename ST>
__device__ __forceinline__ ST from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A score as the rules read it: NaN counts as -inf (masked), +inf as the largest
// finite value, so that no weight is NaN.
template <typename ST>
__device__ __forceinline__ float clean_score(ST raw) {
  const float v = to_f32(raw);
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }

// sigmoid(x) e^-m for x <= m <= 0; sigmoid(x) for m = 0.
__device__ __forceinline__ float scaled_sigmoid(float x, float m) {
  return m < 0.0f ? expf(x - m) / (1.0f + expf(x)) : sigmoid_f32(x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Selection keys: 0 = not to be taken (no such expert, group not kept, already
// taken), 1 = masked expert (taken only after every other), else the
// order-preserving image of the key.
constexpr uint32_t kKeyTaken = 0u, kKeyMasked = 1u;
__device__ __forceinline__ uint32_t live_key(float v) {
  const uint32_t b = score_bits(v);
  return b < 2u ? 2u : b;
}

template <int MAXV>
__device__ __forceinline__ void local_best(const uint32_t (&key)[MAXV], uint32_t& best, int& slot) {
  best = key[0];
  slot = 0;
#pragma unroll
  for (int i = 1; i < MAXV; ++i)
    if (key[i] > best) {
      best = key[i];
      slot = i;
    }
}

template <int MAXV, typename ST>
__global__ void __launch_bounds__(kRouterWarps * 32) route_ex_kernel(const ST* __restrict__ scores, RouteArgs a) {
  extern __shared__ float s_rows[];  // group limits only: one row of E ranking values per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouterWarps + warp;
  dep_wait();
  dep_launch();
  if (t >= a.T) return;  // no block-wide barrier below
  const ST* row = scores + static_cast<size_t>(t) * a.ld;
  const int E = a.E, k = a.k;
  float x[MAXV];
#pragma unroll
  for (int i = 0; i < MAXV; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < E ? clean_score(row[e]) : -INFINITY;
  }
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  const bool sum_ranked = a.n_group > 1 && a.group_best == 2;
  const bool need_p = a.bias != nullptr || sum_ranked;

  // softmax over the whole row: maximum and sum over the experts that are not masked
  float top = 0.0f, total = 0.0f;
  if (softmax && (need_p || !a.renormalise)) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    top = m > -INFINITY ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
    total = warp_sum(total);
  }

  uint32_t key[MAXV];
#pragma unroll
  for (int i = 0; i < MAXV; ++i) {
    const int e = i * 32 + lane;
    const bool live = x[i] > -INFINITY;
    float v = x[i], ranked = x[i];
    if (need_p) {
      const float p = !live ? 0.0f : softmax ? expf(x[i] - top) / total : sigmoid_f32(x[i]);
      if (a.bias) v = p + (e < E ? __ldg(a.bias + e) : 0.0f);
      ranked = sum_ranked && !a.bias ? p : v;
    }
    key[i] = e >= E ? kKeyTaken : live ? live_key(v) : kKeyMasked;
    if (a.n_group > 1 && e < E) s_rows[warp * E + e] = live ? ranked : -INFINITY;
  }

  if (a.n_group > 1) {
    // lpg lanes per group (a power of two) rank it: best key, or sum of the best
    // two keys of experts that are not masked
    __syncwarp();
    const int G = a.n_group, gs = E / G;
    int lpg = 1;
    while (lpg * 2 * G <= 32) lpg *= 2;
    const int g = lane / lpg, sub = lane & (lpg - 1);
    float b1 = -INFINITY, b2 = -INFINITY;
    if (g < G)
      for (int e = sub; e < gs; e += lpg) {
        const float v = s_rows[warp * E + g * gs + e];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
    for (int o = 1; o < lpg; o <<= 1) {
      const float c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
      b1 = fmaxf(b1, c1);
    }
    float rank = b1;
    if (a.group_best == 2 && b2 > -INFINITY) rank = b1 + b2;
    const uint32_t mine = rank > -INFINITY ? live_key(rank) : kKeyMasked;
    int before = 0;  // groups that come before this one
    for (int h = 0; h < G; ++h) {
      const uint32_t other = __shfl_sync(0xffffffffu, mine, h * lpg);
      before += (other > mine || (other == mine && h < g)) ? 1 : 0;
    }
    const unsigned kept = __ballot_sync(0xffffffffu, g < G && sub == 0 && before < a.topk_group);
    // e / gs by a multiplication: e < 512, so e * ceil(2^22 / gs) is exact after the shift
    const unsigned inv = ((1u << 22) + gs - 1) / gs;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const unsigned ge = (static_cast<unsigned>(i * 32 + lane) * inv) >> 22;
      if (key[i] != kKeyTaken && !((kept >> (ge * lpg)) & 1u)) key[i] = kKeyTaken;
    }
  }

  // k rounds: the warp-wide largest key, then the lowest id that holds it
  uint32_t best;
  int slot, my_id = 0;
  local_best(key, best, slot);
  for (int j = 0; j < k; ++j) {
    const uint32_t b = __reduce_max_sync(0xffffffffu, best);
    const unsigned cand = best == b ? static_cast<unsigned>(slot * 32 + lane) : 0xffffffffu;
    const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, cand));
    if (lane == j) my_id = id;
    if ((id & 31) == lane) {
#pragma unroll
      for (int i = 0; i < MAXV; ++i)
        if (i == (id >> 5)) key[i] = kKeyTaken;
      local_best(key, best, slot);
    }
  }

  // weights: lane j holds slot j
  const float xj = lane < k ? clean_score(row[my_id]) : -INFINITY;
  const bool live = xj > -INFINITY;
  float p;
  if (softmax) {
    if (a.renormalise) top = warp_max(xj);
    p = live ? expf(xj - top) : 0.0f;
    if (!a.renormalise) p = live ? p / total : 0.0f;
  } else {
    const float m = a.renormalise ? fminf(warp_max(xj), 0.0f) : 0.0f;
    p = live ? scaled_sigmoid(xj, m) : 0.0f;
  }
  if (a.renormalise) {
    const float sum = warp_sum(p);
    p = sum > 0.0f ? p / sum : 0.0f;
  }
  if (lane < k) {
    a.ids[static_cast<size_t>(t) * k + lane] = my_id;
    a.w[static_cast<size_t>(t) * k + lane] = p * a.scale;
  }
}

// The gradient row is put together in shared memory and written once, coalesced.
template <int MAXV, typename ST, bool WHOLE>
__global__ void __launch_bounds__(kRouterWarps * 32)
    route_backward_kernel(const ST* __restrict__ scores, const int32_t* __restrict__ ids, const float* __restrict__ dw,
                          ST* __restrict__ dscores, RouteArgs a, long long ld_d) {
  extern __shared__ float s_rows[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouterWarps + warp;
  dep_wait();
  dep_launch();
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  const ST* row = scores + static_cast<size_t>(t) * a.ld;
  float* g = s_rows + warp * E;
  int id = -1;
  float gj = 0.0f;
  if (lane < k) {
    id = ids[static_cast<size_t>(t) * k + lane];
    gj = a.scale * dw[static_cast<size_t>(t) * k + lane];
    if (id < 0 || id >= E) id = -1;  // no such expert: no part in the sums, nothing written
  }
  const float xj = id >= 0 ? clean_score(row[id]) : -INFINITY;
  const bool live = xj > -INFINITY;
  float x[MAXV];
  if (WHOLE) {
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int e = i * 32 + lane;
      x[i] = e < E ? clean_score(row[e]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < MAXV; ++i)
    if (i * 32 + lane < E) g[i * 32 + lane] = 0.0f;
  __syncwarp();

  float top = 0.0f, total = 0.0f, d = 0.0f;
  if (WHOLE) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    top = m > -INFINITY ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      x[i] = x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
      total += x[i];
    }
    total = warp_sum(total);
    const float pj = live ? expf(xj - top) / total : 0.0f;
    const float dot = warp_sum(pj * gj);
    if (id >= 0) atomicAdd(g + id, gj);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int e = i * 32 + lane;
      if (e < E) g[e] = x[i] > 0.0f ? x[i] / total * (g[e] - dot) : 0.0f;
    }
  } else {
    if (a.score_fn == MOE_SCORE_SOFTMAX) {  // renormalised
      const float m = warp_max(xj);
      const float e = live ? expf(xj - m) : 0.0f;
      const float sum = warp_sum(e);
      const float r = live ? e / sum : 0.0f;
      d = r * (gj - warp_sum(r * gj));
    } else {
      const float m = a.renormalise ? fminf(warp_max(xj), 0.0f) : 0.0f;
      const float p = live ? scaled_sigmoid(xj, m) : 0.0f;
      const float q = live ? sigmoid_f32(-xj) : 0.0f;  // 1 - sigmoid without cancellation
      if (a.renormalise) {
        const float sum = warp_sum(p);
        const float r = sum > 0.0f ? p / sum : 0.0f;
        d = r * (gj - warp_sum(r * gj)) * q;
      } else {
        d = gj * p * q;
      }
    }
    if (id >= 0) atomicAdd(g + id, d);  // ids of a row differ, so each value is added to a zero once
  }
  __syncwarp();
  ST* out = dscores + static_cast<size_t>(t) * ld_d;
#pragma unroll
  for (int i = 0; i < MAXV; ++i)
    if (i * 32 + lane < E) out[i * 32 + lane] = from_f32<ST>(g[i * 32 + lane]);
}

inline int slots_of(int E) {
  int v = 1;
  while (v * 32 < E) v *= 2;
  return v;
}

template <typename ST>
cudaError_t route_ex_of(const void* scores, const RouteArgs& a, cudaStream_t s) {
  const dim3 grid((a.T + kRouterWarps - 1) / kRouterWarps);
  const size_t smem = a.n_group > 1 ? static_cast<size_t>(kRouterWarps) * a.E * sizeof(float) : 0;
  const ST* sc = static_cast<const ST*>(scores);
  switch (slots_of(a.E)) {
    case 1: return launch_dependent(route_ex_kernel<1, ST>, grid, kRouterWarps * 32, smem, s, sc, a);
    case 2: return launch_dependent(route_ex_kernel<2, ST>, grid, kRouterWarps * 32, smem, s, sc, a);
    case 4: return launch_dependent(route_ex_kernel<4, ST>, grid, kRouterWarps * 32, smem, s, sc, a);
    case 8: return launch_dependent(route_ex_kernel<8, ST>, grid, kRouterWarps * 32, smem, s, sc, a);
    default: return launch_dependent(route_ex_kernel<16, ST>, grid, kRouterWarps * 32, smem, s, sc, a);
  }
}

template <int MAXV, typename ST>
cudaError_t route_backward_of(const ST* sc, const RouteArgs& a, const int32_t* ids, const float* dw, ST* ds, long long ld_d,
                              dim3 grid, size_t smem, cudaStream_t s) {
  if (a.score_fn == MOE_SCORE_SOFTMAX && !a.renormalise)
    return launch_dependent(route_backward_kernel<MAXV, ST, true>, grid, kRouterWarps * 32, smem, s, sc, ids, dw, ds, a, ld_d);
  return launch_dependent(route_backward_kernel<MAXV, ST, false>, grid, kRouterWarps * 32, smem, s, sc, ids, dw, ds, a, ld_d);
}

template <typename ST>
cudaError_t route_backward_of(const void* scores, const RouteArgs& a, const int32_t* ids, const float* dw,
                              void* dscores, long long ld_d, cudaStream_t s) {
  const dim3 grid((a.T + kRouterWarps - 1) / kRouterWarps);
  const size_t smem = static_cast<size_t>(kRouterWarps) * a.E * sizeof(float);
  const ST* sc = static_cast<const ST*>(scores);
  ST* ds = static_cast<ST*>(dscores);
  switch (slots_of(a.E)) {
    case 1: return route_backward_of<1, ST>(sc, a, ids, dw, ds, ld_d, grid, smem, s);
    case 2: return route_backward_of<2, ST>(sc, a, ids, dw, ds, ld_d, grid, smem, s);
    case 4: return route_backward_of<4, ST>(sc, a, ids, dw, ds, ld_d, grid, smem, s);
    case 8: return route_backward_of<8, ST>(sc, a, ids, dw, ds, ld_d, grid, smem, s);
    default: return route_backward_of<16, ST>(sc, a, ids, dw, ds, ld_d, grid, smem, s);
  }
}

}  // namespace

cudaError_t launch_route_ex(const void* scores, int dtype, const RouteArgs& a, cudaStream_t s) {
  stage_begin("route_ex", s);
  const cudaError_t err = dtype == MOE_DTYPE_F32    ? route_ex_of<float>(scores, a, s)
                          : dtype == MOE_DTYPE_BF16 ? route_ex_of<__nv_bfloat16>(scores, a, s)
                                                    : route_ex_of<__half>(scores, a, s);
  stage_end(s);
  return err;
}

cudaError_t launch_route_backward(const void* scores, int dtype, const RouteArgs& a, const int32_t* ids,
                                  const float* dw, void* dscores, long long ld_d, cudaStream_t s) {
  stage_begin("route_backward", s);
  const cudaError_t err =
      dtype == MOE_DTYPE_F32    ? route_backward_of<float>(scores, a, ids, dw, dscores, ld_d, s)
      : dtype == MOE_DTYPE_BF16 ? route_backward_of<__nv_bfloat16>(scores, a, ids, dw, dscores, ld_d, s)
                                : route_backward_of<__half>(scores, a, ids, dw, dscores, ld_d, s);
  stage_end(s);
  return err;
}

}  // namespace moe
