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
// The bytes are one row of E scores in and k pairs out (a row of E gradients out), but
// the selection rounds, and p where the keys need it for every expert, are some hundred
// instructions per row: rows in large numbers are bound by instructions, few rows by the
// length of the chain of rounds.  So the forward gives a row few lanes with 16 experts
// each when there are many rows (a round's bookkeeping is then shared by the 2 to 16 rows
// of a warp), and a whole warp when there are few.
//
// Measured, 16384 tokens of 128 fp32 sigmoid scores with a bias, 4 of 8 groups, top 8:
// 13.7 us against 1.4 us for the bytes; with 256 experts under a profiler 25.7 us, 16.1 M
// warp instructions at 61 % of the issue slots.  Eight tokens: 4.2 us, of which launch and
// drain are 2.2.  The gradient touches k values per row (all of E without renormalised
// softmax weights) and is bound by its bytes and the launch: 4.7 us for 16384 x 128, k = 8.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kRouterWarps = 8;
// Warps of a forward block: two lanes per row keep 16 rows per warp in shared memory, whose
// ids, keys and group ranks for eight warps would pass the 48 KB that a block has unasked.
__host__ __device__ constexpr int router_warps(int sub) { return sub == 2 ? kRouterWarps / 2 : kRouterWarps; }
constexpr int kFewWarps = 4 * 152;  // below: a warp per row leaves no scheduler without one

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
// For the keys, which every expert needs: within 2e-7 of the sigmoid, a third of the instructions.
__device__ __forceinline__ float sigmoid_key(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// sigmoid(x) e^-m for x <= m <= 0; sigmoid(x) for m = 0.
__device__ __forceinline__ float scaled_sigmoid(float x, float m) {
  return m < 0.0f ? expf(x - m) / (1.0f + expf(x)) : sigmoid_f32(x);
}

template <int SUB>
__device__ __forceinline__ float sub_max(float v) {
#pragma unroll
  for (int o = SUB / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int SUB>
__device__ __forceinline__ float sub_sum(float v) {
#pragma unroll
  for (int o = SUB / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int VPL>
__device__ __forceinline__ float best_of(const float (&key)[VPL]) {
  float b = key[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) b = fmaxf(b, key[i]);
  return b;
}

// A lane's VPL consecutive scores, cleaned; -inf past expert E.
template <int VPL, typename ST>
__device__ __forceinline__ void load_scores(float (&x)[VPL], const ST* __restrict__ row, int e0, int E, bool vec) {
  constexpr int PER = 16 / sizeof(ST);  // scores per 16-byte load
  if (VPL % PER == 0 && vec) {          // E is a multiple of PER too
#pragma unroll
    for (int q = 0; q < VPL / PER; ++q) {
      alignas(16) ST raw[PER];
      if (e0 + q * PER < E) {
        *reinterpret_cast<uint4*>(raw) = __ldg(reinterpret_cast<const uint4*>(row + e0 + q * PER));
#pragma unroll
        for (int i = 0; i < PER; ++i) x[q * PER + i] = clean_score(raw[i]);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) x[q * PER + i] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < E ? clean_score(row[e0 + i]) : -INFINITY;
  }
}

template <int VPL>
__device__ __forceinline__ void load_bias(float (&b)[VPL], const float* __restrict__ bias, int e0, int E, bool vec) {
  if (VPL % 4 == 0 && vec) {
#pragma unroll
    for (int q = 0; q < VPL / 4; ++q) {
      const float4 f = e0 + 4 * q < E ? __ldg(reinterpret_cast<const float4*>(bias + e0) + q) : make_float4(0, 0, 0, 0);
      b[4 * q] = f.x; b[4 * q + 1] = f.y; b[4 * q + 2] = f.z; b[4 * q + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) b[i] = e0 + i < E ? __ldg(bias + e0 + i) : 0.0f;
  }
}

// SUB lanes per token with VPL consecutive experts each.  A key is the fp32 value that
// ranks its expert; -inf: masked (taken only after every other); NaN: not to be taken
// (no such expert, group not kept, already taken), which fmaxf passes over and no
// comparison matches.  Equal keys: the lowest lane holds the lowest ids.
template <int VPL, int SUB, typename ST>
__global__ void __launch_bounds__(router_warps(SUB) * 32) route_ex_kernel(const ST* __restrict__ scores, RouteArgs a) {
  constexpr int TOKENS = 32 / SUB;  // per warp
  constexpr int WARPS = router_warps(SUB);
  __shared__ int s_ids[WARPS][TOKENS][kMaxK];
  // group limits only: per token VPL x SUB ranking values, one word of padding for each
  // VPL, and the ranks of up to 32 groups
  extern __shared__ float s_rows[];
  constexpr int PITCH = SUB * (VPL + 1), GPITCH = 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = lane / SUB, sub = lane & (SUB - 1);
  const int t = (blockIdx.x * WARPS + warp) * TOKENS + tok;
  dep_wait();
  dep_launch();
  if ((blockIdx.x * WARPS + warp) * TOKENS >= a.T) return;  // no block-wide barrier below
  const bool mine = t < a.T;  // a warp's last tokens may be missing: they shadow token T - 1
  const ST* row = scores + static_cast<size_t>(mine ? t : a.T - 1) * a.ld;
  const int E = a.E, k = a.k, e0 = sub * VPL;
  float x[VPL];
  load_scores<VPL, ST>(x, row, e0, E, a.vec);
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  const bool sum_ranked = a.n_group > 1 && a.group_best == 2;
  const bool need_p = a.bias != nullptr || sum_ranked;

  // softmax over the whole row: maximum and sum over the experts that are not masked
  float top = 0.0f, total = 0.0f;
  if (softmax && (need_p || !a.renormalise)) {
    const float m = sub_max<SUB>(best_of<VPL>(x));
    top = m > -INFINITY ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += expf(x[i] - top);  // a masked score adds expf(-inf) = 0
    total = sub_sum<SUB>(total);
  }

  // x becomes the key
  float* ranked = s_rows + (warp * TOKENS + tok) * (PITCH + GPITCH);
  if (need_p) {
    const float inv_total = total > 0.0f ? __fdividef(1.0f, total) : 0.0f;
    float bias[VPL];
    if (a.bias) load_bias<VPL>(bias, a.bias, e0, E, a.bias_vec);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool live = x[i] > -INFINITY;  // p of a masked score comes out as 0
      const float p = softmax ? __expf(x[i] - top) * inv_total : sigmoid_key(x[i]);
      float v = x[i];
      if (a.bias) {
        v = p + bias[i];
        v = v == v ? v : -3.402823466e38f;  // a key that is no number (infinite bias) still has a place
      }
      if (sum_ranked) ranked[sub * (VPL + 1) + i] = !live ? -INFINITY : a.bias ? v : p;
      x[i] = live ? v : -INFINITY;
    }
  }
  if (a.n_group > 1 && !sum_ranked) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) ranked[sub * (VPL + 1) + i] = x[i];
  }
  if (SUB * VPL != E) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e0 + i >= E) x[i] = NAN;
  }

  if (a.n_group > 1) {
    // Rank of each group: best key, or sum of the best two keys of experts that are not
    // masked.  Few groups: lpg lanes per group; many: several groups per lane.
    __syncwarp();
    float* rank = ranked + PITCH;
    const int G = a.n_group, gs = E / G;
    int lpg = 1;
    while (lpg * 2 * G <= SUB) lpg *= 2;
    const int per_pass = SUB / lpg;
    for (int g0 = 0; g0 < G; g0 += per_pass) {
      const int g = g0 + sub / lpg;
      float b1 = -INFINITY, b2 = -INFINITY;
      if (g < G)
        for (int i = sub & (lpg - 1); i < gs; i += lpg) {
          const int e = g * gs + i;
          const float v = ranked[e + e / VPL];
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
      for (int o = 1; o < lpg; o <<= 1) {
        const float c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
        b1 = fmaxf(b1, c1);
      }
      if (g < G && (sub & (lpg - 1)) == 0) rank[g] = a.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
    __syncwarp();
    // groups that fewer than topk_group others come before
    unsigned kept = 0u;
    for (int g = sub; g < G; g += SUB) {
      const float r = rank[g];
      int before = 0;
      for (int h = 0; h < G; ++h) {
        const float o = rank[h];
        before += (o > r || (o == r && h < g)) ? 1 : 0;
      }
      if (before < a.topk_group) kept |= 1u << g;
    }
#pragma unroll
    for (int o = SUB / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, o);
    int g = e0 / gs, left = (g + 1) * gs - e0;  // experts of group g from here on
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (g < 32 && !((kept >> g) & 1u)) x[i] = NAN;
      if (--left == 0) {
        ++g;
        left = gs;
      }
    }
  }

  // k rounds: the token's largest key, the lowest lane that holds it, its first expert with it
  float best = best_of<VPL>(x);
  const int base = lane & ~(SUB - 1);
  for (int j = 0; j < k; ++j) {
    const float b = sub_max<SUB>(best);
    unsigned holders = __ballot_sync(0xffffffffu, best == b);
    if (SUB < 32) holders = (holders >> base) & ((1u << (SUB & 31)) - 1u);
    if (holders != 0u && sub == __ffs(holders) - 1) {
      int at = 0;
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i) at = x[i] == b ? i : at;
      s_ids[warp][tok][j] = e0 + at;
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = i == at ? NAN : x[i];
      best = best_of<VPL>(x);
    }
    __syncwarp();
  }

  // weights: lane sub holds slots sub, sub + SUB, ..
  constexpr int SLOTS = (kMaxK + SUB - 1) / SUB;
  float xs[SLOTS];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    const int j = sub + q * SUB;
    if (q * SUB >= k) break;
    xs[q] = j < k ? clean_score(row[s_ids[warp][tok][j]]) : -INFINITY;
    m = fmaxf(m, xs[q]);
  }
  if (a.renormalise) {
    m = sub_max<SUB>(m);
    top = m > -INFINITY ? m : 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    if (q * SUB >= k) break;
    const bool live = xs[q] > -INFINITY;
    xs[q] = !live ? 0.0f : softmax ? expf(xs[q] - top) : scaled_sigmoid(xs[q], a.renormalise ? fminf(m, 0.0f) : 0.0f);
    sum += xs[q];
  }
  float factor = a.scale;
  if (a.renormalise) {
    sum = sub_sum<SUB>(sum);
    factor = sum > 0.0f ? a.scale / sum : 0.0f;
  } else if (softmax) {
    factor = total > 0.0f ? a.scale / total : 0.0f;
  }
  if (!mine) return;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    const int j = sub + q * SUB;
    if (q * SUB >= k) break;
    if (j < k) {
      a.ids[static_cast<size_t>(t) * k + j] = s_ids[warp][tok][j];
      a.w[static_cast<size_t>(t) * k + j] = xs[q] * factor;
    }
  }
}

// SUB lanes per token with VPL experts each, in runs of 16 bytes that alternate between the
// lanes (whole lines are written).  Every lane writes its part of the row (0, or the
// part that every expert has), then the selected experts' values are written over it:
// __syncwarp orders the two.
template <int VPL, int SUB, typename ST, bool WHOLE>
__global__ void __launch_bounds__(kRouterWarps * 32)
    route_backward_kernel(const ST* __restrict__ scores, const int32_t* __restrict__ ids, const float* __restrict__ dw,
                          ST* __restrict__ dscores, RouteArgs a, long long ld_d, bool vec_d) {
  constexpr int TOKENS = 32 / SUB;
  constexpr int SLOTS = (kMaxK + SUB - 1) / SUB;  // lane sub holds slots sub, sub + SUB, ..
  constexpr int PER = 16 / sizeof(ST);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (SUB - 1);
  const int t = (blockIdx.x * kRouterWarps + warp) * TOKENS + lane / SUB;
  dep_wait();
  dep_launch();
  if ((blockIdx.x * kRouterWarps + warp) * TOKENS >= a.T) return;
  const bool mine = t < a.T;  // a warp's last tokens may be missing: they shadow token T - 1 and write nothing
  const int tr = mine ? t : a.T - 1;
  static_assert(VPL % PER == 0, "whole runs");
  const int E = a.E, k = a.k;
  const ST* row = scores + static_cast<size_t>(tr) * a.ld;
  auto first = [&](int q) { return (q * SUB + sub) * PER; };  // expert of run q
  float x[VPL];
  if (WHOLE) {
#pragma unroll
    for (int q = 0; q < VPL / PER; ++q) {
      float run[PER];
      load_scores<PER, ST>(run, row, first(q), E, a.vec);
#pragma unroll
      for (int i = 0; i < PER; ++i) x[q * PER + i] = run[i];
    }
  }
  int id[SLOTS];
  float g[SLOTS], xs[SLOTS];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    if (q * SUB >= k) break;
    const int j = sub + q * SUB;
    id[q] = j < k ? ids[static_cast<size_t>(tr) * k + j] : -1;
    if (id[q] < 0 || id[q] >= E) id[q] = -1;  // no such expert: no part in the sums, nothing written
    g[q] = j < k ? a.scale * dw[static_cast<size_t>(tr) * k + j] : 0.0f;
    xs[q] = id[q] >= 0 ? clean_score(row[id[q]]) : -INFINITY;
    m = fmaxf(m, xs[q]);
  }

  // r: the weights before the constant (p, or p over its sum); d: factor of what they multiply
  float top = 0.0f, total = 0.0f;
  if (WHOLE) {
    top = sub_max<SUB>(best_of<VPL>(x));
    top = top > -INFINITY ? top : 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = expf(x[i] - top);  // 0 for a masked score
      total += x[i];
    }
    total = sub_sum<SUB>(total);
  } else if (a.renormalise) {
    m = sub_max<SUB>(m);
    top = m > -INFINITY ? m : 0.0f;
  }
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  float r[SLOTS], sum = 0.0f;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    if (q * SUB >= k) break;
    const bool live = xs[q] > -INFINITY;
    r[q] = !live ? 0.0f : softmax ? expf(xs[q] - top) : scaled_sigmoid(xs[q], a.renormalise ? fminf(m, 0.0f) : 0.0f);
    sum += r[q];
  }
  if (a.renormalise) sum = sub_sum<SUB>(sum);
  if (WHOLE) sum = total;
  const float inv = (WHOLE || a.renormalise) ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
  float dot = 0.0f;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    if (q * SUB >= k) break;
    r[q] *= inv;
    dot = fmaf(r[q], g[q], dot);
  }
  dot = WHOLE || a.renormalise ? sub_sum<SUB>(dot) : 0.0f;

  ST* out = dscores + static_cast<size_t>(tr) * ld_d;
  if (mine) {
    const float rest = -dot * inv;
#pragma unroll
    for (int q = 0; q < VPL / PER; ++q) {
      const int e = first(q);
      alignas(16) ST v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = from_f32<ST>(WHOLE ? x[q * PER + i] * rest : 0.0f);
      if (vec_d) {
        if (e < E) *reinterpret_cast<uint4*>(out + e) = *reinterpret_cast<const uint4*>(v);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (e + i < E) out[e + i] = v[i];
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    if (q * SUB >= k) break;
    float d = r[q] * (g[q] - dot);
    if (!softmax) d *= xs[q] > -INFINITY ? sigmoid_f32(-xs[q]) : 0.0f;  // 1 - p without cancellation
    if (mine && id[q] >= 0) out[id[q]] = from_f32<ST>(d);
  }
}

template <int VPL, int SUB, typename ST>
cudaError_t route_ex_of(const ST* scores, RouteArgs a, cudaStream_t s) {
  constexpr int TOKENS = 32 / SUB * router_warps(SUB);  // per block
  constexpr size_t kGroupBytes = TOKENS * (SUB * (VPL + 1) + 32) * sizeof(float);
  static_assert(kGroupBytes + TOKENS * kMaxK * sizeof(int) <= 48 * 1024, "dynamic and static shared memory of a block");
  const size_t smem = a.n_group > 1 ? kGroupBytes : 0;
  a.vec = a.ld % (16 / sizeof(ST)) == 0 && a.E % (16 / sizeof(ST)) == 0 && reinterpret_cast<uintptr_t>(scores) % 16 == 0;
  a.bias_vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  return launch_dependent(route_ex_kernel<VPL, SUB, ST>, dim3((a.T - 1) / TOKENS + 1), dim3(router_warps(SUB) * 32),
                          smem, s, scores, a);
}

template <typename ST>
cudaError_t route_ex_of(const void* scores, const RouteArgs& a, cudaStream_t s) {
  const ST* sc = static_cast<const ST*>(scores);
  int lanes = 2;  // with 16 experts each
  while (lanes * 16 < a.E) lanes *= 2;
  // few rows: a warp each
  if (static_cast<long long>(a.T) * lanes / 32 < kFewWarps) {
    if (a.E <= 32) return route_ex_of<1, 32, ST>(sc, a, s);
    if (a.E <= 64) return route_ex_of<2, 32, ST>(sc, a, s);
    if (a.E <= 128) return route_ex_of<4, 32, ST>(sc, a, s);
    if (a.E <= 256) return route_ex_of<8, 32, ST>(sc, a, s);
    return route_ex_of<16, 32, ST>(sc, a, s);
  }
  switch (lanes) {
    case 2: return route_ex_of<16, 2, ST>(sc, a, s);
    case 4: return route_ex_of<16, 4, ST>(sc, a, s);
    case 8: return route_ex_of<16, 8, ST>(sc, a, s);
    case 16: return route_ex_of<16, 16, ST>(sc, a, s);
    default: return route_ex_of<16, 32, ST>(sc, a, s);
  }
}

template <int VPL, int SUB, typename ST, bool WHOLE>
cudaError_t route_backward_of(const ST* sc, RouteArgs a, const int32_t* ids, const float* dw, ST* ds, long long ld_d,
                              cudaStream_t s) {
  constexpr int TOKENS = 32 / SUB * kRouterWarps;  // per block
  constexpr int PER = 16 / sizeof(ST);
  a.vec = a.ld % PER == 0 && a.E % PER == 0 && reinterpret_cast<uintptr_t>(sc) % 16 == 0;
  const bool vec_d = ld_d % PER == 0 && a.E % PER == 0 && reinterpret_cast<uintptr_t>(ds) % 16 == 0;
  const dim3 grid((a.T - 1) / TOKENS + 1);
  return launch_dependent(route_backward_kernel<VPL, SUB, ST, WHOLE>, grid, dim3(kRouterWarps * 32), 0, s, sc, ids, dw,
                          ds, a, ld_d, vec_d);
}

template <typename ST>
cudaError_t route_backward_of(const void* scores, const RouteArgs& a, const int32_t* ids, const float* dw,
                              void* dscores, long long ld_d, cudaStream_t s) {
  const ST* sc = static_cast<const ST*>(scores);
  ST* ds = static_cast<ST*>(dscores);
  if (a.score_fn == MOE_SCORE_SOFTMAX && !a.renormalise) {
    // 16 experts per lane, 8 lanes at least (a token's slots then take four registers at most)
    if (a.E <= 64) return route_backward_of<8, 8, ST, true>(sc, a, ids, dw, ds, ld_d, s);
    if (a.E <= 128) return route_backward_of<16, 8, ST, true>(sc, a, ids, dw, ds, ld_d, s);
    if (a.E <= 256) return route_backward_of<16, 16, ST, true>(sc, a, ids, dw, ds, ld_d, s);
    return route_backward_of<16, 32, ST, true>(sc, a, ids, dw, ds, ld_d, s);
  }
  // only the selected scores are read, a chain of two loads: many warps
  if (a.E <= 64) return route_backward_of<8, 8, ST, false>(sc, a, ids, dw, ds, ld_d, s);
  if (a.E <= 128) return route_backward_of<8, 16, ST, false>(sc, a, ids, dw, ds, ld_d, s);
  if (a.E <= 256) return route_backward_of<8, 32, ST, false>(sc, a, ids, dw, ds, ld_d, s);
  return route_backward_of<16, 32, ST, false>(sc, a, ids, dw, ds, ld_d, s);
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
