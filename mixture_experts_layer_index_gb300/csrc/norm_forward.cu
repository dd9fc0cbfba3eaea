// The boundary between two blocks (moe_norm_forward):
//   h' = beta h + alpha g * N_post(o),   x' = N_pre(h')
// with N(v) = (v - mu) r w + b, r = 1 / sqrt(mean((v - mu)^2) + eps); mu = 0 for RMS norms.
//
// Bound by memory: h and o are read once, h' and x' written once; 16384 x 2048 bf16
// with two RMS norms take 44 us, 6.1 TB/s (a plain copy reaches 6.7), with two layer norms,
// whose means cost two more sums per row in the way of the loads, 64 us.  8 rows of 4096
// take 3.1 us, the launch and the chain of two sums.  A row stays in
// registers between its two norms, the mean and the second moment about it are
// two sums over registers.  All sums are in fp32, at most 16 values per thread,
// then a tree over the block in a fixed order.
#include "norm.cuh"

namespace moe {
namespace norms {
namespace {

// Blocks per SM: 64 registers for up to 8192 columns (80 for short odd rows, whose loads are
// held in registers).
constexpr int min_blocks(int maxt, bool odd_small) { return odd_small ? 768 / maxt : maxt <= 512 ? 1024 / maxt : 1; }

template <typename HT, typename OT, Access A, int MAXT, bool SMALL>
__global__ void __launch_bounds__(MAXT, min_blocks(MAXT, SMALL && A == PLAIN)) norm_forward_kernel(NormArgs a) {
  constexpr bool RING = A != PLAIN;
  constexpr bool HOLD = MAXT <= 512;  // factors and biases in shared memory
  using Whole = BlockSum<1, MAXT>;
  __shared__ __align__(16) float s_sum[2][1][Whole::W];
  extern __shared__ __align__(16) uint8_t s_ring[];
  const int H = a.H;
  const Own me = SMALL ? Own{static_cast<int>(threadIdx.x) & (a.lanes - 1), a.lanes, a.lanes, a.vec}
                       : Own{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 32, a.vec};
  const unsigned rows = SMALL ? blockDim.x / a.lanes : 1, mine = SMALL ? threadIdx.x / a.lanes : 0;
  const unsigned stride = gridDim.x * rows;
  const float inv_h = 1.0f / static_cast<float>(H);
  const int pitch = slot_pitch(blockDim.x), row_pitch = slot_pitch(me.nt);
  // ring | factors of the post and of the pre norm, then their biases where there are any;
  // each column with its thread
  HT* ring_h = reinterpret_cast<HT*>(s_ring);
  OT* ring_o = reinterpret_cast<OT*>(ring_h + a.depth * pitch);  // depth 0 without a ring
  float* s_post = reinterpret_cast<float*>(ring_o + a.depth * pitch);
  float* s_pre = s_post + row_pitch;
  float* s_bpost = s_pre + row_pitch;
  float* s_bpre = s_bpost + (a.b_post ? row_pitch : 0);
  ring_h += mine * row_pitch;
  ring_o += mine * row_pitch;
  if (!SMALL) {
    for (int i = threadIdx.x; i < 2 * Whole::W; i += blockDim.x) (&s_sum[0][0][0])[i] = 0.0f;
    __syncthreads();
  }
  typename SumOf<SMALL, 1, MAXT>::type row_sum = SumOf<SMALL, 1, MAXT>::make(s_sum, a.lanes);
  dep_wait();
  dep_launch();

  if (RING)
    for (int d = 0; d < a.depth; ++d) {
      clear_slot<HT, A>(ring_h + d * pitch, H, me);
      clear_slot<OT, A>(ring_o + d * pitch, H, me);
    }
  const unsigned T = a.T;  // t may pass 2^31 by the rows ahead
  auto fetch = [&](unsigned t, int slot) {
    if (t < T) {
      copy_in<OT, A>(ring_o + slot * pitch, a.o, static_cast<size_t>(t) * a.ld_o, H, me);
      copy_in<HT, A>(ring_h + slot * pitch, a.h, static_cast<size_t>(t) * a.ld_h, H, me);
    }
    cp_async_commit();
  };
  int slot = 0;
  if (RING)
    for (int d = 0; d + 1 < a.depth; ++d) fetch(blockIdx.x * rows + mine + d * stride, d);

  // factor of the normalised (or plain) o, and of the normalised h'
  const bool gate_c = a.gate_kind == MOE_GATE_CHANNEL, gate_f = a.gate_kind == MOE_GATE_FULL;
  auto post_column = [&](float(&f)[EPT], const void* v, float none, int r) {
    load_columns<A>(f, v, a.w_dtype, r, H, me, none);
    if (gate_c) {
      float g[EPT];
      load_columns<A>(g, a.gate, a.w_dtype, r, H, me, 0.0f);
#pragma unroll
      for (int i = 0; i < EPT; ++i) f[i] *= g[i];
    }
  };
  if (HOLD && mine == 0)
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      float f[EPT];
      post_column(f, a.w_post, 1.0f, r);
      put_shared<A>(s_post, r, me, f);
      load_columns<A>(f, a.w_pre, a.w_dtype, r, H, me, 1.0f);
      put_shared<A>(s_pre, r, me, f);
      if (a.b_post) {
        post_column(f, a.b_post, 0.0f, r);
        put_shared<A>(s_bpost, r, me, f);
      }
      if (a.b_pre) {
        load_columns<A>(f, a.b_pre, a.w_dtype, r, H, me, 0.0f);
        put_shared<A>(s_bpre, r, me, f);
      }
    }
  if (SMALL) __syncthreads();

  for (unsigned t0 = blockIdx.x * rows; t0 < T; t0 += stride) {
    // a group past the last row takes part in the shuffles, with a row of no columns
    const unsigned t = t0 + mine;
    const int H = SMALL && t >= T ? 0 : a.H;
    const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
    F2 v[RUNS][PPT];
    if (RING) {
      const int ahead = slot + a.depth - 1;
      fetch(t + (a.depth - 1) * stride, ahead >= a.depth ? ahead - a.depth : ahead);
      cp_async_wait(a.depth);
    }
    F2 hv[RUNS][PPT];  // without a ring: h's loads go out with o's
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if constexpr (RING) {
        copy_out<OT, A>(v[r], ring_o + slot * pitch, r, me);
      } else {
        load_row<OT, A>(v[r], a.o, at_o, r, H, me);
        load_row<HT, A>(hv[r], a.h, at_h, r, H, me);
      }
    }

    // takes the mean off v (layer norms) and returns 1 / std
    auto moments = [&](int kind) {
      if (kind == MOE_NORM_LAYER) {
        F2 s = f2(0.0f);
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
          for (int i = 0; i < PPT; ++i) s = s + v[r][i];
        float sum[1] = {halves_sum(s)};
        row_sum(sum);
        const F2 mu = f2(-sum[0] * inv_h);
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) v[r][i] = v[r][i] + mu;
          clear_past<A>(v[r], r, H, me);
        }
      }
      F2 q = f2(0.0f);
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < PPT; ++i) q = fma2(v[r][i], v[r][i], q);
      float sum[1] = {halves_sum(q)};
      row_sum(sum);
      return inv_std(sum[0], inv_h, a.eps);
    };

    float scale = a.alpha;
    if (a.gate_kind == MOE_GATE_TOKEN && (!SMALL || t < T)) scale *= __ldg(static_cast<const float*>(a.gate) + t);
    const F2 rs = f2(a.post != MOE_NORM_NONE ? scale * moments(a.post) : scale), beta = f2(a.beta);
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      F2 c[PPT];
      float f[EPT];
      if constexpr (HOLD) {
        copy_out<float, A>(c, s_post, r, me);
      } else {
        post_column(f, a.w_post, 1.0f, r);
        pairs_of(c, f);
      }
#pragma unroll
      for (int i = 0; i < PPT; ++i) v[r][i] = v[r][i] * (rs * c[i]);
      if (a.b_post) {
        if constexpr (HOLD) {
          copy_out<float, A>(c, s_bpost, r, me);
        } else {
          post_column(f, a.b_post, 0.0f, r);
          pairs_of(c, f);
        }
#pragma unroll
        for (int i = 0; i < PPT; ++i) v[r][i] = fma2(f2(scale), c[i], v[r][i]);
      }
      if (gate_f) {
        load_row<OT, A>(c, a.gate, at_o, r, H, me);
#pragma unroll
        for (int i = 0; i < PPT; ++i) v[r][i] = v[r][i] * c[i];
      }
      if constexpr (RING) copy_out<HT, A>(hv[r], ring_h + slot * pitch, r, me);
#pragma unroll
      for (int i = 0; i < PPT; ++i) v[r][i] = fma2(beta, hv[r][i], v[r][i]);
      store_row<HT, A>(a.h_out, at_h, r, H, me, v[r]);
    }
    // x' is taken from h' before its rounding: one rounding each
    if (a.pre != MOE_NORM_NONE) {
      const F2 rp = f2(moments(a.pre));
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        F2 c[PPT];
        float f[EPT];
        if constexpr (HOLD) {
          copy_out<float, A>(c, s_pre, r, me);
        } else {
          load_columns<A>(f, a.w_pre, a.w_dtype, r, H, me, 1.0f);
          pairs_of(c, f);
        }
#pragma unroll
        for (int i = 0; i < PPT; ++i) v[r][i] = v[r][i] * (rp * c[i]);
        if (a.b_pre) {
          if constexpr (HOLD) {
            copy_out<float, A>(c, s_bpre, r, me);
          } else {
            load_columns<A>(f, a.b_pre, a.w_dtype, r, H, me, 0.0f);
            pairs_of(c, f);
          }
#pragma unroll
          for (int i = 0; i < PPT; ++i) v[r][i] = v[r][i] + c[i];
        }
        store_row<OT, A>(a.x_out, at_o, r, H, me, v[r]);
      }
    }
    if (++slot >= a.depth) slot = 0;
  }
}

template <typename HT, typename OT, Access A, int MAXT, bool SMALL = false>
cudaError_t forward_of(NormArgs a, int threads, cudaStream_t s) {
  constexpr size_t kSmemMax = 224 * 1024;
  // 64 registers a thread; at most 32 blocks on an SM
  int per_sm = min_blocks(MAXT, SMALL && A == PLAIN) * MAXT / threads;
  if (per_sm > 32) per_sm = 32;
  size_t smem = 0;
  a.depth = 0;
  if (MAXT <= 512) {
    static const cudaError_t attr =
        cudaFuncSetAttribute(norm_forward_kernel<HT, OT, A, MAXT, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemMax));
    if (attr != cudaSuccess) return attr;
    const size_t pitch = slot_pitch(threads), row = pitch * (sizeof(HT) + sizeof(OT));
    const size_t factors = (2 + (a.b_post ? 1 : 0) + (a.b_pre ? 1 : 0)) * slot_pitch(SMALL ? a.lanes : threads) * sizeof(float);
    // two rows on their way; one, or none, where shared memory has no room for them beside the resident blocks
    if (A != PLAIN)
      a.depth = (3 * row + factors + 2048) * per_sm <= kSmemMax ? 3 : 2 * row + factors <= kSmemMax ? 2 : 1;
    smem = a.depth * row + factors;  // at most 64 KB + 128 KB
    while (per_sm > 1 && (smem + 2048) * per_sm > kSmemMax) --per_sm;
  }
  const int rows = SMALL ? threads / a.lanes : 1;
  const int cap = 152 * per_sm, all = (a.T - 1) / rows + 1;
  return launch_dependent(norm_forward_kernel<HT, OT, A, MAXT, SMALL>, dim3(all < cap ? all : cap), dim3(threads), smem, s, a);
}

template <typename HT, typename OT>
cudaError_t forward_types(NormArgs a, cudaStream_t s) {
  const int threads = norm_threads(a.H);
  if (takes_small(a)) {
    a.lanes = norm_lanes(a.H);
    const int block = small_threads(a.T, a.lanes);
    return a.vec ? forward_of<HT, OT, VEC16, 128, true>(a, block, s) : forward_of<HT, OT, PLAIN, 128, true>(a, block, s);
  }
  if (threads > 512) return forward_of<HT, OT, PLAIN, 1024>(a, threads, s);
  if (a.vec) {
    if (threads <= 128) return forward_of<HT, OT, VEC16, 128>(a, threads, s);
    if (threads <= 256) return forward_of<HT, OT, VEC16, 256>(a, threads, s);
    return forward_of<HT, OT, VEC16, 512>(a, threads, s);
  }
  constexpr Access odd = sizeof(HT) == 4 && sizeof(OT) == 4 ? WORD4 : PLAIN;
  if (threads <= 128) return forward_of<HT, OT, odd, 128>(a, threads, s);
  return forward_of<HT, OT, odd, 512>(a, threads, s);
}

}  // namespace
}  // namespace norms

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  using namespace norms;
  stage_begin("norm_forward", s);
  cudaError_t err;
  if (a.h_dtype == MOE_DTYPE_F32)
    err = a.o_dtype == MOE_DTYPE_F32    ? forward_types<float, float>(a, s)
          : a.o_dtype == MOE_DTYPE_BF16 ? forward_types<float, __nv_bfloat16>(a, s)
                                        : forward_types<float, __half>(a, s);
  else
    err = a.h_dtype == MOE_DTYPE_BF16 ? forward_types<__nv_bfloat16, __nv_bfloat16>(a, s)
                                      : forward_types<__half, __half>(a, s);
  stage_end(s);
  return err;
}

}  // namespace moe
