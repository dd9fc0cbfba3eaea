// Gradient of the block norms (moe_norm_backward).  With u = (v - mu) r the
// normalised value and dn the gradient of N(v) = u w + b:
//   dv = r (dn w - u mean(dn w u) - mean(dn w)),   dw = sum_t dn u,   db = sum_t dn
// (the last mean for layer norms only).  With G = dh' + dv of the pre norm:
//   dh = beta G,   dn of the post norm = alpha g G,   dg = alpha G N_post(o).
//
// Bound by memory: four rows in, two out.  A row's moments and the means of its
// gradient come from the same sum over the block (the means of RMS norms need no
// second look), so a row takes two block-wide sums, three with a layer norm.
// Column sums stay in shared memory, each column with the thread that owns
// it; a block writes them to the workspace once and a second kernel adds the
// blocks' sums in block order.
#include "norm.cuh"

namespace moe {
namespace norms {
namespace {

// A block's column sums, one vector of `pitch` floats each.
template <Access A>
__device__ __forceinline__ void add_columns(float* acc, int run, int H, bool vec, const float (&v)[EPT]) {
  if (A == VEC16 || (A == PLAIN && vec)) {
    const int c = col_of<A>(run, 0, vec);
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
      const int c = col_of<A>(run, i, vec);
      if (c < H) acc[c] += v[i];
    }
  }
}

template <typename HT, typename OT, Access A, int RUNS, int MAXT>
__global__ void __launch_bounds__(MAXT, 1024 / MAXT) norm_backward_kernel(NormArgs a) {
  __shared__ __align__(16) float s_sum[2][4][32];
  extern __shared__ __align__(16) uint8_t s_mem[];
  static_assert(A == PLAIN || RUNS == 1, "a ring holds one run per thread");
  const int H = a.H;
  const bool vec = A == VEC16 || (A == PLAIN && a.vec);
  const float inv_h = 1.0f / static_cast<float>(H);
  const size_t pitch = static_cast<size_t>((H + EPT - 1) / EPT * EPT);
  const bool pre = a.pre != MOE_NORM_NONE, post = a.post != MOE_NORM_NONE;
  const bool layer_pre = a.pre == MOE_NORM_LAYER, layer_post = a.post == MOE_NORM_LAYER;
  // ring slots: o | dh' | h' | dx', then the column sums
  OT* ring_o = reinterpret_cast<OT*>(s_mem);
  HT* ring_g = reinterpret_cast<HT*>(ring_o + a.depth * pitch);
  HT* ring_h = ring_g + (a.dh_out ? a.depth * pitch : 0);
  OT* ring_x = reinterpret_cast<OT*>(ring_h + (pre ? a.depth * pitch : 0));
  uint8_t* after = reinterpret_cast<uint8_t*>(ring_x + (pre ? a.depth * pitch : 0));
  float* part = a.partials + static_cast<size_t>(blockIdx.x) * a.nacc * pitch;
  float* acc = a.acc_in_smem ? reinterpret_cast<float*>(A == PLAIN ? s_mem : after) : part;

  for (int i = threadIdx.x; i < 256; i += blockDim.x) (&s_sum[0][0][0])[i] = 0.0f;
  __syncthreads();
  BlockSum<4> block_sum{s_sum, 0};
  dep_wait();
  dep_launch();
  for (int j = 0; j < a.nacc; ++j)
#pragma unroll
    for (int r = 0; r < RUNS; ++r)
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int c = col_of<A>(r, i, vec);
        if (c < H) acc[j * pitch + c] = 0.0f;
      }

  auto fetch = [&](int t, int slot) {
    if (t < a.T) {
      const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
      if (pre) {
        copy_in<HT, A>(ring_h + slot * pitch, a.h, at_h, H);
        copy_in<OT, A>(ring_x + slot * pitch, a.dx_out, at_o, H);
      }
      copy_in<OT, A>(ring_o + slot * pitch, a.o, at_o, H);
      if (a.dh_out) copy_in<HT, A>(ring_g + slot * pitch, a.dh_out, at_h, H);
    }
    cp_async_commit();
  };
  int slot = 0;
  if (A != PLAIN)
    for (int d = 0; d + 1 < a.depth; ++d) fetch(blockIdx.x + d * gridDim.x, d);

  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
    if constexpr (A != PLAIN) {
      const int ahead = slot + a.depth - 1;
      fetch(t + (a.depth - 1) * gridDim.x, ahead >= a.depth ? ahead - a.depth : ahead);
      cp_async_wait(a.depth);
    }
    auto get_o = [&](float(&v)[EPT], int r) {
      if constexpr (A != PLAIN) copy_out<OT, A>(v, ring_o + slot * pitch, H);
      else load_row<A>(v, a.o, a.o_dtype, at_o, r, H, vec);
    };
    auto get_g = [&](float(&v)[EPT], int r) {
      if constexpr (A != PLAIN) copy_out<HT, A>(v, ring_g + slot * pitch, H);
      else load_row<A>(v, a.dh_out, a.h_dtype, at_h, r, H, vec);
    };
    auto get_h = [&](float(&v)[EPT], int r) {
      if constexpr (A != PLAIN) copy_out<HT, A>(v, ring_h + slot * pitch, H);
      else load_row<A>(v, a.h, a.h_dtype, at_h, r, H, vec);
    };
    auto get_x = [&](float(&v)[EPT], int r) {
      if constexpr (A != PLAIN) copy_out<OT, A>(v, ring_x + slot * pitch, H);
      else load_row<A>(v, a.dx_out, a.o_dtype, at_o, r, H, vec);
    };
    float hc[RUNS][EPT], oc[RUNS][EPT], dx[RUNS][EPT], G[RUNS][EPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      get_o(oc[r], r);
      if (pre) {
        get_h(hc[r], r);
        get_x(dx[r], r);
      }
      if (a.dh_out) {
        get_g(G[r], r);
      } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) G[r][i] = 0.0f;
      }
    }
    if (layer_pre || layer_post) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          if (layer_pre) s[0] += hc[r][i];
          s[1] += oc[r][i];
        }
      block_sum(s);
      const float mh = s[0] * inv_h, mo = layer_post ? s[1] * inv_h : 0.0f;
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const bool in = col_of<A>(r, i, vec) < H;
          if (layer_pre) hc[r][i] = in ? hc[r][i] - mh : 0.0f;
          oc[r][i] = in ? oc[r][i] - mo : 0.0f;
        }
    }
    // second moments, and the two means of the pre norm's gradient
    float ro = 1.0f;
    if (pre || post) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        if (pre) {
          float w[EPT];
          load_columns<A>(w, a.w_pre, a.w_dtype, r, H, vec, 1.0f);
#pragma unroll
          for (int i = 0; i < EPT; ++i) {
            const float dxw = dx[r][i] * w[i];
            s[0] = fmaf(hc[r][i], hc[r][i], s[0]);
            s[1] = fmaf(dxw, hc[r][i], s[1]);
            s[2] += dxw;
          }
        }
#pragma unroll
        for (int i = 0; i < EPT; ++i) s[3] = fmaf(oc[r][i], oc[r][i], s[3]);
      }
      block_sum(s);
      if (pre) {
        const float rs = inv_std(s[0], inv_h, a.eps);
        const float m1 = s[1] * rs * inv_h;                // mean(dx w u)
        const float m0 = layer_pre ? s[2] * inv_h : 0.0f;  // mean(dx w)
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
          float w[EPT];
          load_columns<A>(w, a.w_pre, a.w_dtype, r, H, vec, 1.0f);
          if (a.acc_db_pre >= 0) add_columns<A>(acc + a.acc_db_pre * pitch, r, H, vec, dx[r]);
#pragma unroll
          for (int i = 0; i < EPT; ++i) {
            const float u = hc[r][i] * rs;
            G[r][i] = fmaf(rs, fmaf(-u, m1, fmaf(dx[r][i], w[i], -m0)), G[r][i]);
            dx[r][i] *= u;
          }
          if (a.acc_dw_pre >= 0) add_columns<A>(acc + a.acc_dw_pre * pitch, r, H, vec, dx[r]);
        }
      }
      if (post) {
        ro = inv_std(s[3], inv_h, a.eps);
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
          for (int i = 0; i < EPT; ++i) oc[r][i] *= ro;  // u of the post norm
      }
    }
    if (a.dh) {
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        float d[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) d[i] = a.beta * G[r][i];
        store_row<A>(a.dh, a.h_dtype, at_h, r, H, vec, d);
      }
    }
    // the block's side: ag = alpha G is the gradient of g N(o); G becomes dn w
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      float w[EPT], dn[EPT], c[EPT];
      load_columns<A>(w, post ? a.w_post : nullptr, a.w_dtype, r, H, vec, 1.0f);
#pragma unroll
      for (int i = 0; i < EPT; ++i) dn[i] = col_of<A>(r, i, vec) < H ? a.alpha * G[r][i] : 0.0f;
      if (a.dgate) {
        load_columns<A>(c, post ? a.b_post : nullptr, a.w_dtype, r, H, vec, 0.0f);
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          c[i] = dn[i] * fmaf(oc[r][i], w[i], c[i]);
          d[2] += c[i];
        }
        if (a.gate_kind == MOE_GATE_CHANNEL) add_columns<A>(acc + a.acc_dgate * pitch, r, H, vec, c);
        else if (a.gate_kind == MOE_GATE_FULL) store_row<A>(a.dgate, a.o_dtype, at_o, r, H, vec, c);
      }
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL) {
        if (a.gate_kind == MOE_GATE_CHANNEL) load_columns<A>(c, a.gate, a.w_dtype, r, H, vec, 0.0f);
        else load_row<A>(c, a.gate, a.o_dtype, at_o, r, H, vec);
#pragma unroll
        for (int i = 0; i < EPT; ++i) dn[i] *= c[i];
      } else if (a.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) dn[i] *= gt;
      }
      if (a.acc_db_post >= 0) add_columns<A>(acc + a.acc_db_post * pitch, r, H, vec, dn);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        c[i] = dn[i] * oc[r][i];
        G[r][i] = dn[i] * w[i];
        d[0] = fmaf(c[i], w[i], d[0]);
        d[1] += G[r][i];
      }
      if (a.acc_dw_post >= 0) add_columns<A>(acc + a.acc_dw_post * pitch, r, H, vec, c);
    }
    const bool token_sum = a.dgate && a.gate_kind == MOE_GATE_TOKEN;
    if (post || token_sum) block_sum(d);
    if (token_sum && threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = d[2];
    if (a.d_o) {
      const float m1 = post ? d[0] * inv_h : 0.0f, m0 = layer_post ? d[1] * inv_h : 0.0f;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) G[r][i] = ro * (fmaf(-oc[r][i], m1, G[r][i]) - m0);
        store_row<A>(a.d_o, a.o_dtype, at_o, r, H, vec, G[r]);
      }
    }
    if (++slot >= a.depth) slot = 0;
  }
  if (a.acc_in_smem) {  // each thread hands over the columns that it summed
    for (int j = 0; j < a.nacc; ++j)
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int c = col_of<A>(r, i, vec);
          if (c < H) part[j * pitch + c] = acc[j * pitch + c];
        }
  }
}

// out[j][c] = sum over the blocks' partials, 32 columns per block; 32 rows of
// threads add every 32nd partial in ascending order and the 32 sums are added in
// order, so the result does not depend on timing.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ partials, int nparts, size_t stride,
                                                           int width, size_t pitch, ColumnOutputs out) {
  __shared__ float s[32][33];
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float* p = partials + blockIdx.y * pitch + c;
  float v = 0.0f;
  if (c < width) {
#pragma unroll 4
    for (int i = threadIdx.y; i < nparts; i += 32) v += p[static_cast<size_t>(i) * stride];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    out.p[blockIdx.y][c] = sum;
  }
}

// At most as many blocks as are resident at 1024 threads per SM of a 152-SM part (a
// pure function of the problem: the workspace holds one set of sums for each).
inline int most_blocks_per_sm(int H) {
  const int n = 1024 / norm_threads(H);
  return n > 8 ? 8 : n;
}

constexpr size_t kSmemMax = 224 * 1024;  // of one block's dynamic shared memory
constexpr size_t kSmemSm = 228 * 1024;   // of an SM; a block takes 1 KB of its own and 1 KB static

template <typename HT, typename OT, Access A, int RUNS, int MAXT>
cudaError_t backward_of(NormArgs& a, int threads, cudaStream_t s) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(norm_backward_kernel<HT, OT, A, RUNS, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemMax));
  if (attr != cudaSuccess) return attr;
  const size_t pitch = static_cast<size_t>((a.H + EPT - 1) / EPT * EPT);
  const size_t sums = a.nacc * pitch * sizeof(float);
  int per_sm = most_blocks_per_sm(a.H);
  size_t ring = 0;
  a.depth = 0;
  if (A != PLAIN) {
    // rows of the ring: two, a third if it costs no block, one if two do not fit
    const size_t row = pitch * (sizeof(OT) + (a.dh_out ? sizeof(HT) : 0) + (a.pre ? sizeof(HT) + sizeof(OT) : 0));
    auto fit = [&](int depth) { return static_cast<int>(kSmemSm / (depth * row + sums + 2048)); };
    a.depth = fit(2) < 1 ? 1 : fit(3) >= (fit(2) < per_sm ? fit(2) : per_sm) ? 3 : 2;
    ring = a.depth * row;
  }
  a.acc_in_smem = ring + sums <= kSmemMax;  // else the sums are kept in the workspace itself
  const size_t smem = ring + (a.acc_in_smem ? sums : 0);
  const int fits = static_cast<int>(kSmemSm / (smem + 2048));
  if (fits < per_sm) per_sm = fits;
  a.blocks = a.T < 152 * per_sm ? a.T : 152 * per_sm;
  return launch_dependent(norm_backward_kernel<HT, OT, A, RUNS, MAXT>, dim3(a.blocks), dim3(threads), smem, s, a);
}

template <typename HT, typename OT, Access A>
cudaError_t backward_ring(NormArgs& a, int threads, cudaStream_t s) {
  if (threads <= 256) return backward_of<HT, OT, A, 1, 256>(a, threads, s);
  if (threads <= 512) return backward_of<HT, OT, A, 1, 512>(a, threads, s);
  return backward_of<HT, OT, A, 1, 1024>(a, threads, s);
}

}  // namespace
}  // namespace norms

size_t norm_partials_bytes(int T, int H) {
  const size_t pitch = static_cast<size_t>((H + norms::EPT - 1) / norms::EPT * norms::EPT);
  const int most = 152 * norms::most_blocks_per_sm(H);
  return static_cast<size_t>(T < most ? T : most) * 5 * pitch * sizeof(float);
}

cudaError_t launch_norm_backward(const NormArgs& args, float* const (&sums)[5], cudaStream_t s) {
  using namespace norms;
  NormArgs a = args;
  // the sums that are wanted, packed: vector j of a block's partials is out.p[j]
  int* slot[5] = {&a.acc_dw_post, &a.acc_db_post, &a.acc_dw_pre, &a.acc_db_pre, &a.acc_dgate};
  ColumnOutputs out{};
  a.nacc = 0;
  for (int j = 0; j < 5; ++j) {
    *slot[j] = sums[j] ? a.nacc : -1;
    if (sums[j]) out.p[a.nacc++] = sums[j];
  }
  const int threads = norm_threads(a.H);
  const int pair = a.h_dtype * 3 + a.o_dtype;
  stage_begin("norm_backward", s);
  cudaError_t err;
  if (a.H > threads * EPT) {
    err = backward_of<float, float, PLAIN, 2, 1024>(a, threads, s);
  } else if (a.vec) {
    switch (pair) {
      case MOE_DTYPE_F32 * 3 + MOE_DTYPE_F32: err = backward_ring<float, float, VEC16>(a, threads, s); break;
      case MOE_DTYPE_F32 * 3 + MOE_DTYPE_BF16: err = backward_ring<float, __nv_bfloat16, VEC16>(a, threads, s); break;
      case MOE_DTYPE_F32 * 3 + MOE_DTYPE_F16: err = backward_ring<float, __half, VEC16>(a, threads, s); break;
      case MOE_DTYPE_BF16 * 3 + MOE_DTYPE_BF16:
        err = backward_ring<__nv_bfloat16, __nv_bfloat16, VEC16>(a, threads, s);
        break;
      default: err = backward_ring<__half, __half, VEC16>(a, threads, s);
    }
  } else if (pair == MOE_DTYPE_F32 * 3 + MOE_DTYPE_F32) {
    err = backward_ring<float, float, WORD4>(a, threads, s);
  } else if (threads <= 512) {
    err = backward_of<float, float, PLAIN, 1, 512>(a, threads, s);
  } else {
    err = backward_of<float, float, PLAIN, 1, 1024>(a, threads, s);
  }
  stage_end(s);
  if (err == cudaSuccess && a.nacc > 0) {
    const size_t pitch = static_cast<size_t>((a.H + EPT - 1) / EPT * EPT);
    err = launch_column_sums(a.partials, a.blocks, a.nacc * pitch, a.nacc, a.H, pitch, out, s);
  }
  return err;
}

cudaError_t launch_column_sums(const float* partials, int nparts, size_t stride, int nsums, int width, size_t pitch,
                               const ColumnOutputs& out, cudaStream_t s) {
  stage_begin("column_sums", s);
  const cudaError_t err = launch_dependent(norms::column_sums_kernel, dim3((width + 31) / 32, nsums), dim3(32, 32), 0, s,
                                           partials, nparts, stride, width, pitch, out);
  stage_end(s);
  return err;
}

}  // namespace moe
