// Gradient of the block norms (moe_norm_backward).  With u = (v - mu) r the
// normalised value and dn the gradient of N(v) = u w + b:
//   dv = r (dn w - u mean(dn w u) - mean(dn w)),   dw = sum_t dn u,   db = sum_t dn
// (the last mean for layer norms only).  With G = dh' + dv of the pre norm:
//   dh = beta G,   dn of the post norm = alpha g G,   dg = alpha G N_post(o).
//
// Bound by memory: four rows in, two out; 16384 x 2048 bf16 with RMS norms and a gate per
// column take 67.6 us, 5.95 TB/s (a plain copy reaches 6.7) at 60 % of the issue slots.  With
// layer norms 101 us: a third sum per row and the sums for the biases, whose
// registers leave three blocks of 128 threads per SM instead of four.  Odd rows are
// bound by instructions (an element at a time), see Access in norm.cuh.
// A row's moments and the means of its
// gradient come from the same sum over the block (the means of RMS norms need no
// second look), so a row takes two block-wide sums, three with a layer norm.
// Column sums stay with the thread that owns the column, in registers up to
// 8192 columns, else in shared memory; a block writes them to the workspace once
// and a second kernel adds the blocks' sums in a fixed order.
#include "norm.cuh"

namespace moe {
namespace norms {
namespace {

// A block's column sums, one vector of `pitch` floats each.
template <Access A>
__device__ __forceinline__ void add_columns(float* acc, int run, int H, const Own& me, const F2 (&p2)[PPT]) {
  float v[EPT];
  values_of(v, p2);
  if (in_runs<A>(me)) {
    const int c = col_of<A>(run, 0, me);
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
      const int c = col_of<A>(run, i, me);
      if (c < H) acc[c] += v[i];
    }
  }
}

__host__ __device__ inline bool bias_in_smem(const NormArgs& a) {
  return a.b_post && a.dgate && a.gate_kind != MOE_GATE_CHANNEL;
}

// Sums over tokens, per column: post1 = sum alpha G' u, post0 = sum alpha G', with G'
// = G for a per-column gate g (then dw = g post1, db = g post0, dg = w post1 + b post0)
// and G' = g G otherwise (dw = post1, db = post0); pre1 = sum dx u, pre0 = sum dx.
// GENERAL: layer norms, post0 or pre0, a gate per token or value; otherwise RMS norms with
// at most a per-column gate, which need fewer registers (a resident block more) and
// instructions.
constexpr int min_blocks(int maxt, bool general) {
  return maxt <= 128 ? (general ? 3 : 4) : maxt <= 256 && !general ? 2 : 1;
}

template <typename HT, typename OT, Access A, int MAXT, bool GENERAL, bool SMALL>
__global__ void __launch_bounds__(MAXT, min_blocks(MAXT, GENERAL)) norm_backward_kernel(NormArgs a) {
  constexpr bool RING = A != PLAIN;
  constexpr bool HOLD = MAXT <= 512;  // column sums in registers, factors in shared memory
  using Whole = BlockSum<4, MAXT>;
  __shared__ __align__(16) float s_sum[2][4][Whole::W];
  extern __shared__ __align__(16) uint8_t s_mem[];
  const int H = a.H;
  const Own me = SMALL ? Own{static_cast<int>(threadIdx.x) & (a.lanes - 1), a.lanes, a.lanes, a.vec}
                       : Own{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 32, a.vec};
  const unsigned rows = SMALL ? blockDim.x / a.lanes : 1, mine = SMALL ? threadIdx.x / a.lanes : 0;
  const unsigned stride = gridDim.x * rows;
  const float inv_h = 1.0f / static_cast<float>(H);
  const int pitch = slot_pitch(blockDim.x), row_pitch = slot_pitch(me.nt), sums_pitch = (H + EPT - 1) / EPT * EPT;
  const bool pre = a.pre != MOE_NORM_NONE, post = a.post != MOE_NORM_NONE;
  const bool layer_pre = a.pre == MOE_NORM_LAYER, layer_post = a.post == MOE_NORM_LAYER;
  const bool gate_c = a.gate_kind == MOE_GATE_CHANNEL, gate_f = a.gate_kind == MOE_GATE_FULL;
  const bool gate_t = a.gate_kind == MOE_GATE_TOKEN;
  // ring slots: o | dh' | h' | dx', then the factors of the post and of the pre norm; rows
  // of over 8192 columns: the column sums (in the workspace itself where they do not fit)
  const int my_row = mine * row_pitch;
  const int slot_h = slot_elements<HT, A>(pitch), slot_o = slot_elements<OT, A>(pitch);
  OT* ring_o = reinterpret_cast<OT*>(s_mem);
  HT* ring_g = reinterpret_cast<HT*>(ring_o + a.depth * slot_o);
  HT* ring_h = ring_g + (a.dh_out ? a.depth * slot_h : 0);
  OT* ring_x = reinterpret_cast<OT*>(ring_h + (pre ? a.depth * slot_h : 0));
  float* s_post = reinterpret_cast<float*>(ring_x + (pre ? a.depth * slot_o : 0));
  if (A == SHIFT) {
    for (uint4* p = reinterpret_cast<uint4*>(s_mem) + threadIdx.x; p < reinterpret_cast<uint4*>(s_post); p += blockDim.x)
      *p = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  ring_o += my_row;
  ring_g += my_row;
  ring_h += my_row;
  ring_x += my_row;
  float* s_pre = s_post + row_pitch;
  float* s_bias = s_pre + row_pitch;  // post norm's bias, for the gradient of a gate per token or value
  float* part = a.partials + static_cast<size_t>(blockIdx.x) * a.nacc * sums_pitch;
  float* acc = a.acc_in_smem ? reinterpret_cast<float*>(s_mem) : part;

  if (!SMALL) {
    for (int i = threadIdx.x; i < 8 * Whole::W; i += blockDim.x) (&s_sum[0][0][0])[i] = 0.0f;
    __syncthreads();
  }
  typename SumOf<SMALL, 4, MAXT>::type row_sum = SumOf<SMALL, 4, MAXT>::make(s_sum, a.lanes);
  dep_wait();
  dep_launch();

  if (RING)
    for (int d = 0; d < a.depth; ++d) {
      clear_slot<OT, A>(ring_o + d * slot_o, H, me);
      if (a.dh_out) clear_slot<HT, A>(ring_g + d * slot_h, H, me);
      if (pre) {
        clear_slot<HT, A>(ring_h + d * slot_h, H, me);
        clear_slot<OT, A>(ring_x + d * slot_o, H, me);
      }
    }
  HT edge_h = {}, edge_g = {};
  OT edge_o = {}, edge_x = {};
  const unsigned T = a.T;  // t may pass 2^31 by the rows ahead
  auto fetch = [&](unsigned t, int slot) {
    if (t < T) {
      const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
      if constexpr (A == SHIFT) {
        if (pre) {
          start_row<HT, A>(ring_h + slot * slot_h, edge_h, a.h, at_h, H);
          start_row<OT, A>(ring_x + slot * slot_o, edge_x, a.dx_out, at_o, H);
        }
        start_row<OT, A>(ring_o + slot * slot_o, edge_o, a.o, at_o, H);
        if (a.dh_out) start_row<HT, A>(ring_g + slot * slot_h, edge_g, a.dh_out, at_h, H);
      } else {
        if (pre) {
          copy_in<HT, A>(ring_h + slot * slot_h, a.h, at_h, H, me);
          copy_in<OT, A>(ring_x + slot * slot_o, a.dx_out, at_o, H, me);
        }
        copy_in<OT, A>(ring_o + slot * slot_o, a.o, at_o, H, me);
        if (a.dh_out) copy_in<HT, A>(ring_g + slot * slot_h, a.dh_out, at_h, H, me);
      }
    }
    cp_async_commit();
  };
  int slot = 0;
  if (RING)
    for (int d = 0; d + 1 < a.depth; ++d) fetch(blockIdx.x * rows + mine + d * stride, d);

  // factors of dn: the pre norm's weight; the post norm's, with a per-column gate
  auto post_factor = [&](float(&f)[EPT], int r) {
    load_columns<A>(f, a.w_post, a.w_dtype, r, H, me, 1.0f);
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
      post_factor(f, r);
      put_shared<A>(s_post, r, me, f);
      load_columns<A>(f, a.w_pre, a.w_dtype, r, H, me, 1.0f);
      put_shared<A>(s_pre, r, me, f);
      if (bias_in_smem(a)) {
        load_columns<A>(f, a.b_post, a.w_dtype, r, H, me, 0.0f);
        put_shared<A>(s_bias, r, me, f);
      }
    }
  if (SMALL) __syncthreads();
  auto factor = [&](F2(&f)[PPT], bool of_post, int r) {
    if constexpr (HOLD) {
      copy_out<float, A>(f, of_post ? s_post : s_pre, r, me);
    } else {
      float v[EPT];
      if (of_post) post_factor(v, r);
      else load_columns<A>(v, a.w_pre, a.w_dtype, r, H, me, 1.0f);
      pairs_of(f, v);
    }
  };
  F2 post1[RUNS][PPT], post0[RUNS][PPT], pre1[RUNS][PPT], pre0[RUNS][PPT];  // HOLD
#pragma unroll
  for (int r = 0; r < RUNS; ++r)
#pragma unroll
    for (int i = 0; i < PPT; ++i) post1[r][i] = post0[r][i] = pre1[r][i] = pre0[r][i] = f2(0.0f);
  if (!HOLD)
    for (int j = 0; j < a.nacc; ++j)
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int c = col_of<A>(r, i, me);
          if (c < H) acc[j * sums_pitch + c] = 0.0f;
        }

  for (unsigned t0 = blockIdx.x * rows; t0 < T; t0 += stride) {
    // a group past the last row takes part in the shuffles, with a row of zeros and no columns
    const unsigned t = t0 + mine;
    const bool live = !SMALL || t < T;
    const int H = live ? a.H : 0;
    const size_t at_h = static_cast<size_t>(t) * a.ld_h, at_o = static_cast<size_t>(t) * a.ld_o;
    const int ahead = slot + a.depth - 1;
    if constexpr (A == SHIFT) {
      // one row ahead, or none where shared memory holds only one
      if (a.depth == 1) {
        __syncthreads();
        fetch(t, 0);
      }
      cp_async_wait(1);
      if (pre) {
        finish_row<HT, A>(ring_h + slot * slot_h, edge_h, a.h, at_h, H);
        finish_row<OT, A>(ring_x + slot * slot_o, edge_x, a.dx_out, at_o, H);
      }
      finish_row<OT, A>(ring_o + slot * slot_o, edge_o, a.o, at_o, H);
      if (a.dh_out) finish_row<HT, A>(ring_g + slot * slot_h, edge_g, a.dh_out, at_h, H);
      __syncthreads();  // this row is there, and all are done with the last one
      if (a.depth == 2) fetch(t + stride, slot ^ 1);
    } else if (RING) {
      fetch(t + (a.depth - 1) * stride, ahead >= a.depth ? ahead - a.depth : ahead);
      cp_async_wait(a.depth);
    }
    const OT* in_o = ring_o + slot * slot_o + shift_of<OT, A>(a.o, at_o);
    const OT* in_x = ring_x + slot * slot_o + shift_of<OT, A>(a.dx_out, at_o);
    const HT* in_h = ring_h + slot * slot_h + shift_of<HT, A>(a.h, at_h);
    const HT* in_g = ring_g + slot * slot_h + shift_of<HT, A>(a.dh_out, at_h);
    F2 hc[RUNS][PPT], oc[RUNS][PPT], dx[RUNS][PPT], G[RUNS][PPT];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if constexpr (RING) copy_out<OT, A>(oc[r], in_o, r, me);
      else load_row<OT, A>(oc[r], a.o, at_o, r, H, me);
      if (pre) {
        if constexpr (RING) {
          copy_out<HT, A>(hc[r], in_h, r, me);
          copy_out<OT, A>(dx[r], in_x, r, me);
        } else {
          load_row<HT, A>(hc[r], a.h, at_h, r, H, me);
          load_row<OT, A>(dx[r], a.dx_out, at_o, r, H, me);
        }
      }
      if constexpr (!RING)
        if (a.dh_out) load_row<HT, A>(G[r], a.dh_out, at_h, r, H, me);
      if (SMALL && !live)
#pragma unroll
        for (int i = 0; i < PPT; ++i) hc[r][i] = oc[r][i] = dx[r][i] = f2(0.0f);
    }
    if (GENERAL && (layer_pre || layer_post)) {
      F2 sh = f2(0.0f), so = f2(0.0f);
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
          if (layer_pre) sh = sh + hc[r][i];
          so = so + oc[r][i];
        }
      float s[4] = {halves_sum(sh), halves_sum(so), 0.0f, 0.0f};
      row_sum(s);
      const F2 mh = f2(-s[0] * inv_h), mo = f2(-s[1] * inv_h);
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        if (layer_pre) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) hc[r][i] = hc[r][i] + mh;
          clear_past<A>(hc[r], r, H, me);
        }
        if (layer_post) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) oc[r][i] = oc[r][i] + mo;
          clear_past<A>(oc[r], r, H, me);
        }
      }
    }
    // second moments, and the two means of the pre norm's gradient
    float ro = 1.0f, rs = 0.0f, m1 = 0.0f, m0 = 0.0f;
    if (pre || post) {
      F2 q0 = f2(0.0f), q1 = q0, q2 = q0, q3 = q0;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        if (pre) {
          F2 f[PPT];
          factor(f, false, r);
#pragma unroll
          for (int i = 0; i < PPT; ++i) {
            const F2 dxw = dx[r][i] * f[i];
            q0 = fma2(hc[r][i], hc[r][i], q0);
            q1 = fma2(dxw, hc[r][i], q1);
            if (GENERAL) q2 = q2 + dxw;
          }
        }
#pragma unroll
        for (int i = 0; i < PPT; ++i) q3 = fma2(oc[r][i], oc[r][i], q3);
      }
      float s[4] = {halves_sum(q0), halves_sum(q1), GENERAL ? halves_sum(q2) : 0.0f, halves_sum(q3)};
      row_sum(s);
      if (post && live) ro = inv_std(s[3], inv_h, a.eps);
      if (pre && live) {
        rs = inv_std(s[0], inv_h, a.eps);
        m1 = s[1] * rs * inv_h;                 // mean(dx w u)
        m0 = layer_pre ? s[2] * inv_h : 0.0f;   // mean(dx w)
      }
    }
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if (!a.dh_out || !live) {
#pragma unroll
        for (int i = 0; i < PPT; ++i) G[r][i] = f2(0.0f);
      } else if constexpr (RING) {
        copy_out<HT, A>(G[r], in_g, r, me);
      }
      if (pre) {
        F2 f[PPT];
        factor(f, false, r);
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
          const F2 u = hc[r][i] * f2(rs);
          F2 d = dx[r][i] * f[i];
          if (GENERAL) d = d + f2(-m0);
          G[r][i] = fma2(f2(rs), fma2(u, f2(-m1), d), G[r][i]);
          hc[r][i] = u;
        }
        if (GENERAL) clear_past<A>(G[r], r, H, me);
        if (HOLD) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) pre1[r][i] = fma2(dx[r][i], hc[r][i], pre1[r][i]);
          if (GENERAL)
#pragma unroll
            for (int i = 0; i < PPT; ++i) pre0[r][i] = pre0[r][i] + dx[r][i];
        } else {
          if (a.acc_pre0 >= 0) add_columns<A>(acc + a.acc_pre0 * sums_pitch, r, H, me, dx[r]);
          if (a.acc_pre1 >= 0) {
#pragma unroll
            for (int i = 0; i < PPT; ++i) dx[r][i] = dx[r][i] * hc[r][i];
            add_columns<A>(acc + a.acc_pre1 * sums_pitch, r, H, me, dx[r]);
          }
        }
      }
      if (a.dh) {
        F2 d[PPT];
#pragma unroll
        for (int i = 0; i < PPT; ++i) d[i] = f2(a.beta) * G[r][i];
        store_row<HT, A>(a.dh, at_h, r, H, me, d);
      }
    }
    // the block's side: alpha G is the gradient of g N(o); G becomes dn w
    const float gt = gate_t && live ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
    F2 d0 = f2(0.0f), d1 = d0, d2 = d0;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      F2 c[PPT];
#pragma unroll
      for (int i = 0; i < PPT; ++i) {
        G[r][i] = G[r][i] * f2(a.alpha);
        oc[r][i] = oc[r][i] * f2(ro);  // u of the post norm, or o itself
      }
      if (GENERAL && a.dgate && !gate_c) {  // gradient of a gate per token or value: alpha G N(o)
        F2 w[PPT];
        factor(w, true, r);
#pragma unroll
        for (int i = 0; i < PPT; ++i) w[i] = w[i] * oc[r][i];
        if (a.b_post) {
          if constexpr (HOLD) {
            copy_out<float, A>(c, s_bias, r, me);
          } else {
            float v[EPT];
            load_columns<A>(v, a.b_post, a.w_dtype, r, H, me, 0.0f);
            pairs_of(c, v);
          }
#pragma unroll
          for (int i = 0; i < PPT; ++i) w[i] = w[i] + c[i];
        }
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
          c[i] = G[r][i] * w[i];
          d2 = d2 + c[i];
        }
        if (gate_f) store_row<OT, A>(a.dgate, at_o, r, H, me, c);
      }
      if (GENERAL && gate_f) {
        load_row<OT, A>(c, a.gate, at_o, r, H, me);
#pragma unroll
        for (int i = 0; i < PPT; ++i) G[r][i] = G[r][i] * c[i];
      } else if (GENERAL && gate_t) {
#pragma unroll
        for (int i = 0; i < PPT; ++i) G[r][i] = G[r][i] * f2(gt);
      }
      if (HOLD) {
#pragma unroll
        for (int i = 0; i < PPT; ++i) post1[r][i] = fma2(G[r][i], oc[r][i], post1[r][i]);
        if (GENERAL)
#pragma unroll
          for (int i = 0; i < PPT; ++i) post0[r][i] = post0[r][i] + G[r][i];
      } else {
        if (a.acc_post0 >= 0) add_columns<A>(acc + a.acc_post0 * sums_pitch, r, H, me, G[r]);
        if (a.acc_post1 >= 0) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) c[i] = G[r][i] * oc[r][i];
          add_columns<A>(acc + a.acc_post1 * sums_pitch, r, H, me, c);
        }
      }
      factor(c, true, r);
#pragma unroll
      for (int i = 0; i < PPT; ++i) {
        G[r][i] = G[r][i] * c[i];
        d0 = fma2(G[r][i], oc[r][i], d0);
        if (GENERAL) d1 = d1 + G[r][i];
      }
    }
    const bool token_sum = GENERAL && a.dgate && gate_t;
    float d[4] = {halves_sum(d0), GENERAL ? halves_sum(d1) : 0.0f, GENERAL ? halves_sum(d2) : 0.0f, 0.0f};
    if (post || token_sum) row_sum(d);
    if (token_sum && live && me.tid == 0) static_cast<float*>(a.dgate)[t] = d[2];
    if (a.d_o) {
      const F2 n1 = f2(-d[0] * inv_h), n0 = f2(layer_post ? -d[1] * inv_h : 0.0f);
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        if (post) {
#pragma unroll
          for (int i = 0; i < PPT; ++i) {
            F2 v = fma2(oc[r][i], n1, G[r][i]);
            if (GENERAL) v = v + n0;
            G[r][i] = f2(ro) * v;
          }
        }
        store_row<OT, A>(a.d_o, at_o, r, H, me, G[r]);
      }
    }
    if (++slot >= a.depth) slot = 0;
  }
  // each thread hands over the columns that it summed; groups of lanes add theirs up first
  if (HOLD) {
    const bool join = SMALL && rows > 1;
    float* all = reinterpret_cast<float*>(s_mem);
    if (join) {
      cp_async_wait(1);
      __syncthreads();  // all have read their last rows and factors
    }
    auto hand_over = [&](int j, F2(&sum)[RUNS][PPT]) {
      if (j < 0) return;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        float v[EPT];
        values_of(v, sum[r]);
        if (join) put_shared<A>(all + j * pitch + my_row, r, me, v);
        else store_row<float, A>(part + j * sums_pitch, 0, r, H, me, v);
      }
    };
    hand_over(a.acc_post1, post1);
    hand_over(a.acc_post0, post0);
    hand_over(a.acc_pre1, pre1);
    hand_over(a.acc_pre0, pre0);
    if (join) {
      __syncthreads();
      const int quads = sums_pitch / 4;
      for (int i = threadIdx.x; i < a.nacc * quads; i += blockDim.x) {
        const int j = i / quads, c = (i - j * quads) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (unsigned q = 0; q < rows; ++q) {
          const float4 x = *reinterpret_cast<const float4*>(all + j * pitch + q * row_pitch + c);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        *reinterpret_cast<float4*>(part + j * sums_pitch + c) = v;
      }
    }
  } else if (a.acc_in_smem) {
    for (int j = 0; j < a.nacc; ++j)
#pragma unroll
      for (int r = 0; r < RUNS; ++r)
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int c = col_of<A>(r, i, me);
          if (c < H) part[j * sums_pitch + c] = acc[j * sums_pitch + c];
        }
  }
}

// out[c] = sum over the blocks' partials, 32 columns per block; 32 rows of threads add
// every 32nd partial in ascending order and the 32 sums are added in order, so the
// result does not depend on timing.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ partials, int nparts, int width,
                                                           float* __restrict__ out) {
  __shared__ float s[32][33];
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < width) {
#pragma unroll 4
    for (int i = threadIdx.y; i < nparts; i += 32) v += partials[static_cast<size_t>(i) * width + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    out[c] = sum;
  }
}

// The same for the sums of the norms' gradient, one per row of blocks, with the factors of
// the outputs that they go into.
__global__ void __launch_bounds__(1024) norm_sums_kernel(NormArgs a, NormSums out) {
  __shared__ float s[32][33];
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 32 + threadIdx.x;
  const size_t pitch = (a.H + EPT - 1) / EPT * EPT;
  auto total = [&](int j) {
    float v = 0.0f;
    if (c < a.H) {
      const float* p = a.partials + j * pitch + c;
      const size_t stride = a.nacc * pitch;
      constexpr int AHEAD = 10;  // loads on their way: one or two batches for all blocks
      for (int i = threadIdx.y; i < a.blocks; i += 32 * AHEAD) {
        float u[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) u[q] = i + 32 * q < a.blocks ? p[(i + 32 * q) * stride] : 0.0f;
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) v += u[q];
      }
    }
    __syncthreads();
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    float sum = 0.0f;
    if (threadIdx.y == 0)
#pragma unroll
      for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    return sum;
  };
  const int j = blockIdx.y;
  const float sum = total(j);
  const float other = j == a.acc_post1 && out.dgate && a.acc_post0 >= 0 ? total(a.acc_post0) : 0.0f;
  if (threadIdx.y != 0 || c >= a.H) return;
  auto value = [&](const void* v, float none) { return v ? load_one(v, a.w_dtype, c) : none; };
  const float g = a.gate_kind == MOE_GATE_CHANNEL ? load_one(a.gate, a.w_dtype, c) : 1.0f;
  if (j == a.acc_post1) {
    if (out.dw_post) out.dw_post[c] = g * sum;
    if (out.dgate) out.dgate[c] = value(a.w_post, 1.0f) * sum + value(a.b_post, 0.0f) * other;
  }
  if (j == a.acc_post0 && out.db_post) out.db_post[c] = g * sum;
  if (j == a.acc_pre1) out.dw_pre[c] = sum;
  if (j == a.acc_pre0) out.db_pre[c] = sum;
}

// At most as many blocks as the registers of a 152-SM part hold (a pure function of
// the problem: the workspace has room for the sums of each).
inline int most_blocks_per_sm(int H) {
  const int n = 512 / norm_threads(H);
  return n > 16 ? 16 : n < 1 ? 1 : n;
}

constexpr size_t kSmemMax = 226 * 1024;  // of one block's dynamic shared memory, beside up to 1 KB static
constexpr size_t kSmemSm = 228 * 1024;   // of an SM; a block takes 1 KB of its own and 1 KB static

template <typename HT, typename OT, Access A, int MAXT, bool GENERAL, bool SMALL = false>
cudaError_t backward_of(NormArgs& a, int threads, cudaStream_t s) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(norm_backward_kernel<HT, OT, A, MAXT, GENERAL, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemMax));
  if (attr != cudaSuccess) return attr;
  const size_t pitch = slot_pitch(threads);
  int per_sm = min_blocks(MAXT, GENERAL) * MAXT / threads;
  if (per_sm > most_blocks_per_sm(a.H)) per_sm = most_blocks_per_sm(a.H);
  size_t smem = 0;
  a.depth = 0;
  auto fits = [&](size_t bytes, int blocks) { return bytes <= kSmemMax && (bytes + 2048) * blocks <= kSmemSm; };
  if (MAXT <= 512) {
    const size_t factors = (bias_in_smem(a) ? 3 : 2) * slot_pitch(SMALL ? a.lanes : threads) * sizeof(float);
    if (A != PLAIN) {
      // a row that is worked on and, where they fit with the resident blocks, one or two
      // on their way; 128 KB at most for one row, beside 96 KB of factors
      const size_t row_o = slot_elements<OT, A>(pitch) * sizeof(OT), row_h = slot_elements<HT, A>(pitch) * sizeof(HT);
      const size_t row = row_o + (a.dh_out ? row_h : 0) + (a.pre ? row_h + row_o : 0);
      a.depth = A == SHIFT ? 2 : 3;
      while (a.depth > 1 && !fits(a.depth * row + factors, A == SHIFT ? 1 : per_sm)) --a.depth;
      smem = a.depth * row;
    }
    smem += factors;
    const size_t sums = a.nacc * pitch * sizeof(float);  // of the groups
    if (SMALL && smem < sums) smem = sums;
  } else {
    smem = a.nacc * norm_pitch(a.H) * sizeof(float);
    a.acc_in_smem = smem <= kSmemMax;  // else the sums are kept in the workspace itself
    if (!a.acc_in_smem) smem = 0;
  }
  while (per_sm > 1 && !fits(smem, per_sm)) --per_sm;
  const int all = (a.T - 1) / (SMALL ? threads / a.lanes : 1) + 1;
  a.blocks = all < 152 * per_sm ? all : 152 * per_sm;
  return launch_dependent(norm_backward_kernel<HT, OT, A, MAXT, GENERAL, SMALL>, dim3(a.blocks), dim3(threads), smem, s, a);
}

template <typename HT, typename OT>
cudaError_t backward_types(NormArgs& a, cudaStream_t s) {
  const int threads = norm_threads(a.H);
  if (threads > 512) return backward_of<HT, OT, PLAIN, 1024, true>(a, threads, s);
  const bool general = a.acc_post0 >= 0 || a.acc_pre0 >= 0 || a.post == MOE_NORM_LAYER || a.pre == MOE_NORM_LAYER ||
                       a.gate_kind == MOE_GATE_TOKEN || a.gate_kind == MOE_GATE_FULL;
  if (takes_small(a)) {
    // few rows: one per warp, so that no block has rows' sums to join (300 x 256: 6.8 -> 6.1 us)
    a.lanes = a.T <= 2 * 152 ? 32 : norm_lanes(a.H);
    const int block = small_threads(a.T, a.lanes);
    if (!a.vec) return backward_of<HT, OT, PLAIN, 128, true, true>(a, block, s);
    return general ? backward_of<HT, OT, VEC16, 128, true, true>(a, block, s)
                   : backward_of<HT, OT, VEC16, 128, false, true>(a, block, s);
  }
  if (a.vec) {
    if (general) {
      if (threads <= 128) return backward_of<HT, OT, VEC16, 128, true>(a, threads, s);
      if (threads <= 256) return backward_of<HT, OT, VEC16, 256, true>(a, threads, s);
      return backward_of<HT, OT, VEC16, 512, true>(a, threads, s);
    }
    if (threads <= 128) return backward_of<HT, OT, VEC16, 128, false>(a, threads, s);
    if (threads <= 256) return backward_of<HT, OT, VEC16, 256, false>(a, threads, s);
    return backward_of<HT, OT, VEC16, 512, false>(a, threads, s);
  }
  constexpr Access odd = sizeof(HT) == 4 && sizeof(OT) == 4 ? WORD4 : SHIFT;
  if (general) {
    if (threads <= 128) return backward_of<HT, OT, odd, 128, true>(a, threads, s);
    return backward_of<HT, OT, odd, 512, true>(a, threads, s);
  }
  if (threads <= 128) return backward_of<HT, OT, odd, 128, false>(a, threads, s);
  return backward_of<HT, OT, odd, 512, false>(a, threads, s);
}

}  // namespace
}  // namespace norms

size_t norm_partials_bytes(int T, int H) {
  const int most = 152 * norms::most_blocks_per_sm(H);
  return static_cast<size_t>(T < most ? T : most) * 4 * norms::norm_pitch(H) * sizeof(float);
}

cudaError_t launch_norm_backward(const NormArgs& args, const NormSums& out, cudaStream_t s) {
  using namespace norms;
  NormArgs a = args;
  a.nacc = 0;
  auto want = [&](bool yes) { return yes ? a.nacc++ : -1; };
  a.acc_post1 = want(out.dw_post || out.dgate);
  a.acc_post0 = want(out.db_post || (out.dgate && a.b_post));
  a.acc_pre1 = want(out.dw_pre);
  a.acc_pre0 = want(out.db_pre);
  stage_begin("norm_backward", s);
  cudaError_t err;
  if (a.h_dtype == MOE_DTYPE_F32)
    err = a.o_dtype == MOE_DTYPE_F32    ? backward_types<float, float>(a, s)
          : a.o_dtype == MOE_DTYPE_BF16 ? backward_types<float, __nv_bfloat16>(a, s)
                                        : backward_types<float, __half>(a, s);
  else
    err = a.h_dtype == MOE_DTYPE_BF16 ? backward_types<__nv_bfloat16, __nv_bfloat16>(a, s)
                                      : backward_types<__half, __half>(a, s);
  stage_end(s);
  if (err == cudaSuccess && a.nacc > 0) {
    stage_begin("column_sums", s);
    err = launch_dependent(norm_sums_kernel, dim3((a.H + 31) / 32, a.nacc), dim3(32, 32), 0, s, a, out);
    stage_end(s);
  }
  return err;
}

cudaError_t launch_column_sums(const float* partials, int nparts, int width, float* out, cudaStream_t s) {
  stage_begin("column_sums", s);
  const cudaError_t err =
      launch_dependent(norms::column_sums_kernel, dim3((width + 31) / 32), dim3(32, 32), 0, s, partials, nparts, width, out);
  stage_end(s);
  return err;
}

}  // namespace moe
