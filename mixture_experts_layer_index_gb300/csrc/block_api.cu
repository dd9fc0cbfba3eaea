// C entry points of the operators around the routed FFN (include/moe.h: routing
// rules, block norms, linear layer): argument validation, then the launches.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool is_dtype(int d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
size_t size_of(int d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
// An array of dtype that may be absent.
bool fits(const void* p, int dtype) { return aligned(p, size_of(dtype)); }

// ------------------------------------------------------------------ routing
moe_status check_route(const moe_route_options* o, int T, int E, int k) {
  if (!o || T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (o->score_fn != MOE_SCORE_SOFTMAX && o->score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (o->renormalise != 0 && o->renormalise != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(o->scale) || o->scale == 0.0f || !is_dtype(o->dtype)) return MOE_ERR_INVALID_ARG;
  if (o->group_best != 1 && o->group_best != 2) return MOE_ERR_INVALID_ARG;
  if (o->n_group < 1 || E % o->n_group || o->topk_group < 1 || o->topk_group > o->n_group) return MOE_ERR_INVALID_ARG;
  if (k > o->topk_group * (E / o->n_group)) return MOE_ERR_INVALID_ARG;
  if ((o->ld != 0 && o->ld < E) || (o->ld_grad != 0 && o->ld_grad < E)) return MOE_ERR_INVALID_ARG;
  if (!aligned(o->bias, 4)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || k > kMaxK || o->n_group > 32 || static_cast<long long>(T) * k >= (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

RouteArgs route_args(const moe_route_options& o, int T, int E, int k) {
  RouteArgs a{};
  a.T = T;
  a.E = E;
  a.k = k;
  a.score_fn = o.score_fn;
  a.renormalise = o.renormalise;
  a.scale = o.scale;
  a.n_group = o.n_group;
  a.topk_group = o.topk_group;
  a.group_best = o.group_best;
  a.bias = o.bias;
  a.ld = o.ld ? o.ld : E;
  return a;
}

// ------------------------------------------------------------------ norms
bool is_norm(int n) { return n == MOE_NORM_NONE || n == MOE_NORM_RMS || n == MOE_NORM_LAYER; }

moe_status check_norm(const moe_norm_problem* p) {
  if (!p || p->T < 0 || p->H < 1 || !is_norm(p->post_norm) || !is_norm(p->pre_norm)) return MOE_ERR_INVALID_ARG;
  if (p->gate < MOE_GATE_NONE || p->gate > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(p->h_dtype) || !is_dtype(p->o_dtype) || !is_dtype(p->w_dtype)) return MOE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps) || !std::isfinite(p->alpha) || !std::isfinite(p->beta))
    return MOE_ERR_INVALID_ARG;
  if ((p->ld_h != 0 && p->ld_h < p->H) || (p->ld_o != 0 && p->ld_o < p->H)) return MOE_ERR_INVALID_ARG;
  if (p->h_dtype != p->o_dtype && p->h_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (p->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

NormArgs norm_args(const moe_norm_problem& p) {
  NormArgs a{};
  a.T = p.T;
  a.H = p.H;
  a.h_dtype = p.h_dtype;
  a.o_dtype = p.o_dtype;
  a.post = p.post_norm;
  a.pre = p.pre_norm;
  a.gate_kind = p.gate;
  a.w_dtype = p.w_dtype;
  a.eps = p.eps;
  a.alpha = p.alpha;
  a.beta = p.beta;
  a.ld_h = p.ld_h ? p.ld_h : p.H;
  a.ld_o = p.ld_o ? p.ld_o : p.H;
  return a;
}

// 16-byte accesses fit: eight columns are 16 or 32 bytes, so rows of H % 8 == 0 columns
// whose strides are multiples of 8 elements keep the bases' alignment.
template <typename... P>
bool norm_vec(const NormArgs& a, P... ptrs) {
  const void* list[] = {ptrs...};
  if (a.H % 8 || a.ld_h % 8 || a.ld_o % 8) return false;
  for (const void* q : list)
    if (!aligned(q, 16)) return false;
  return true;
}

moe_status check_gate(const moe_norm_problem& p, const void* gate) {
  if ((p.gate == MOE_GATE_NONE) != (gate == nullptr)) return MOE_ERR_INVALID_ARG;
  const int dtype = p.gate == MOE_GATE_CHANNEL ? p.w_dtype : p.gate == MOE_GATE_TOKEN ? MOE_DTYPE_F32 : p.o_dtype;
  return fits(gate, dtype) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------ linear
moe_status check_linear(const moe_linear_problem* p) {
  if (!p || p->M < 0 || p->N < 0 || p->K < 1) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(p->dtype) || !is_dtype(p->out_dtype) || !is_dtype(p->bias_dtype)) return MOE_ERR_INVALID_ARG;
  if (p->act < MOE_ACT_NONE || p->act > MOE_ACT_GELU_TANH || !std::isfinite(p->alpha)) return MOE_ERR_INVALID_ARG;
  if ((p->ld_x != 0 && p->ld_x < p->K) || (p->ld_w != 0 && p->ld_w < p->K) || (p->ld_y != 0 && p->ld_y < p->N))
    return MOE_ERR_INVALID_ARG;
  if (p->dtype == MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  const long long ld_x = p->ld_x ? p->ld_x : p->K, ld_w = p->ld_w ? p->ld_w : p->K;
  if (ld_x % 8 || ld_w % 8 || ld_x >= (1ll << 38) || ld_w >= (1ll << 38)) return MOE_ERR_UNSUPPORTED;
  // tile coordinates are 32-bit, and a product's grid (128 columns x at least 16 rows, up to eight blocks) below 2^31
  if (p->M > (1 << 30) || p->N > (1 << 30) || p->K > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  auto blocks = [](long long cols, long long rows) { return (cols / 128 + 1) * (rows / 16 + 1) * 8; };
  if (blocks(p->N, p->M) >= (1ll << 31) || blocks(p->K, p->M) >= (1ll << 31) || blocks(p->K, p->N) >= (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

constexpr size_t kHeaderBytes = 256;

// An empty problem needs no workspace, but where one is given its status is this call's.
cudaError_t clear_status(void* ws, size_t ws_bytes, cudaStream_t s) {
  if (!ws || !aligned(ws, 256) || ws_bytes < kHeaderBytes) return cudaSuccess;
  return launch_reset_header(static_cast<DeviceHeader*>(ws), s);
}

struct LinearBackwardLayout {
  size_t partials, dz, total;
};
LinearBackwardLayout plan_linear_backward(int M, int N) {
  LinearBackwardLayout L;
  L.partials = kHeaderBytes;
  L.dz = align_up(L.partials + linear_partials_bytes(M, N), 256);
  L.total = align_up(L.dz + linear_dz_bytes(M, N), 256);
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_ex(const moe_route_options* opt, const void* scores, int T, int E, int k, int32_t* ids, float* w,
                        moe_stream_t stream) {
  const moe_status st = check_route(opt, T, E, k);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!scores || !ids || !w || !fits(scores, opt->dtype) || !aligned(ids, 4) || !aligned(w, 4))
    return MOE_ERR_INVALID_ARG;
  RouteArgs a = route_args(*opt, T, E, k);
  a.ids = ids;
  a.w = w;
  return from_cuda(launch_route_ex(scores, opt->dtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_route_backward(const moe_route_options* opt, const void* scores, int T, int E, int k,
                              const int32_t* ids, const float* dw, void* dscores, moe_stream_t stream) {
  const moe_status st = check_route(opt, T, E, k);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!scores || !ids || !dw || !dscores || !fits(scores, opt->dtype) || !fits(dscores, opt->dtype) ||
      !aligned(ids, 4) || !aligned(dw, 4))
    return MOE_ERR_INVALID_ARG;
  return from_cuda(launch_route_backward(scores, opt->dtype, route_args(*opt, T, E, k), ids, dw, dscores,
                                         opt->ld_grad ? opt->ld_grad : E, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_forward(const moe_norm_problem* p, const void* h, const void* o, const void* gate,
                            const void* w_post, const void* b_post, const void* w_pre, const void* b_pre, void* h_out,
                            void* x_out, moe_stream_t stream) {
  moe_status st = check_norm(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  st = check_gate(*p, gate);
  if (st != MOE_OK) return st;
  const bool pre = p->pre_norm != MOE_NORM_NONE, post = p->post_norm != MOE_NORM_NONE;
  if (!h || !o || !h_out || pre != (x_out != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((!post && (w_post || b_post)) || (!pre && (w_pre || b_pre))) return MOE_ERR_INVALID_ARG;
  if (!fits(h, p->h_dtype) || !fits(h_out, p->h_dtype) || !fits(o, p->o_dtype) || !fits(x_out, p->o_dtype) ||
      !fits(w_post, p->w_dtype) || !fits(b_post, p->w_dtype) || !fits(w_pre, p->w_dtype) || !fits(b_pre, p->w_dtype))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = norm_args(*p);
  a.h = h;
  a.o = o;
  a.gate = gate;
  a.w_post = w_post;
  a.b_post = b_post;
  a.w_pre = w_pre;
  a.b_pre = b_pre;
  a.h_out = h_out;
  a.x_out = x_out;
  a.vec = norm_vec(a, h, o, p->gate == MOE_GATE_TOKEN ? nullptr : gate, w_post, b_post, w_pre, b_pre,
                            static_cast<const void*>(h_out), static_cast<const void*>(x_out));
  return from_cuda(launch_norm_forward(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_norm_backward_workspace_size(const moe_norm_problem* p) {
  if (check_norm(p) != MOE_OK) return 0;
  const size_t n = norm_partials_bytes(p->T, p->H);
  return n ? n : 16;
}

moe_status moe_norm_backward(const moe_norm_problem* p, const void* dh_out, const void* dx_out, const void* h_out,
                             const void* o, const void* gate, const void* w_post, const void* b_post,
                             const void* w_pre, void* dh, void* d_o, void* dgate, float* dw_post, float* db_post,
                             float* dw_pre, float* db_pre, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_norm(p);
  if (st != MOE_OK) return st;
  const bool pre = p->pre_norm != MOE_NORM_NONE, post = p->post_norm != MOE_NORM_NONE;
  if ((!post && (w_post || b_post || dw_post || db_post)) || (!pre && (w_pre || dw_pre || db_pre || dx_out)))
    return MOE_ERR_INVALID_ARG;
  if (p->gate == MOE_GATE_NONE && dgate) return MOE_ERR_INVALID_ARG;
  const int dgate_dtype = p->gate == MOE_GATE_FULL ? p->o_dtype : MOE_DTYPE_F32;
  if (!fits(dgate, dgate_dtype) || !aligned(dw_post, 4) || !aligned(db_post, 4) || !aligned(dw_pre, 4) ||
      !aligned(db_pre, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const NormSums sums{dw_post, db_post, dw_pre, db_pre,
                      p->gate == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr};
  if (p->T == 0) {
    cudaError_t e = cudaSuccess;
    for (float* v : {sums.dw_post, sums.db_post, sums.dw_pre, sums.db_pre, sums.dgate})
      if (v && e == cudaSuccess) e = cudaMemsetAsync(v, 0, static_cast<size_t>(p->H) * 4, s);
    return from_cuda(e);
  }
  st = check_gate(*p, gate);
  if (st != MOE_OK) return st;
  if (!o || (pre && (!dx_out || !h_out))) return MOE_ERR_INVALID_ARG;
  if (!fits(dh_out, p->h_dtype) || !fits(dx_out, p->o_dtype) || !fits(h_out, p->h_dtype) || !fits(o, p->o_dtype) ||
      !fits(w_post, p->w_dtype) || !fits(b_post, p->w_dtype) || !fits(w_pre, p->w_dtype) || !fits(dh, p->h_dtype) ||
      !fits(d_o, p->o_dtype))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < moe_norm_backward_workspace_size(p)) return MOE_ERR_WORKSPACE;
  NormArgs a = norm_args(*p);
  a.dh_out = dh_out;
  a.dx_out = dx_out;
  a.h = h_out;
  a.o = o;
  a.gate = gate;
  a.w_post = w_post;
  a.b_post = b_post;
  a.w_pre = w_pre;
  a.dh = dh;
  a.d_o = d_o;
  a.dgate = dgate;
  a.partials = static_cast<float*>(ws);
  a.vec = norm_vec(a, dh_out, dx_out, h_out, o, p->gate == MOE_GATE_TOKEN ? nullptr : gate, w_post, b_post,
                            w_pre, static_cast<const void*>(dh), static_cast<const void*>(d_o),
                            p->gate == MOE_GATE_FULL ? static_cast<const void*>(dgate) : nullptr);
  return from_cuda(launch_norm_backward(a, sums, s));
}

size_t moe_linear_workspace_size(const moe_linear_problem* p) { return check_linear(p) == MOE_OK ? kHeaderBytes : 0; }

moe_status moe_linear(const moe_linear_problem* p, const void* x, const void* w, const void* bias,
                      const void* residual, void* y, void* z, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const moe_status st = check_linear(p);
  if (st != MOE_OK) return st;
  if (p->M == 0 || p->N == 0) return from_cuda(clear_status(ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream)));
  if (!x || !w || !y || !aligned(x, 16) || !aligned(w, 16) || !fits(y, p->out_dtype) || !fits(z, p->dtype) ||
      !fits(residual, p->out_dtype) || !fits(bias, p->bias_dtype))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < kHeaderBytes) return MOE_ERR_WORKSPACE;
  LinearArgs a{};
  a.M = p->M;
  a.N = p->N;
  a.K = p->K;
  a.dtype = p->dtype;
  a.out_dtype = p->out_dtype;
  a.bias_dtype = p->bias_dtype;
  a.act = p->act;
  a.alpha = p->alpha;
  a.ld_x = p->ld_x ? p->ld_x : p->K;
  a.ld_w = p->ld_w ? p->ld_w : p->K;
  a.ld_y = p->ld_y ? p->ld_y : p->N;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.z = z;
  a.hdr = static_cast<DeviceHeader*>(ws);
  return from_cuda(launch_linear(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_linear_backward_workspace_size(const moe_linear_problem* p) {
  return check_linear(p) == MOE_OK ? plan_linear_backward(p->M, p->N).total : 0;
}

moe_status moe_linear_backward(const moe_linear_problem* p, const void* dy, const void* x, const void* w,
                               const void* z, void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes,
                               moe_stream_t stream) {
  const moe_status st = check_linear(p);
  if (st != MOE_OK) return st;
  if (!fits(dx, p->dtype) || !fits(dw, p->dtype) || !aligned(dbias, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->M == 0 || p->N == 0) {  // empty sums
    cudaError_t e = clear_status(ws, ws_bytes, s);
    if (e == cudaSuccess && dx && p->M) e = cudaMemsetAsync(dx, 0, static_cast<size_t>(p->M) * p->K * 2, s);
    if (e == cudaSuccess && dw && p->N) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(p->N) * p->K * 2, s);
    if (e == cudaSuccess && dbias && p->N) e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(p->N) * 4, s);
    return from_cuda(e);
  }
  if (!dy || (dw && !x) || (dx && !w) || ((p->act != MOE_ACT_NONE) != (z != nullptr))) return MOE_ERR_INVALID_ARG;
  if (!fits(dy, p->out_dtype) || !aligned(x, 16) || !aligned(w, 16) || !fits(z, p->dtype)) return MOE_ERR_INVALID_ARG;
  const LinearBackwardLayout L = plan_linear_backward(p->M, p->N);
  if (!ws || !aligned(ws, 256) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  LinearBackwardArgs a{};
  a.M = p->M;
  a.N = p->N;
  a.K = p->K;
  a.dtype = p->dtype;
  a.dy_dtype = p->out_dtype;
  a.act = p->act;
  a.alpha = p->alpha;
  a.ld_x = p->ld_x ? p->ld_x : p->K;
  a.ld_w = p->ld_w ? p->ld_w : p->K;
  a.ld_y = p->ld_y ? p->ld_y : p->N;
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.z = z;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.partials = reinterpret_cast<float*>(base + L.partials);
  a.dz = base + L.dz;
  a.hdr = static_cast<DeviceHeader*>(ws);
  return from_cuda(launch_linear_backward(a, s));
}

}  // extern "C"
