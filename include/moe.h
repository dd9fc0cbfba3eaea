/*
 * moe.h - C ABI of the GB300 (sm_103a) routed Mixture-of-Experts FFN forward.
 *
 * The library computes, on one GPU, the routed MoE FFN forward pass whose
 * expert-grouped pipeline the Motivation of "perf: add small-batch route MMA
 * for MoE" describes: top-k routing; grouping the routes by expert (counts and
 * a stable order); gathering the rows; prefix sums and a GEMM task map; the
 * Gate/Up grouped GEMM; SwiGLU with optional FP8 re-quantisation; the Down
 * grouped GEMM; and the weighted reduction of each token's k expert outputs
 * (the index_shuffling and scatter_add_dense_tokens steps of "Port necessary
 * FBGEMM MoE kernels").  It also has the route-direct small-batch path of the
 * route-MMA page's Summary: each route reads its expert directly, with no
 * sort, gather, prefix sum or task map; the long Gate/Up K dimension is split
 * for parallelism; and the split reduction, SwiGLU and the quantisation of the
 * Down input are done in one pass.
 *
 * Definitions used throughout:
 *   T tokens, E experts, k = top_k, H hidden size, I expert intermediate size,
 *   R = T*k routes; route r = t*k + j is slot j of token t.
 *   Routing: ids[t, 0..k-1] = the k experts with the largest router score,
 *   ordered by score descending, ties to the lower expert id (-0.0 == +0.0);
 *   w[t, j] = softmax over the k selected scores.
 *   Gate/Up weights W1 [E, 2I, H]: rows 0..I-1 of W1[e] are the gate
 *   projection, rows I..2I-1 the up projection.  Down weights W2 [E, H, I].
 *   y[t] = sum_j w[t, j] * W2[ids[t, j]] (silu(gate) * up), rounded to bf16.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers to row-major, contiguous
 *     arrays, unless stated otherwise.  Bases of bf16 / e4m3 arrays and of
 *     the workspace must be 16-byte aligned (a TMA requirement); int32 and
 *     fp32 arrays 4-byte aligned.
 *   - The caller owns and allocates every buffer, including outputs and the
 *     workspace.  The library never allocates, frees or synchronises inside
 *     moe_route / moe_shuffle / moe_tile_map / moe_forward / moe_forward_ex /
 *     moe_forward_routed / moe_round_bf16 / moe_route_ex / moe_route_backward /
 *     moe_norm_forward / moe_norm_backward / moe_linear / moe_linear_backward /
 *     moe_gated / moe_gated_backward / moe_quantise / moe_linear_fp8 /
 *     moe_gated_fp8: work is enqueued on `stream` in order, with no device-to-host copy, so these calls can be
 *     captured in a CUDA graph.  Inputs are never written.
 *   - A workspace serves one call at a time: calls whose work may overlap (on two
 *     streams, or in graphs that run side by side) need workspaces of their own.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).
 *   - A process uses the library on one device, the one current at its first call.
 *   - Arguments are validated on the host BEFORE anything is enqueued; on a
 *     validation error nothing is launched and outputs are untouched.
 *   - A launch failure returns MOE_ERR_CUDA.  Conditions detected on the device
 *     (a bounded wait that timed out, an index out of range) are recorded in
 *     a status word at the head of the workspace and reported by
 *     moe_read_device_status(); the library never traps.
 *   - Results are deterministic: the same inputs give bitwise identical
 *     outputs, eager or replayed from a CUDA graph.
 */
#ifndef MOE_GB300_MOE_H_
#define MOE_GB300_MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared here so that the header needs no CUDA headers. */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,    /* bad shape, null or misaligned pointer, inconsistent scales */
  MOE_ERR_UNSUPPORTED = 2,    /* valid, but outside what this library implements (limits below) */
  MOE_ERR_WORKSPACE = 3,      /* workspace missing or smaller than the *_workspace_size() value */
  MOE_ERR_CUDA = 4,           /* a CUDA runtime/driver call or a launch failed, or no usable GPU */
  MOE_ERR_DEVICE_TIMEOUT = 5, /* a kernel's bounded wait expired (reported by moe_read_device_status) */
  MOE_ERR_DEVICE_BOUNDS = 6   /* a kernel saw an out-of-range index (reported by moe_read_device_status) */
} moe_status;

typedef enum {
  MOE_BF16 = 0,           /* bf16 x, W1, W2; bf16 h; fp32 accumulation */
  MOE_FP8_PER_TENSOR = 1, /* e4m3 W1/W2 with one fp32 scale per expert matrix; x and h quantised to
                             e4m3 with one dynamic scale each (amax/448 over the whole tensor) */
  MOE_FP8_BLOCK128 = 2,   /* e4m3 W1/W2 with fp32 scales per 128x128 block; x quantised per
                             (token, 128 columns); h per (route, 128 columns) */
  MOE_MXFP8 = 3           /* MXFP8: e4m3 W1/W2 with one E8M0 (power-of-two) scale per 32
                             consecutive values of a row along K; x and h quantised the same
                             way (grouped path only; see moe_forward) */
} moe_quant;

typedef enum {
  MOE_PATH_AUTO = 0,        /* library chooses (see moe_select_path) */
  MOE_PATH_GROUPED = 1,     /* group routes by expert, tile map, grouped GEMMs, combine */
  MOE_PATH_ROUTE_DIRECT = 2 /* route-order decode path, no sort / gather / tile map */
} moe_path;

typedef struct {
  int T, E, k, H, I;
  moe_quant quant;
  moe_path path;
} moe_problem;

/* Limits of this library (MOE_ERR_UNSUPPORTED beyond them):
 *   1 <= E <= 512;  1 <= k <= min(E, 32);  0 <= T;  T*k < 2^31;
 *   H % 64 == 0, I % 64 == 0 (bf16, FP8 per-tensor);  H % 128 == 0, I % 64 == 0 (FP8
 *   blockwise, whose last 128-column scale group of I may hold 64 columns, and MXFP8);
 *   MOE_PATH_GROUPED: all four modes;  MOE_PATH_ROUTE_DIRECT: per-tensor and blockwise
 *   FP8, T*k <= 1024. */

/* ---------------------------------------------------------------- routing
 * moe_route - top-k routing (the routing step of "perf: add small-batch route
 * MMA for MoE", Motivation).
 *   scores [T, E] fp32 (finite; NaN/inf are outside the contract)
 *   ids    [T, k] int32 out: selected experts in slot order (score desc, id asc)
 *   w      [T, k] fp32  out: softmax over the k selected scores
 * ids are exact; w is computed in fp32 (expf, IEEE division).
 * T == 0 is a no-op.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
moe_status moe_route(const float* scores, int T, int E, int k, int32_t* ids, float* w,
                     moe_stream_t stream);

/* ---------------------------------------------------------------- shuffle
 * moe_shuffle - index shuffling (index_shuffling of "Port necessary FBGEMM
 * MoE kernels"; the counting and sorting step of the route-MMA page's
 * Motivation).
 *   ids     [T, k] int32 in: expert of each route, each in [0, E)
 *   counts  [E]    int32 out: routes per expert
 *   offsets [E+1]  int32 out: exclusive prefix sum of counts (offsets[E] = R)
 *   perm    [R]    int32 out: sorted position -> route r; stable (routes of one
 *                             expert keep increasing r, i.e. token order)
 *   inv     [R]    int32 out: route -> sorted position (inv[perm[p]] == p)
 *   ws      device scratch of at least moe_shuffle_workspace_size(T, E, k) bytes
 * All outputs are unique and therefore bit-exact.  An id outside [0, E) is
 * recorded as MOE_ERR_DEVICE_BOUNDS in the status word at the head of ws and
 * that route is left out of the outputs.  Errors: INVALID_ARG, UNSUPPORTED,
 * WORKSPACE, CUDA. */
size_t moe_shuffle_workspace_size(int T, int E, int k);
moe_status moe_shuffle(const int32_t* ids, int T, int E, int k, int32_t* counts, int32_t* offsets,
                       int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- shuffle, no allocation
 * moe_shuffle_noalloc - moe_shuffle without a caller-provided workspace.  The
 * pages have no counterpart to this entry point: it exists for callers that
 * cannot allocate device memory when they need the shuffle - code running while
 * a stream is captured into a CUDA graph (cudaMalloc is not allowed there),
 * plugins of a host framework that owns all device memory and provides no
 * scratch, and serving loops that forbid allocation after start-up.
 *   Arguments and outputs: as moe_shuffle (caller-owned device arrays).
 *   Scratch: a fixed array of MOE_NOALLOC_SCRATCH_BYTES inside the library;
 *   every GPU that loads the library holds it until the process exits.  Neither
 *   this call nor the library allocates or frees anything.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture.  The looked-up address is cached for the life
 *   of the process: destroying the device's context after the first call
 *   (cudaDeviceReset) and calling again is not supported.
 *   Every call uses the same array: calls whose work overlaps on the GPU (e.g.
 *   on two streams) race and must be serialised by the caller.
 *   Errors: as moe_shuffle; MOE_ERR_WORKSPACE when the problem needs more than
 *   the fixed array (moe_shuffle_workspace_size(T, E, k) >
 *   MOE_NOALLOC_SCRATCH_BYTES; e.g. up to 131072 routes with E = 128 fit).
 *   An out-of-range id is skipped as in moe_shuffle; its status word is the
 *   array's and is not exposed. */
#define MOE_NOALLOC_SCRATCH_BYTES (1u << 20)
moe_status moe_shuffle_noalloc(const int32_t* ids, int T, int E, int k, int32_t* counts, int32_t* offsets,
                               int32_t* perm, int32_t* inv, moe_stream_t stream);

/* ---------------------------------------------------------------- tile map
 * moe_tile_map - the grouped GEMMs' task map (the task-map step of the
 * route-MMA page's Motivation, sized by the experts that actually have routes,
 * as its Code changes do), built on the device with no device-to-host copy.
 *   counts    [E] int32 in (e.g. from moe_shuffle)
 *   BM        row-tile height (1..1024; moe_forward uses 128)
 *   tiles     [max_tiles, 4] int32 out: {expert, first sorted row, rows, 0} for
 *             each tile, experts in id order, ceil(counts[e]/BM) tiles each
 *   num_tiles [1] int32 out: number of tiles written
 *   max_tiles capacity of `tiles`; floor(sum(counts)/BM) + E always suffices.
 * If the tiles do not fit, num_tiles holds the required count, only
 * max_tiles tiles are written and MOE_ERR_DEVICE_BOUNDS is recorded in the
 * status word at the head of ws.  ws needs moe_shuffle_workspace_size(0, E, 1)
 * bytes.  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
moe_status moe_tile_map(const int32_t* counts, int E, int BM, int32_t* tiles, int32_t* num_tiles,
                        int max_tiles, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- forward
 * moe_select_path - the path moe_forward takes for *p (AUTO resolved):
 * bf16 and MXFP8 -> GROUPED; per-tensor FP8 -> ROUTE_DIRECT for T <= 96,
 * blockwise FP8 -> ROUTE_DIRECT for T <= 64 (both also need T*k <= 1024), else
 * GROUPED: the crossovers measured on GB300.  Returns p->path when it is not
 * AUTO. */
moe_path moe_select_path(const moe_problem* p);

/* moe_workspace_size - bytes of device workspace moe_forward needs for *p
 * (0 if *p is invalid or unsupported). */
size_t moe_workspace_size(const moe_problem* p);

/* moe_forward - the whole routed MoE FFN forward.
 *   x        [T, H]  bf16 activations
 *   scores   [T, E]  fp32 router scores
 *   w1       [E, 2I, H] bf16 (MOE_BF16) or e4m3 codes (FP8 modes); rows 0..I-1 gate, I..2I-1 up
 *   w2       [E, H, I]  bf16 or e4m3
 *   w1_scale NULL (bf16) | fp32 [E] (per-tensor) | fp32 [E, 2I/128, H/128] (blockwise; a block
 *            row of W1 may hold the last gate rows and the first up rows when I % 128 == 64)
 *            | uint8 E8M0 codes [E, 2I, H/32] (MXFP8, passed through this pointer)
 *   w2_scale NULL (bf16) | fp32 [E] (per-tensor) | fp32 [E, H/128, ceil(I/128)] (blockwise)
 *            | uint8 E8M0 codes [E, H, I/32] (MXFP8)
 *   y        [T, H]  bf16 out, preallocated by the caller (written, never read)
 *   ws       device workspace of at least moe_workspace_size(p) bytes; its
 *            contents on entry do not matter and are overwritten
 * Quantisation (FP8 modes): scale = amax/448 in fp32 (1 when amax == 0),
 * code = e4m3(v / scale) rounded to nearest even with saturation.  MXFP8 (the
 * OCP Microscaling format named by "[mxfp8 moe training] add per group blocked
 * scale kernels"): each run of 32 values along the contraction dimension
 * shares the scale 2^X, X = floor(log2(amax)) - 8 clamped to [-127, 127] (-127
 * for a zero run), stored as the E8M0 code X + 127; code = e4m3(v / 2^X), RNE,
 * saturating.  The MXFP8 forward converts x's, h's and the weights' scales
 * into the blocked layout of moe_mx_blocked_scales (groups = the experts'
 * row segments) on every call and multiplies with the tensor cores'
 * block-scaled MMA; h is quantised in the Gate/Up epilogue.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
moe_status moe_forward(const moe_problem* p, const void* x, const float* scores, const void* w1,
                       const void* w2, const float* w1_scale, const float* w2_scale, void* y,
                       void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- forward, extended
 * moe_forward_ex - moe_forward with the optional parts below (opt NULL or all
 * zero = moe_forward).
 *
 * Shared experts (the "shared output" that the Summary of "perf: add small-batch
 * route MMA for MoE" lists; the page does not define it, and this library takes
 * the common reading): n_shared = S experts, each with the routed experts'
 * shapes and formats, that every token passes through with weight 1:
 *   y[t] = sum_j w[t, j] * o_(t, j)  +  sum_s FFN_shared[s](x_t),
 * summed j ascending then s ascending, rounded once.  Their rows are more rows
 * of the same intermediate tensor: x is quantised once for both, and in
 * per-tensor FP8 the dynamic scale of h spans the routed and the shared rows.
 *   w1_shared        [S, 2I, H] bf16 | e4m3 (rows 0..I-1 gate, I..2I-1 up)
 *   w2_shared        [S, H, I]
 *   w1_shared_scale  NULL (bf16) | fp32 [S] | fp32 [S, 2I/128, H/128]
 *   w2_shared_scale  NULL (bf16) | fp32 [S] | fp32 [S, H/128, ceil(I/128)]
 * Shared experts run on the grouped path (AUTO takes it; an explicit
 * MOE_PATH_ROUTE_DIRECT with S > 0 is UNSUPPORTED).  0 <= S <= 16.
 *
 * Unrounded output (y_fp32 = 1): y is fp32 [T, H], the sum above before its
 * rounding.  This is the partial output of one slice of a tensor-parallel
 * split of I (the TP8 deployment in the route-MMA page's Performance section):
 * each slice holds gate rows and up rows [p*I/P, (p+1)*I/P) of every W1[e] (and
 * the same columns of W2[e], and for blockwise FP8 the matching scale blocks, so
 * I/P must be a multiple of 128) and runs moe_forward_ex with I/P as its I; the
 * caller sums the slices' partial outputs (e.g. an all-reduce) and rounds the sum
 * with moe_round_bf16.  In bf16 and blockwise FP8 that equals the unsplit
 * forward up to fp32 summation order; per-tensor FP8 then scales h per slice.
 *
 * moe_workspace_size_ex gives the workspace for (*p, *opt); moe_forward_views_ex
 * the views of that workspace.  Errors: as moe_forward. */
typedef struct {
  int n_shared;
  const void* w1_shared;
  const void* w2_shared;
  const float* w1_shared_scale;
  const float* w2_shared_scale;
  int y_fp32;
  int mx_weight_scales_blocked; /* MXFP8: 1 = the weight scale pointers (routed and shared) hold
                                   the blocked layouts of moe_mx_weight_scales instead of the
                                   row-major E8M0 codes (no per-call conversion) */
} moe_forward_options;
size_t moe_workspace_size_ex(const moe_problem* p, const moe_forward_options* opt);
moe_status moe_forward_ex(const moe_problem* p, const moe_forward_options* opt, const void* x, const float* scores,
                          const void* w1, const void* w2, const float* w1_scale, const float* w2_scale, void* y,
                          void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_forward_routed - moe_forward_ex with a given routing in the place of scores, as
 * moe_route or moe_route_ex writes it:
 *   ids [T, k] int32, w [T, k] fp32: y[t] = sum_j w[t, j] * FFN_{ids[t, j]}(x_t) + shared
 * Weights are used as they are; views' ids and w hold copies.  An id outside [0, E)
 * is recorded as MOE_ERR_DEVICE_BOUNDS in the status word at the head of ws; its route
 * is not computed, adds nothing to y (its copy of w is 0) and has no part in the
 * per-tensor scale of h.  Everything else as moe_forward_ex. */
moe_status moe_forward_routed(const moe_problem* p, const moe_forward_options* opt, const void* x, const int32_t* ids,
                              const float* w, const void* w1, const void* w2, const float* w1_scale,
                              const float* w2_scale, void* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_mx_weight_scales - the MXFP8 weights' scales in the blocked layout the
 * forward's block-scaled MMAs read, converted once (e.g. when the weights are
 * loaded) instead of on every call (moe_forward_options.mx_weight_scales_blocked).
 *   w1_scale [E, 2I, H/32], w2_scale [E, H, I/32] uint8 E8M0 codes (4-byte aligned)
 *   w1_blocked, w2_blocked  outputs of moe_mx_weight_scales_bytes(E, H, I, 1 / 2)
 *                           bytes (16-byte aligned): W1 as the B operands of the
 *                           Gate/Up units (96 gate rows and the matching 96 up rows
 *                           of one expert, two 128-row blocks per unit, adjacent
 *                           per column block), W2 likewise as the B operands of the
 *                           Down units (192 rows, two blocks each); blocks are the
 *                           512-byte blocks of moe_mx_blocked_scales.
 * Errors: INVALID_ARG, UNSUPPORTED (the MXFP8 shape limits), CUDA. */
size_t moe_mx_weight_scales_bytes(int E, int H, int I, int which);
moe_status moe_mx_weight_scales(const uint8_t* w1_scale, const uint8_t* w2_scale, int E, int H, int I,
                                uint8_t* w1_blocked, uint8_t* w2_blocked, moe_stream_t stream);

/* moe_round_bf16 - y[i] = bf16(y32[i]) for i < n (round to nearest even): the
 * single rounding of a sum of partial outputs (moe_forward_ex, y_fp32 = 1).
 * y32 fp32 [n], y bf16 [n], both 16-byte aligned, n a multiple of 8.
 * Errors: INVALID_ARG, CUDA. */
moe_status moe_round_bf16(const float* y32, void* y, size_t n, moe_stream_t stream);

/* ---------------------------------------------------------------- MX scale layout
 * moe_mx_blocked_scales - the per-group blocked scale conversion of "[mxfp8 moe
 * training] add per group blocked scale kernels" (Summary): MX scales of row
 * groups (e.g. the expert groups of a grouped GEMM's activations) converted
 * into the blocked, swizzled layout that block-scaled tensor-core MMAs read,
 * each group on its own and padded to whole 128-row blocks, with every group's
 * start row in the padded output computed on the device (no device-to-host
 * copy).
 *   scales        [rows, cols] uint8 (one byte per scale, row-major; base 4-byte aligned)
 *   group_offsets [groups + 1] int32: group g = rows [off[g], off[g+1]),
 *                 nondecreasing, off[groups] <= rows
 *   out           blocked output, at least moe_mx_blocked_bytes(rows, cols,
 *                 groups) bytes; group g's padded rows start at row
 *                 group_starts[g] of an [*, ceil(cols/4)*4] byte matrix
 *   group_starts  [groups + 1] int32 out: padded start rows; entry groups = total
 *   ws            scratch of moe_mx_blocked_workspace_size(rows, groups) bytes
 * Layout: each group's scales are zero-padded to a multiple of 128 rows and of
 * 4 columns and cut into 128 x 4 blocks, stored block row by block row; inside
 * a 512-byte block the scale of (row r, column c) is at byte (r % 32) * 16 +
 * (r / 32) * 4 + c.  Output bytes past group_starts[groups] rows are not
 * written.  A negative group size is recorded as MOE_ERR_DEVICE_BOUNDS (status
 * word at the head of ws) and treated as empty.  1 <= groups <= 4096.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
size_t moe_mx_blocked_bytes(int rows, int cols, int groups);
size_t moe_mx_blocked_workspace_size(int rows, int groups);
moe_status moe_mx_blocked_scales(const uint8_t* scales, int rows, int cols, const int32_t* group_offsets,
                                 int groups, uint8_t* out, size_t out_bytes, int32_t* group_starts, void* ws,
                                 size_t ws_bytes, moe_stream_t stream);

/* moe_forward_views - device pointers to the intermediate results moe_forward
 * leaves in the workspace (read-only diagnostics; valid after the call's
 * work on the stream completed).  Pointers not produced by the path chosen
 * for *p are set to NULL.  ids/w: [T, k]; counts [E]; offsets [E+1];
 * perm/inv [R]; tiles [*, 4] and num_tiles [1] as for moe_tile_map (BM 128).
 * The activations as the Gate/Up GEMM reads them (the quantisation of x is
 * unique, so these can be checked bit for bit):
 *   xs       grouped path: [R, H] rows in expert-sorted order, row p = x row
 *            of token perm[p] / k (bf16 copies, or e4m3 codes in the FP8
 *            modes); route-direct path: [T, H] e4m3 codes in token order.
 *            NULL for the bf16 variant that gathers x inside the GEMM.
 *   x_scale  blockwise FP8: fp32 scales of xs, one per row and 128 columns
 *            ([R, H/128] sorted, or [T, H/128] route-direct); MXFP8: uint8
 *            E8M0 codes, one per row and 32 columns ([R, H/32] sorted); else
 *            NULL.
 *   amax_x   per-tensor FP8: the fp32 amax of x over the whole [T, H]
 *            (scale = amax / 448, 1 when it is 0); else NULL. */
typedef struct {
  const int32_t* ids;
  const float* w;
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* perm;
  const int32_t* inv;
  const int32_t* tiles;
  const int32_t* num_tiles;
  const void* xs;
  const float* x_scale;
  const float* amax_x;
} moe_views;
moe_status moe_forward_views(const moe_problem* p, const void* ws, size_t ws_bytes, moe_views* out);
/* The same for a workspace of moe_forward_ex(p, opt, ...); with shared experts
 * xs (and x_scale) hold T*k + S*T rows, shared expert s's row of token t at
 * T*k + s*T + t. */
moe_status moe_forward_views_ex(const moe_problem* p, const moe_forward_options* opt, const void* ws,
                                size_t ws_bytes, moe_views* out);

/* ---------------------------------------------------------------- around the routed FFN
 * The operators that a model runs next to the forward above: other routing
 * rules, the norms at a block's two ends, and a linear layer (the router's
 * logits, projections, dense FFN layers), each with its gradient.  They follow
 * the conventions at the top of this file (the entry points that take no
 * workspace detect nothing on the device).  Rows may be strided where a descriptor
 * has an `ld`: elements between the starts of two rows, 0 for contiguous rows. */

/* Element types of the arrays whose type a descriptor names.  MOE_DTYPE_E4M3, codes with a scale
 * per block of 128, is taken by the entry points that say so. */
typedef enum { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_F16 = 2, MOE_DTYPE_E4M3 = 3 } moe_dtype;

/* ---------------------------------------------------------------- routing rules
 * moe_route_ex - routing with a score function, a selection bias, expert groups
 * and renormalised, scaled weights:
 *   p_e = softmax over all E scores, or sigmoid(s_e)
 *   key_e = p_e + bias_e (with a bias: it takes part in the selection only), else s_e
 *   groups: the experts are n_group runs of E / n_group; a group ranks by its best
 *     key (group_best = 1) or by the sum of its two best keys (2; p in the place of
 *     s without a bias); experts of the topk_group best groups can be selected
 *   ids[t, 0..k-1] = the k largest keys, descending; w = p[ids], divided by their
 *     sum if renormalise, then times scale.
 * Ties, among experts and among groups, go to the lower index; -0.0 == +0.0.
 * A score of -inf (or NaN) masks its expert: p = 0, it comes after every other
 * expert of the selectable groups and counts as absent in its group's rank (a
 * group of masked experts ranks last).  If fewer than k experts are left, masked
 * ones fill the slots in id order with weight 0; a row that is masked as a whole
 * gets valid ids and weights 0.  +inf counts as the largest finite fp32.  bias
 * values are finite.  All arithmetic is in fp32: weights from expf and IEEE
 * divisions; the p of a key with a bias from the hardware's exponential and
 * division, within 2e-7, so experts whose keys differ by less may change places.
 *   scores [T, E] of dtype, ld elements between rows
 *   ids    [T, k] int32 out;  w [T, k] fp32 out
 * Limits: those of moe_route, n_group <= 32 (UNSUPPORTED); n_group divides E,
 * 1 <= topk_group <= n_group, k <= topk_group * (E / n_group) (INVALID_ARG).
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_fn;
typedef struct {
  int score_fn;      /* moe_score_fn */
  int renormalise;   /* 0 or 1 */
  float scale;       /* factor of the weights, finite and not 0 */
  int n_group;       /* 1: every expert can be selected */
  int topk_group;
  int group_best;    /* 1 or 2 */
  const float* bias; /* [E] or NULL */
  int dtype;         /* moe_dtype of scores (and of dscores) */
  long long ld;      /* of scores */
  long long ld_grad; /* of dscores */
} moe_route_options;
moe_status moe_route_ex(const moe_route_options* opt, const void* scores, int T, int E, int k, int32_t* ids, float* w,
                        moe_stream_t stream);

/* moe_route_backward - the gradient of moe_route_ex's weights into the scores, for
 * the selection it made (which has no gradient, and the bias with it):
 *   ids [T, k] as moe_route_ex wrote them (a row's ids differ; an id outside [0, E)
 *       has no part in the result), dw [T, k] fp32
 *   dscores [T, E] of dtype, every element written (0 where the score has no part).
 * Nothing of the forward but ids is needed.  Errors: as moe_route_ex. */
moe_status moe_route_backward(const moe_route_options* opt, const void* scores, int T, int E, int k,
                              const int32_t* ids, const float* dw, void* dscores, moe_stream_t stream);

/* ---------------------------------------------------------------- block norms
 * moe_norm_forward - the boundary between two blocks of a model in one pass over
 * the residual stream h and a block's output o:
 *   h_out = beta * h + alpha * gate * N_post(o)
 *   x_out = N_pre(h_out)                          (the next block's input)
 * N(v) = (v - mu) / sqrt(mean((v - mu)^2) + eps) * w + b over the H columns of a
 * row; mu = 0 for MOE_NORM_RMS, the row's mean for MOE_NORM_LAYER; N_post = identity
 * for MOE_NORM_NONE, and no x_out for a pre_norm of MOE_NORM_NONE.
 * x_out is taken from h_out before h_out is rounded to its type.
 *   h, h_out     [T, H] of h_dtype, ld_h between rows (h_out == h is allowed)
 *   o, x_out     [T, H] of o_dtype, ld_o between rows (x_out == o is allowed)
 *   gate         by `gate`: NULL | [H] of w_dtype | [T] fp32 | [T, H] of o_dtype, ld_o
 *   w_*, b_*     [H] of w_dtype, each may be NULL (ones / zeros)
 * o_dtype is h_dtype, or any type under an fp32 h.  1 <= H <= 16384.
 * Any address, ld and H is taken; rows whose addresses and strides are
 * multiples of 16 bytes (and H of 8) are read 16 bytes at a time.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef enum { MOE_NORM_NONE = 0, MOE_NORM_RMS = 1, MOE_NORM_LAYER = 2 } moe_norm_kind;
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2, MOE_GATE_FULL = 3 } moe_gate_kind;
typedef struct {
  int T, H;
  int post_norm, pre_norm; /* moe_norm_kind */
  int gate;                /* moe_gate_kind */
  int h_dtype, o_dtype, w_dtype;
  float eps, alpha, beta;
  long long ld_h, ld_o;
} moe_norm_problem;
moe_status moe_norm_forward(const moe_norm_problem* p, const void* h, const void* o, const void* gate,
                            const void* w_post, const void* b_post, const void* w_pre, const void* b_pre, void* h_out,
                            void* x_out, moe_stream_t stream);

/* moe_norm_backward - its gradient.
 *   dh_out [T, H] of h_dtype (gradient into h_out from what follows; NULL: zero),
 *   dx_out [T, H] of o_dtype (with a pre_norm), h_out (with a pre_norm) and o as the
 *   forward left and read them, gate and vectors as in the forward
 *   dh [T, H] of h_dtype, d_o [T, H] of o_dtype: outputs, either may be NULL
 *   dgate: [H] fp32 | [T] fp32 | [T, H] of o_dtype, ld_o;  dw_*, db_*: [H] fp32;
 *   each may be NULL and is written, not added to.
 * dgate needs b_post and w_post, the others only what the formulas hold.
 * Sums over tokens are in fp32 in a fixed order.  dh may be dh_out, d_o may be o or
 * dx_out.  T == 0 writes zeros to the [H] outputs.
 * ws: moe_norm_backward_workspace_size(p) bytes, 16-byte aligned.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
size_t moe_norm_backward_workspace_size(const moe_norm_problem* p);
moe_status moe_norm_backward(const moe_norm_problem* p, const void* dh_out, const void* dx_out, const void* h_out,
                             const void* o, const void* gate, const void* w_post, const void* b_post,
                             const void* w_pre, void* dh, void* d_o, void* dgate, float* dw_post, float* db_post,
                             float* dw_pre, float* db_pre, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- linear layer
 * moe_linear - y = alpha * act(z) + residual, z = x W^T + bias, fp32 accumulation,
 * one rounding each of y and z:
 *   x [M, K], w [N, K] of dtype (bf16 or fp16), ld_x / ld_w between rows: multiples of
 *     8, bases 16-byte aligned (a TMA requirement; K itself is free)
 *   bias [N] of bias_dtype or NULL;  residual [M, N] of out_dtype, ld_y, or NULL
 *   y [M, N] of out_dtype, ld_y (y == residual is allowed)
 *   z [M, N] of dtype, contiguous, or NULL (kept for the gradient of an activation)
 * act: MOE_ACT_GELU is the erf form, MOE_ACT_GELU_TANH the tanh form.  NaN and
 * infinities give what the formulas do (ReLU keeps NaN, GELU(+inf) = +inf).
 * K == 0 is INVALID_ARG; M == 0 or N == 0 computes nothing and needs no ws.
 * ws: moe_linear_workspace_size(p) bytes, 256-byte aligned: the status word
 * (moe_read_device_status), cleared by the call (by an empty one too, where ws is given).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,
  MOE_ACT_GELU = 3,
  MOE_ACT_GELU_TANH = 4
} moe_act;
typedef struct {
  int M, N, K;
  int dtype;      /* of x, w, z (and dx, dw): MOE_DTYPE_BF16 or MOE_DTYPE_F16 */
  int out_dtype;  /* of y, residual (and dy) */
  int bias_dtype;
  int act;        /* moe_act */
  float alpha;
  long long ld_x, ld_w, ld_y;
} moe_linear_problem;
size_t moe_linear_workspace_size(const moe_linear_problem* p);
moe_status moe_linear(const moe_linear_problem* p, const void* x, const void* w, const void* bias,
                      const void* residual, void* y, void* z, void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_linear_backward - dz = alpha * dy * act'(z), dx = dz W, dw = dz^T x,
 * dbias = the column sums of dz (the residual's gradient is dy itself):
 *   dy [M, N] of out_dtype, ld_y;  x, w as in the forward;  z as the forward kept it
 *   (NULL without an activation)
 *   dx [M, K] and dw [N, K] of dtype, contiguous;  dbias [N] fp32;  each may be NULL.
 * dz is rounded to dtype for the two products (the tensor cores' operand type; dy
 * itself is read where it already is dz; in fp16 a dz past 65504 is infinite there),
 * dbias sums it unrounded in fp32, in a fixed order.  M == 0 writes zeros to dw and dbias, N == 0 to dx; they need no ws.
 * ws: moe_linear_backward_workspace_size(p) bytes, 256-byte aligned, status word at
 * its head, cleared as moe_linear's, whichever outputs are wanted.  Errors: as moe_linear. */
size_t moe_linear_backward_workspace_size(const moe_linear_problem* p);
moe_status moe_linear_backward(const moe_linear_problem* p, const void* dy, const void* x, const void* w,
                               const void* z, void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes,
                               moe_stream_t stream);

/* ---------------------------------------------------------------- gated linear layer
 * moe_gated - the first half of a gated feed-forward block (the linear layer above is its
 * second half), both projections, the activation and the product in one kernel:
 *   z = [g, u] = x W^T + bias;  h = act(g) * u      fp32 accumulation, one rounding each
 *   x [M, K] of dtype (bf16 or fp16), ld_x;  w [2 N, K] of dtype, ld_w: N gate rows, then N
 *     up rows; strides and bases as the linear layer's
 *   bias [2 N] of bias_dtype or NULL
 *   h [M, N] of out_dtype, ld_h
 *   z [M, 2 N] of dtype, contiguous, or NULL (kept for the gradient)
 * act: a moe_act; MOE_ACT_NONE gives g * u.  h is computed from z before z is rounded.
 * NaN and infinities give what the formulas do.  K == 0 is INVALID_ARG; M == 0 or N == 0
 * computes nothing and needs no ws.
 * ws: moe_gated_workspace_size(p) bytes, 256-byte aligned: the status word, as moe_linear's.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
typedef struct {
  int M, N, K;
  int dtype;      /* of x, w, z (and dx, dw): MOE_DTYPE_BF16 or MOE_DTYPE_F16 */
  int out_dtype;  /* of h (and dh) */
  int bias_dtype;
  int act;        /* moe_act */
  long long ld_x, ld_w, ld_h;
} moe_gated_problem;
size_t moe_gated_workspace_size(const moe_gated_problem* p);
moe_status moe_gated(const moe_gated_problem* p, const void* x, const void* w, const void* bias, void* h, void* z,
                     void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_gated_backward - dg = dh * u * act'(g), du = dh * act(g), dz = [dg, du], dx = dz W,
 * dw = dz^T x, dbias = the column sums of dz:
 *   dh [M, N] of out_dtype, ld_h;  x, w as in the forward;  z as the forward kept it
 *   dx [M, K] and dw [2 N, K] of dtype, contiguous;  dbias [2 N] fp32;  each may be NULL.
 * dz is rounded to dtype for the two products (the tensor cores' operand type), so that dx and
 * dw are some 1.4 times as far from exact ones as an unrounded dz would leave them; in fp16 one
 * past 65504 is infinite there (a loss scale has to stay below).  dbias sums dz unrounded in fp32,
 * in a fixed order.  M == 0 writes zeros to dw and dbias, N == 0 to dx; they need no ws.
 * ws: moe_gated_backward_workspace_size(p) bytes, 256-byte aligned, status word at its head,
 * cleared as moe_linear's, whichever outputs are wanted.  Errors: as moe_gated. */
size_t moe_gated_backward_workspace_size(const moe_gated_problem* p);
moe_status moe_gated_backward(const moe_gated_problem* p, const void* dh, const void* x, const void* w, const void* z,
                              void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- e4m3 with block scales
 * The format of MOE_FP8_BLOCK128 for dense layers: e4m3 codes with fp32 scales, one per (row,
 * 128 columns) for activations, one per 128 x 128 block for weights.  Rows of codes lie ld
 * bytes apart.
 *
 * moe_quantise - s = amax / 448 (fp32; 1 where that is 0), q = e4m3(x / s) of the IEEE quotient,
 * to nearest even:
 *   x [M, K] of dtype (f32, bf16, fp16), ld_x, any alignment
 *   q [M, K] codes out, ld_q;  scale [ceil(M / block_rows), ceil(K / 128)] fp32 out
 *   block_rows: 1 (activations) or 128 (weights); blocks end at M and K
 * A NaN has no part in amax and becomes a NaN code; an infinity makes its block's scale infinite
 * and its codes 0 or NaN, so that products with it are NaN.  No workspace.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
  int M, K;
  int dtype;      /* of x */
  int block_rows; /* 1 or 128 */
  long long ld_x, ld_q;
} moe_quantise_problem;
moe_status moe_quantise(const moe_quantise_problem* p, const void* x, uint8_t* q, float* scale, moe_stream_t stream);

/* moe_linear_fp8 - moe_linear on such operands (inference: there is no z and no gradient):
 *   z[m][n] = sum over groups kb of 128 of (x_scale[m][kb] w_scale[n / 128][kb]) (sum of x q in kb)
 *   y = alpha * act(z + bias) + residual, fp32 accumulation, one rounding
 * p->dtype is MOE_DTYPE_E4M3; out_dtype, bias_dtype, act, alpha and ld_y as in moe_linear
 *   x [M, K], w [N, K] codes, ld_x / ld_w: multiples of 16, bases 16-byte aligned; K is free
 *   x_scale [M, ceil(K / 128)], w_scale [ceil(N / 128), ceil(K / 128)] fp32
 * Every group's products are summed by themselves, so its scales need not be near the others'.  The product of
 * its two scales is rounded to fp32 first: below 1.2e-38 it loses bits, where it overflows it is infinite (times a
 * sum of 0 NaN).  Scales of 0 and of 2^-63 .. 2^63 (of amax 5e-17 .. 4e21) keep clear of both.
 * ws: moe_linear_fp8_workspace_size(p) bytes, 256-byte aligned: the status word, as moe_linear's.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
size_t moe_linear_fp8_workspace_size(const moe_linear_problem* p);
moe_status moe_linear_fp8(const moe_linear_problem* p, const void* x, const float* x_scale, const void* w,
                          const float* w_scale, const void* bias, const void* residual, void* y, void* ws,
                          size_t ws_bytes, moe_stream_t stream);

/* moe_gated_fp8 - moe_gated on such operands (no z, no gradient):
 *   p->dtype is MOE_DTYPE_E4M3;  x, x_scale as in moe_linear_fp8
 *   w [2 N, K] codes;  w_scale [2, ceil(N / 128), ceil(K / 128)]: the gate rows and the up rows
 *     are quantised apart
 *   h [M, N] of out_dtype, ld_h; h_scale NULL
 *   out_dtype MOE_DTYPE_E4M3: h in codes (ld_h a multiple of 16, base 16-byte aligned), h_scale
 *     [M, ceil(N / 128)] fp32: moe_quantise's rule on the unrounded fp32 h, the operand of a
 *     following moe_linear_fp8
 * ws: moe_gated_fp8_workspace_size(p) bytes, 256-byte aligned.  Errors: as moe_linear_fp8. */
size_t moe_gated_fp8_workspace_size(const moe_gated_problem* p);
moe_status moe_gated_fp8(const moe_gated_problem* p, const void* x, const float* x_scale, const void* w,
                         const float* w_scale, const void* bias, void* h, float* h_scale, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

/* ---------------------------------------------------------------- diagnostics
 * moe_read_device_status - synchronises `stream`, then returns the status
 * recorded on the device in the status word at the head of `ws` (MOE_OK,
 * MOE_ERR_DEVICE_TIMEOUT or MOE_ERR_DEVICE_BOUNDS), or MOE_ERR_CUDA if the
 * synchronisation failed.  Diagnostic only: it blocks, so it is never part of
 * the hot path.  Each moe_forward / moe_shuffle / moe_tile_map call resets the
 * word at its start. */
moe_status moe_read_device_status(const void* ws, moe_stream_t stream);

/* ---------------------------------------------------------------- stage timing
 * While profiling is on, each kernel launch of the entry points above is
 * bracketed by a pair of CUDA events recorded on the caller's stream (host-side
 * records only: nothing is synchronised or allocated on the device, and
 * launches on a stream that is being captured into a graph are not timed).
 *
 * moe_profile_start - clears earlier records and turns profiling on.
 * moe_profile_stop  - waits for the recorded events, writes one entry per
 *   kernel stage (in order of first launch) to out[0 .. max_stages-1], turns
 *   profiling off and returns the number of stages, or -1 if waiting on an
 *   event failed.  total_ms sums the stage's launches; launches counts them.
 * moe_profile_start_stage - the same, but only launches of the stage named
 *   `stage` are timed (NULL or "" times every stage).  Each event pair recorded
 *   between two kernels costs GPU time (about 2 us per stage on GB300), so a
 *   measurement of the whole call brackets only the kernel it needs.
 * Stage names: route_rank (with the per-tensor FP8 amax of x), scan_tiles,
 * scatter_gather, gateup_gemm, quant_h, down_gemm, combine (grouped path);
 * rd_prep, rd_gateup, rd_reduce, rd_down, combine (route-direct path); scatter,
 * tile_map, header_reset; route_ex, route_backward, norm_forward, norm_backward,
 * linear, linear_dz, linear_dx, linear_dw, linear_dx_dw, column_sums; gated, gated_dz
 * (a gated gradient's products are timed as the linear layer's), quantise, linear_fp8, gated_fp8. */
typedef struct {
  char name[32];
  double total_ms;
  int launches;
} moe_stage_time;
int moe_profile_start(void);
int moe_profile_start_stage(const char* stage);
int moe_profile_stop(moe_stage_time* out, int max_stages);

/* moe_status_string - static, NUL-terminated description of a status code. */
const char* moe_status_string(moe_status status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_MOE_H_ */
