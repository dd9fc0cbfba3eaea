// Parts shared by the block norms' forward (norm_forward.cu) and gradient
// (norm_backward.cu) kernels: how rows come in and go out, and block-wide sums.
//
// A block takes whole rows, a thread two runs of eight columns of a row, and blocks
// walk over rows.  (Sixteen columns per thread halve what the block-wide sums and
// the addresses cost per column against eight: the gradient kernel is bound by
// instructions as much as by memory.)  Where rows can be read asynchronously
// (cp.async), each block keeps a ring of rows in shared memory: the rows in flight
// cost no registers.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace norms {

constexpr int EPT = 8;   // columns per thread and run
constexpr int RUNS = 2;

// How a thread's columns of a row lie and come in.
//   VEC16: columns [run*8*NT + tid*8, + 8), 16-byte copies into the ring (widths, strides and
//          addresses that are multiples of 16 bytes)
//   WORD4: a warp takes 512 columns, its lane l columns (run*8 + i)*32 + l of them: whole
//          128-byte lines, and constant distances between a thread's columns; 4-byte
//          copies into the ring (fp32 rows)
//   SHIFT: columns like WORD4, of 16-bit rows at any address.  The 16-byte parts between a
//          row's first and last 16-byte boundary are copied by whichever threads are next, to
//          the same misalignment in a slot; the few elements around them go by way of
//          registers.  The gradient's form, 4202 x 2046 bf16: 73 -> 51 us against PLAIN; the
//          forward, which holds half as many rows in registers, gains nothing (17 us, 8192 x
//          1001: 16.5 -> 19), nor do fp32 rows against WORD4 (4099 x 1023: 29 -> 35 us).
//   PLAIN: columns like WORD4, or like VEC16 where the row allows it (`vec`), all of a row's
//          loads issued together when the row's turn comes: 16-bit rows at odd addresses, which
//          asynchronous copies of single elements do not take, and rows too long for a ring
// With VEC16 and WORD4 a thread copies exactly the columns it will read itself, so the ring
// needs no barrier; with SHIFT it takes one per row.
enum Access { VEC16, WORD4, SHIFT, PLAIN };

// Which of the threads of a row this one is.  Rows of up to 512 columns (SMALL) leave part
// of a warp idle if a block takes them one by one, and a block's fixed cost per row is
// then most of its time; there a group of 4, 8, 16 or 32 lanes takes a row (32768 x 64
// bf16: forward 21 -> 5 us, gradient 42 -> 12 us; 32768 x 512: 23.5 -> 20.3, 44 -> 42).  Odd
// rows gain nothing over 256 columns (32768 x 300: 26 -> 31 us) or where every row finds a
// free warp (600 x 151: 3.1 -> 3.9 us, but 19443 x 68: 17 -> 7.5), and stay one by one.
constexpr int SMALL_H = 32 * EPT * RUNS;
struct Own {
  int tid, nt;  // number and count of the row's threads
  int step;     // distance of a thread's columns in the layout of WORD4: 32, or nt < 32
  bool vec;
};
template <Access A>
__device__ __forceinline__ bool in_runs(const Own& me) {
  return A == VEC16 || (A == PLAIN && me.vec);
}
template <Access A>
__device__ __forceinline__ int col_of(int run, int i, const Own& me) {
  if (in_runs<A>(me)) return (run * me.nt + me.tid) * EPT + i;
  return (me.tid >> 5) * (32 * RUNS * EPT) + (me.tid & 31) + (run * EPT + i) * me.step;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most `depth - 1` of the newest rows are still on their way.
__device__ __forceinline__ void cp_async_wait(int depth) {
  if (depth >= 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Two fp32 values that packed instructions (mul / add / fma .rn.f32x2, each half rounded
// like the scalar one) work on: half the instructions of the elementwise parts.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ float halves_sum(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
constexpr int PPT = EPT / 2;  // pairs per run

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }

// Eight values from 16-byte aligned memory (16 or 32 bytes).
__device__ __forceinline__ void unpack(float (&v)[EPT], const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void unpack(float (&v)[EPT], const __nv_bfloat16* p) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(float (&v)[EPT], const __half* p) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void pack(float* p, const float (&v)[EPT]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void pack(__nv_bfloat16* p, const float (&v)[EPT]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(__half* p, const float (&v)[EPT]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// A thread's columns of the row at element `at` of p; 0 past column H.
template <typename T, Access A>
__device__ __forceinline__ void load_row(float (&v)[EPT], const void* p, size_t at, int run, int H, const Own& me) {
  const T* row = static_cast<const T*>(p) + at;
#pragma unroll
  for (int i = 0; i < EPT; ++i) v[i] = 0.0f;
  if (in_runs<A>(me)) {
    const int c = col_of<A>(run, 0, me);
    if (c < H) unpack(v, row + c);
  } else {
    T raw[EPT] = {};
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<A>(run, i, me);
      if (c < H) raw[i] = row[c];
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] = as_f32(raw[i]);
  }
}
template <typename T, Access A>
__device__ __forceinline__ void store_row(void* p, size_t at, int run, int H, const Own& me, const float (&v)[EPT]) {
  T* row = static_cast<T*>(p) + at;
  if (in_runs<A>(me)) {
    const int c = col_of<A>(run, 0, me);
    if (c < H) pack(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = col_of<A>(run, i, me);
      if (c < H) row[c] = rounded<T>(v[i]);
    }
  }
}

// A per-column vector (16-byte aligned where rows are read 16 bytes at a time) of one of the
// three types; `none` where there is no vector.
__device__ __forceinline__ float load_one(const void* p, int dtype, size_t i) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
template <Access A>
__device__ __forceinline__ void load_columns(float (&v)[EPT], const void* p, int dtype, int run, int H, const Own& me,
                                             float none) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] = none;
  } else if (dtype == MOE_DTYPE_F32) {
    load_row<float, A>(v, p, 0, run, H, me);
  } else if (dtype == MOE_DTYPE_BF16) {
    load_row<__nv_bfloat16, A>(v, p, 0, run, H, me);
  } else {
    load_row<__half, A>(v, p, 0, run, H, me);
  }
}

// A thread's columns of an fp32 vector in shared memory, for itself.
template <Access A>
__device__ __forceinline__ void put_shared(float* slot, int run, const Own& me, const float (&v)[EPT]) {
  if (in_runs<A>(me)) {
    pack(slot + col_of<A>(run, 0, me), v);
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) slot[col_of<A>(run, i, me)] = v[i];
  }
}

// The ring: slots of one row each of up to four arrays.
template <typename T, Access A>
__device__ __forceinline__ void copy_in(T* slot, const void* p, size_t at, int H, const Own& me) {
  const T* row = static_cast<const T*>(p) + at;
  constexpr int PER = 16 / sizeof(T);
#pragma unroll
  for (int r = 0; r < RUNS; ++r) {
    if (A == VEC16) {
      const int c = col_of<A>(r, 0, me);
      if (c < H)
#pragma unroll
        for (int q = 0; q < EPT / PER; ++q) cp_async16(slot + c + q * PER, row + c + q * PER);
    } else if (A == WORD4) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int c = col_of<A>(r, i, me);
        if (c < H) cp_async4(slot + c, row + c);
      }
    }
  }
}
// Zeros are put past column H of a slot once, so that reads need no test.
template <typename T, Access A>
__device__ __forceinline__ void clear_slot(T* slot, int H, const Own& me) {
  if (A == VEC16 || A == WORD4)
#pragma unroll
    for (int r = 0; r < RUNS; ++r)
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int c = col_of<A>(r, i, me);
        if (c >= H) slot[c] = T(0.0f);
      }
}
// SHIFT: elements of a slot for rows of up to `pitch` columns: the row, its shift (up to 14
// bytes) and eight zeros behind it.
template <typename T, Access A>
__host__ __device__ constexpr int slot_elements(int pitch) {
  return pitch + (A == SHIFT ? 48 / static_cast<int>(sizeof(T)) : 0);
}
// SHIFT: where in its slot a row starts.
template <typename T, Access A>
__device__ __forceinline__ int shift_of(const void* p, size_t at) {
  return A != SHIFT ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(p) + at * sizeof(T)) & 15) / static_cast<int>(sizeof(T));
}
// SHIFT: the column that threads 0 to 15 carry by register, before the first 16-byte boundary
// (threads 0 to 7) or from the last one on; -1: none.
template <typename T>
__device__ __forceinline__ int edge_column(int shift, int H) {
  constexpr int PER = 16 / sizeof(T);
  int head = (PER - shift) & (PER - 1);
  if (head > H) head = H;
  int tail = (shift + H) & (PER - 1);
  if (tail > H - head) tail = H - head;
  const int e = threadIdx.x & 7;
  return threadIdx.x >= 16 ? -1 : threadIdx.x < 8 ? (e < head ? e : -1) : (e < tail ? H - tail + e : -1);
}
template <typename T, Access A>
__device__ __forceinline__ void start_row(T* slot, T& edge, const void* p, size_t at, int H) {
  constexpr int PER = 16 / sizeof(T);
  const T* row = static_cast<const T*>(p) + at;
  const int shift = shift_of<T, A>(p, at);
  const int head = (PER - shift) & (PER - 1);
  const int parts = (shift + H) / PER - (shift + head) / PER;  // may be negative
#pragma unroll
  for (int i = 0; i < EPT * RUNS / PER; ++i) {
    const int q = i * blockDim.x + threadIdx.x;
    if (q < parts) cp_async16(slot + shift + head + q * PER, row + head + q * PER);
  }
  const int c = edge_column<T>(shift, H);
  if (c >= 0) edge = row[c];
}
// The elements at the ends of a row, and the zeros behind it (another row may have ended later).
template <typename T, Access A>
__device__ __forceinline__ void finish_row(T* slot, T edge, const void* p, size_t at, int H) {
  const int shift = shift_of<T, A>(p, at);
  const int c = edge_column<T>(shift, H);
  if (c >= 0) slot[shift + c] = edge;
  if (threadIdx.x >= 16 && threadIdx.x < 24) slot[shift + H + threadIdx.x - 16] = T(0.0f);
}
template <typename T, Access A>
__device__ __forceinline__ void copy_out(float (&v)[EPT], const T* slot, int r, const Own& me) {
  if (in_runs<A>(me)) {
    unpack(v, slot + col_of<A>(r, 0, me));
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] = as_f32(slot[col_of<A>(r, i, me)]);
  }
}

// The same as pairs.
__device__ __forceinline__ void pairs_of(F2 (&p)[PPT], const float (&v)[EPT]) {
#pragma unroll
  for (int i = 0; i < PPT; ++i) p[i] = f2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void values_of(float (&v)[EPT], const F2 (&p)[PPT]) {
#pragma unroll
  for (int i = 0; i < PPT; ++i) split(p[i], v[2 * i], v[2 * i + 1]);
}
template <typename T, Access A>
__device__ __forceinline__ void copy_out(F2 (&p)[PPT], const T* slot, int r, const Own& me) {
  float v[EPT];
  copy_out<T, A>(v, slot, r, me);
  pairs_of(p, v);
}
template <typename T, Access A>
__device__ __forceinline__ void load_row(F2 (&p)[PPT], const void* q, size_t at, int run, int H, const Own& me) {
  float v[EPT];
  load_row<T, A>(v, q, at, run, H, me);
  pairs_of(p, v);
}
template <typename T, Access A>
__device__ __forceinline__ void store_row(void* q, size_t at, int run, int H, const Own& me, const F2 (&p)[PPT]) {
  float v[EPT];
  values_of(v, p);
  store_row<T, A>(q, at, run, H, me, v);
}
// v = 0 for columns past H (after a mean was taken off).
template <Access A>
__device__ __forceinline__ void clear_past(F2 (&p)[PPT], int run, int H, const Own& me) {
  if (in_runs<A>(me)) {
    if (col_of<A>(run, 0, me) >= H)
#pragma unroll
      for (int i = 0; i < PPT; ++i) p[i] = f2(0.0f);
  } else {
    float v[EPT];
    values_of(v, p);
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      if (col_of<A>(run, i, me) >= H) v[i] = 0.0f;
    pairs_of(p, v);
  }
}

// Sums of N (1 or 4) values over a block of up to MAXT threads, for every thread, in a
// fixed order: a butterfly in each warp, then one over the warps' sums, which every
// warp reads from shared memory.  For four values the lanes trade values on the way (6
// shuffles instead of 20).  Two buffers taken in turn: a warp can be at most one sum
// ahead of the others' reads.  buf: zeroed before the first use.
template <int N, int MAXT>
struct BlockSum {
  static constexpr int W = MAXT / 32 < 8 ? 8 : MAXT / 32;
  float (*buf)[N][W];
  int turn;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if constexpr (N == 4) {
      const bool hi = lane & 16, mid = lane & 8;
      float a0 = hi ? v[2] : v[0], a1 = hi ? v[3] : v[1];
      a0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
      a1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
      float b = mid ? a1 : a0;
      b += __shfl_xor_sync(0xffffffffu, mid ? a0 : a1, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
      if ((lane & 7) == 0) buf[turn][lane >> 3][warp] = b;
      __syncthreads();
      // eight lanes per value
      const float* from = &buf[turn][lane >> 3][(lane & 7) * (W / 8)];
      b = from[0];
#pragma unroll
      for (int i = 1; i < W / 8; ++i) b += from[i];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __shfl_sync(0xffffffffu, b, j * 8);
    } else {
      float b = v[0];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
      if (lane == 0) buf[turn][0][warp] = b;
      __syncthreads();
      b = buf[turn][0][lane & (W - 1)];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
      v[0] = b;
    }
    turn ^= 1;
  }
};

// The same over the `nt` lanes (a power of two, at least 4) of a row's group.
template <int N>
struct GroupSum {
  int nt;
  __device__ __forceinline__ void operator()(float (&v)[N]) const {
    if constexpr (N == 4) {
      const bool hi = threadIdx.x & (nt >> 1), mid = threadIdx.x & (nt >> 2);
      float a0 = hi ? v[2] : v[0], a1 = hi ? v[3] : v[1];
      a0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], nt >> 1);
      a1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], nt >> 1);
      float b = mid ? a1 : a0;
      b += __shfl_xor_sync(0xffffffffu, mid ? a0 : a1, nt >> 2);
      for (int o = nt >> 3; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __shfl_sync(0xffffffffu, b, j * (nt >> 2), nt);
    } else {
      for (int o = nt >> 1; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
};

template <bool SMALL, int N, int MAXT>
struct SumOf {
  using type = BlockSum<N, MAXT>;
  static __device__ __forceinline__ type make(float (*buf)[N][type::W], int) { return type{buf, 0}; }
};
template <int N, int MAXT>
struct SumOf<true, N, MAXT> {
  using type = GroupSum<N>;
  static __device__ __forceinline__ type make(float (*)[N][BlockSum<N, MAXT>::W], int lanes) { return type{lanes}; }
};

// 1 / sqrt of the second moment, whose sum over H columns is given, plus eps.  rsqrtf
// is within 2 ulp, a tenth of the instructions of a square root and a division.
__device__ __forceinline__ float inv_std(float sum, float inv_h, float eps) { return rsqrtf(sum * inv_h + eps); }

// Threads of a block for rows of H columns.
inline int norm_threads(int H) {
  const int t = (H + EPT * RUNS - 1) / (EPT * RUNS);
  return (t + 31) / 32 * 32;
}
inline bool takes_small(const NormArgs& a) { return a.vec ? a.H <= SMALL_H : a.H <= SMALL_H / 2 && a.T > 8 * 152; }
// The same for SMALL: lanes per row, and threads of a block, fewer where that leaves SMs idle.
inline int norm_lanes(int H) {
  int n = 4;
  while (n * EPT * RUNS < H) n *= 2;
  return n;
}
inline int small_threads(int T, int lanes) {
  int n = 128;
  while (n > 32 && static_cast<long long>(T) * lanes < 152ll * n) n /= 2;
  return n;
}
inline size_t norm_pitch(int H) { return static_cast<size_t>(H + EPT - 1) / EPT * EPT; }
// Elements of a row or vector in shared memory.
__host__ __device__ inline int slot_pitch(int threads) {
  return threads * EPT * RUNS;
}

}  // namespace norms
}  // namespace moe
