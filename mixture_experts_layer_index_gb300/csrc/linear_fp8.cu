// Products of e4m3 operands with block scales (moe_linear_fp8, moe_gated_fp8) on the
// 5th-generation tensor cores:
//   z[m][n] = sum over kb of (sx[m][kb] sw[n / 128][kb]) (sum over the 128 k of kb of x[m][k] w[n][k])
// then bias, activation and residual, or the gate times the up projection, h optionally in
// e4m3 with a scale per (row, 128 columns): the next product's operand.
//
// Scales are any fp32 values, so the tensor cores cannot sum over more than one group of 128.
// Each 128-byte stage of the sum is a partial product of its own in tensor memory
// (tcgen05.mma kind::f8f6f4, four of K = 32), which sixteen epilogue warps read, multiply by
// its row's and block's scales and add to fp32 registers while the tensor cores fill the next
// partial ("promotion").  A row of x lies on a TMEM lane, so a thread's scale is the same for
// all columns of a weight block.  It is the product of two, rounded to fp32 first: taking care of products that are
// no normal numbers cost 3 to 17% in every form tried (the loop's registers are all in use), so it is the definition.
//
// Two forms of one kernel.  Large products: pairs of SMs, persistent, tiles of 256 x 256
// (linear_pair.cu has the reason: 64 bytes of operands per SM and clock instead of 96).  Others:
// one SM, tiles of 128 x BN, the sum split over the blocks of a cluster, which join their
// shares of the rows through shared memory in rank order: no workspace, no atomics, the same
// result every time.
//
// Bound by the promoting warps' loop, some 1200 clocks per stage of a 256 x 256 tile whose MMAs take
// 512: wait, four trips to tensor memory with as many rounds of additions, and the release.  Measured
// (16384 x 2048 x 4096: 131 us, 2.1 PFLOP/s, with a residual 149; gated, 16384 x 4096 x 2048, to bf16 252 us,
// 2.2 PFLOP/s, to e4m3 278; the bf16 layers' times for these are 149, 160 and 285): in trials at 131 us, without the additions 91 us, without the scales' loads 112.  So the
// loop is kept short: 16 columns on their way while 16 are added, a release that waits for no other
// access of the thread (with a release at cluster scope 269 us), the next partial's barrier looked at
// before the last additions, the next scales loaded behind the release, and registers that are moved here from the
// other warps, so that the linear form spills none (the gated one in pairs 24 bytes).  Slower in trials: eight warps with 128 accumulators and two
// buffers (139), 32 columns at a time (141), partials of 128 columns (170), the scales through shared
// memory (140 to 144), additions that are not packed in pairs (138).
#include "linear_fp8.cuh"
#include "linear_pair.cuh"

namespace moe {
namespace f8 {
namespace {

using namespace lin;

constexpr int BM = 128;   // rows of x per SM
constexpr int BKB = 128;  // codes of the sum per stage: one scale group
constexpr int QW = 4;     // epilogue warps per TMEM quadrant
constexpr int EPI_WARPS = 4 * QW;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
constexpr int MAX_SPLITS = 8;
constexpr int MAX_STAGES = 8;
constexpr int MAX_BUFS = 4;
// Registers per thread: 96 at launch (640 threads), then 56 for the four control warps and 104 for
// the sixteen that promote, no more in all.
constexpr int LAUNCH_REGS = 96, CONTROL_REGS = 56, EPI_REGS = 104;
static_assert(4 * CONTROL_REGS + EPI_WARPS * EPI_REGS <= (4 + EPI_WARPS) * LAUNCH_REGS, "registers of the launch");

template <int CG, int BN>
struct Shape {
  static constexpr int OP_A = BM * BKB;
  static constexpr int OP_B = BN / CG * BKB;
  static constexpr int STAGE = OP_A + OP_B;
  static constexpr int BUFS = BN >= 256 ? 2 : 4;  // partials in tensor memory
  static constexpr int STAGES = CG == 2 ? 5 : BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
  static constexpr int COLS = BN / QW;              // accumulators of an epilogue thread
  static constexpr int PITCH = BN + 4;              // fp32 values of a row on its way between threads
  // pairs: a store box per epilogue warp, or for e4m3 output the row maxima [2][16][32]
  static constexpr int BOX_OFFSET = STAGES * STAGE;
  static constexpr size_t SMEM = 1024 + BOX_OFFSET + (CG == 2 ? EPI_WARPS * BOX_BYTES : 0);
  static_assert(SMEM <= 227 * 1024 - 512, "shared memory of one block");
  static_assert(CG == 2 || BM * PITCH * 4 <= STAGES * STAGE, "a tile's sums lie over the ring");
};

struct Fp8Params {
  int M, N, nk;    // N: output columns
  int nR, nC;      // tiles
  int splits;      // blocks per tile (one SM)
  int half;        // gated: rows of the gate in w, else 0
  int blocks;      // scale rows of w (of the gate's half)
  const float* x_scale;  // [M][nk]
  const float* w_scale;  // [blocks][nk], gated [2][blocks][nk]
  int act, bias_dtype, out_dtype;
  float alpha;
  long long ld_y;
  const void* bias;
  const void* residual;
  void* y;
  float* h_scale;  // e4m3 output: [M][ceil(N / 128)]
  int y_tma;       // pairs: whether TMA stores the output
  int h_wide;      // pairs: whether rows of codes take stores of 32 bytes
  int sx_vec;      // rows of x_scale start at 16-byte boundaries
  DeviceHeader* hdr;
};

__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(map_rank(addr, rank))
               : "memory");
  return v;
}

// Tile t's row and column of tiles: groups of 8 row tiles, column by column within a group, so
// that the blocks in flight share both operands in L2.
__device__ __forceinline__ void tile_at(const Fp8Params& p, int t, int& r, int& c) {
  constexpr int GR = 8;
  const int group = t / (GR * p.nC), in_group = t - group * (GR * p.nC);
  const int rows_here = min(GR, p.nR - group * GR);
  c = in_group / rows_here;
  r = group * GR + in_group % rows_here;
}

__device__ __forceinline__ float vmax(float m, float v) { return fmaxf(m, fabsf(v)); }  // without a NaN's part

__device__ __forceinline__ void st_global_32(void* to, const uint32_t* a, const uint32_t* b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a[0]), "r"(a[1]), "r"(a[2]),
               "r"(a[3]), "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
               : "memory");
}

// Four values of a row from column c to an array of out_dtype; `n` of them exist.
template <typename T>
__device__ __forceinline__ void store4(T* to, const float (&v)[4], int n) {
  alignas(16) T out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = as_type<T>(v[i]);
  if (n >= 4 && reinterpret_cast<uintptr_t>(to) % (4 * sizeof(T)) == 0) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(out);
    else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(out);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) to[i] = out[i];
  }
}
__device__ __forceinline__ void store4(void* y, int dtype, size_t at, const float (&v)[4], int n) {
  if (dtype == MOE_DTYPE_F32) store4(static_cast<float*>(y) + at, v, n);
  else if (dtype == MOE_DTYPE_BF16) store4(static_cast<__nv_bfloat16*>(y) + at, v, n);
  else store4(static_cast<__half*>(y) + at, v, n);
}
__device__ __forceinline__ void add4(float (&v)[4], const void* p, int dtype, size_t at, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] += load_as_f32(p, dtype, at + i);
}

// The epilogue of a pair's tile for one warp: 32 rows from r0 (a row per thread), 64 columns from
// c0 (GATED: the gate's and the up projection's 32 columns of h from c0).
template <bool GATED>
__device__ __forceinline__ void pair_tile(const Fp8Params& p, const CUtensorMap* my, float (&acc)[64], uint8_t* box, int lane,
                                          int r0, int c0) {
  const bool row_in = r0 + lane < p.M;
  auto box_free = [&]() {
    if (lane == 0) bulk_wait_group_read0();
    __syncwarp();
  };
  auto store_box = [&](int c) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (r0 < p.M && c < p.N) tma_store_2d(my, smem_u32(box), c, r0);
      bulk_commit_group();
    }
  };
  if constexpr (GATED) {
    box_free();
    if (p.y_tma && p.out_dtype != MOE_DTYPE_F32) {
#pragma unroll
      for (int j = 0; j < 2; ++j) put_half_box(box, lane, j, p.out_dtype, &acc[16 * j]);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) put_box(box, lane, j, MOE_DTYPE_F32, *reinterpret_cast<float(*)[16]>(&acc[16 * j]));
    }
    if (p.y_tma) {
      store_box(c0);
    } else {
      __syncwarp();
      flush_box(box, lane, p.y, p.out_dtype, p.ld_y, nullptr, r0, p.M, c0, p.N);
    }
  } else {
    const bool wide = p.out_dtype == MOE_DTYPE_F32;
    const bool bias_wide = reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
    const bool residual_wide = reinterpret_cast<uintptr_t>(p.residual) % 16 == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float(&v)[16] = *reinterpret_cast<float(*)[16]>(&acc[16 * j]);
      const int c = c0 + 16 * j;
      if (p.bias) add16(v, p.bias, p.bias_dtype, c, p.N - c, bias_wide);
      act_all<16>(v, p.act);
      if (p.alpha != 1.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= p.alpha;
      }
      if (!p.y_tma) {
        if (j == 0) box_free();
        put_box(box, lane, j & 1, MOE_DTYPE_F32, v);
        if (j & 1) {
          __syncwarp();
          flush_box(box, lane, p.y, p.out_dtype, p.ld_y, p.residual, r0, p.M, c - 16, p.N);
        }
        continue;
      }
      if (p.residual && row_in)  // its rows are aligned as y's, which TMA stores
        add16(v, p.residual, p.out_dtype, static_cast<size_t>(r0 + lane) * p.ld_y + c, p.N - c, residual_wide);
      if (j == 0 || (wide && j == 2)) box_free();
      put_box(box, lane, wide ? j & 1 : j, p.out_dtype, v);
      if (j == 3 || (wide && j == 1)) store_box(wide ? c - 16 : c0);
    }
  }
}

// CG: SMs that share a tile's MMAs (1 or 2); BN: weight rows of a tile, GATED half of them gate
// rows, half the up rows of the same columns of h.  Warps: 0 loads, 1 issues MMAs, 2 owns
// tensor memory, 4-19 promote and finish.
template <int CG, int BN, bool GATED>
__global__ void __launch_bounds__(THREADS, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Fp8Params p) {
  using S = Shape<CG, BN>;
  constexpr int STAGES = S::STAGES, BUFS = S::BUFS, COLS = S::COLS;
  constexpr int OUT_COLS = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int TILE_ROWS = CG * BM;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * MAX_STAGES + 2 * MAX_BUFS + 1];
  __shared__ uint32_t tmem_slot[1];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // uniform, for the compiler too
  const uint32_t rank = cluster_rank();
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * MAX_STAGES;
  const uint32_t pfull0 = empty0 + 8 * MAX_STAGES, pempty0 = pfull0 + 8 * MAX_BUFS;
  const uint32_t done = pempty0 + 8 * MAX_BUFS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < BUFS; ++b) {
      mbar_init(pfull0 + 8 * b, 1);
      mbar_init(pempty0 + 8 * b, CG * EPI_WARPS);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 2) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(BUFS * BN)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(smem_u32(tmem_slot), BUFS * BN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // the other block's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dep_wait();
  dep_launch();
  // a wait that records a timeout lasts seconds: nothing of this launch is lost here
  if (blockIdx.x == 0 && threadIdx.x == 0) p.hdr->status = p.hdr->info = 0u;

  // A pair walks over tiles; on one SM a cluster has one tile, this block kb0 .. kb1 of its sum.
  const int tiles = p.nR * p.nC;
  const int first = CG == 2 ? static_cast<int>(blockIdx.x) >> 1 : static_cast<int>(blockIdx.x) / p.splits;
  const int step = CG == 2 ? static_cast<int>(gridDim.x) >> 1 : tiles;
  const int kb0 = CG == 2 ? 0 : static_cast<int>(static_cast<long long>(p.nk) * rank / p.splits);
  const int kb1 = CG == 2 ? p.nk : static_cast<int>(static_cast<long long>(p.nk) * (rank + 1) / p.splits);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    if (warp == 0) {
      // Uniform control flow: addresses stay in uniform registers, one lane issues, the next
      // slot's barrier is looked at ahead.
      const bool leader = elect_one();
      const uint32_t bar0 = CG == 2 ? map_rank(full0, 0) : full0, ring = smem_u32(smem);
      uint32_t stage = 0, phase = 1;
      int issued = 0;
      bool ok = true, ready = true;
      for (int t = first; ok && t < tiles; t += step) {
        int tr, tc;
        tile_at(p, t, tr, tc);
        const int r0 = tr * TILE_ROWS + (CG == 2 ? rank * BM : 0);
        const int c0 = tc * OUT_COLS + (CG == 2 ? rank * (GATED ? p.half : BM) : 0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!ready && !mbar_wait(empty0 + 8 * stage, phase, abort_flag, p.hdr, 0x710000u)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8 * stage, bar = bar0 + 8 * stage, a = ring + stage * S::STAGE, b = a + S::OP_A;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (leader) {
            const int k = kb * BKB;
            if constexpr (CG == 2) {
              if (rank == 0) mbar_arrive_expect_tx(full, 2 * S::STAGE);  // the bytes of both blocks
              tma_load_2d_pair(a, &tmA, k, r0, bar);
              tma_load_2d_pair(b, &tmB, k, c0, bar);
            } else {
              mbar_arrive_expect_tx(full, S::STAGE);
              tma_load_2d(a, &tmA, k, r0, full);
              tma_load_2d(b, &tmB, k, c0, full);
              if (GATED) tma_load_2d(b + S::OP_B / 2, &tmB, k, p.half + c0, full);
            }
          }
          __syncwarp();
          ++issued;
          ready = mbar_try_wait(empty0 + 8 * stage, phase);
        }
      }
      if (!ok && (CG == 1 || rank == 0) && leader) {  // let the copies already issued land before shared memory is given up
        for (int i = 0; i < min(issued, STAGES); ++i) {
          stage = (stage + STAGES - 1) % STAGES;
          if (stage == STAGES - 1) phase ^= 1;
          mbar_wait_quiet(full0 + 8 * stage, phase ^ 1, 50000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (CG == 1 || rank == 0) {
        const bool leader = elect_one();
        constexpr uint32_t idesc = make_idesc(0, 0, TILE_ROWS, BN);
        const uint32_t ring = smem_u32(smem);
        const OperandWalk walk(false);  // K-major: 32 codes are 32 bytes on, like 16 values of 16 bits
        uint32_t stage = 0, phase = 0, pb = 0, pphase = 1;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
          bool ready = mbar_try_wait(full0 + 8 * stage, phase);
          for (int kb = kb0; kb < kb1; ++kb) {
            if ((!ready && !mbar_wait(full0 + 8 * stage, phase, abort_flag, p.hdr, 0x720000u)) ||
                !mbar_wait(pempty0 + 8 * pb, pphase, abort_flag, p.hdr, 0x730000u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = ring + stage * S::STAGE, b = a + S::OP_A, empty = empty0 + 8 * stage;
            const uint32_t d = tmem + pb * BN, pfull = pfull0 + 8 * pb;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
            if (++pb == BUFS) {
              pb = 0;
              pphase ^= 1;
            }
            ready = kb + 1 < kb1 && mbar_try_wait(full0 + 8 * stage, phase);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {  // a fresh partial for this group of the sum
                if constexpr (CG == 2) mma_f8_pair(d, walk.at(a, kk), walk.at(b, kk), idesc, kk != 0);
                else mma_f8(d, walk.at(a, kk), walk.at(b, kk), idesc, kk != 0);
              }
              if constexpr (CG == 2) {
                mma_commit_pair(pfull);
                mma_commit_pair(empty);
              } else {
                mma_commit(pfull);
                mma_commit(empty);
              }
            }
            __syncwarp();
          }
        }
        if (leader) {
          if constexpr (CG == 2) mma_commit_pair(done);
          else mma_commit(done);
          mbar_wait_quiet(done, 0, 1000000000ull);
        }
      }
      __syncwarp();
    }
    __syncwarp();
    if constexpr (CG == 1) {
      if (p.splits > 1) {  // as the epilogue warps
        cluster_sync_all();
        cluster_sync_all();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int e = warp - 4, q = warp & 3, h = e >> 2;
    uint8_t* box = smem + S::BOX_OFFSET + e * BOX_BYTES;
    float* rowmax = reinterpret_cast<float*>(smem + S::BOX_OFFSET);
    const uint32_t free0 = CG == 2 ? map_rank(pempty0, 0) : pempty0;
    uint32_t pb = 0, pphase = 0, turn = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int tr, tc;
      tile_at(p, t, tr, tc);
      const int r0 = tr * TILE_ROWS + (CG == 2 ? static_cast<int>(rank) * BM : 0) + q * 32;  // this warp's rows
      const int c0 = tc * OUT_COLS + h * (OUT_COLS / QW);                                    // and columns
      // columns past the last stand in for it, rows likewise; neither is stored
      const float* sw = p.w_scale + static_cast<size_t>(min(c0 / 128, p.blocks - 1)) * p.nk;
      const float* su = sw + static_cast<size_t>(GATED ? p.blocks : 0) * p.nk;
      const float* sx = p.x_scale + static_cast<size_t>(min(r0 + lane, p.M - 1)) * p.nk;
      float acc[COLS];
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
      // Scales of x four groups at a time where rows allow it: a row per lane costs the L1 32 lines.
      float x4[4];
      auto load_sx = [&](int kb) {
        if (p.sx_vec) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(sx + kb));
          x4[0] = v.x; x4[1] = v.y; x4[2] = v.z; x4[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) x4[i] = __ldg(sx + min(kb + i, p.nk - 1));
        }
      };
      load_sx(kb0);
      if constexpr (CG == 2 && !GATED) {
        // the residual's part of this thread's row comes into L2 while the product is computed
        if (p.residual && r0 + lane < p.M && c0 < p.N) {
          const int es = p.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
          const uint8_t* row = static_cast<const uint8_t*>(p.residual) + (static_cast<size_t>(r0 + lane) * p.ld_y + c0) * es;
          const int bytes = min(COLS, p.N - c0) * es;
          for (int b = 0; b < bytes; b += 128) prefetch_l2(row + b);
          prefetch_l2(row + bytes - 1);
        }
      }
      float sw_kb = __ldg(sw + kb0), su_kb = GATED ? __ldg(su + kb0) : 0.0f;
      bool ready = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        const float f0 = x4[0] * sw_kb, f1 = GATED ? x4[0] * su_kb : f0;
        if (!__all_sync(0xffffffffu, ready)) {
          int good = 1;
          if (lane == 0) good = mbar_wait(pfull0 + 8 * pb, pphase, abort_flag, p.hdr, 0x740000u);
          if (!__shfl_sync(0xffffffffu, good, 0)) {
            ok = false;
            break;
          }
        }
        tc_fence_after();
        const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + pb * BN;
        auto column = [&](int j) {
          return tb + (!GATED ? h * COLS + j * 16
                       : j < COLS / 32 ? h * (COLS / 2) + j * 16
                                       : BN / 2 + h * (COLS / 2) + (j - COLS / 32) * 16);
        };
        float v[2][16];  // 16 columns on their way while 16 are added
        tmem_ld16(column(0), v[0]);
        tmem_ld_wait_regs16(v[0]);
#pragma unroll
        for (int j = 0; j < COLS / 16; ++j) {
          if (j + 1 < COLS / 16) {
            tmem_ld16(column(j + 1), v[(j + 1) & 1]);
          } else {  // the last columns are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CG == 2) mbar_arrive_cluster_relaxed(free0 + 8 * pb);
              else mbar_arrive(free0 + 8 * pb);
            }
            if (++pb == BUFS) {
              pb = 0;
              pphase ^= 1;
            }
            ready = mbar_test_wait(pfull0 + 8 * pb, pphase);
          }
          const float f = GATED && j >= COLS / 32 ? f1 : f0;
#pragma unroll
          for (int i = 0; i < 16; i += 2) fma2(acc[16 * j + i], acc[16 * j + i + 1], v[j & 1][i], v[j & 1][i + 1], f, f);
          if (j + 1 < COLS / 16) tmem_ld_wait_regs16(v[(j + 1) & 1]);
        }
        if (kb + 1 < kb1) {
          x4[0] = x4[1];
          x4[1] = x4[2];
          x4[2] = x4[3];
          if ((kb - kb0) % 4 == 3) load_sx(kb + 1);
          sw_kb = __ldg(sw + kb + 1);
          if (GATED) su_kb = __ldg(su + kb + 1);
        }
      }
      if (!ok) {
        if (CG == 2 && GATED && p.h_scale) quad_all(q, false);  // the quadrant's other warps go no further either
        break;
      }
      if constexpr (CG == 2) {
        if constexpr (GATED) {
          constexpr int H = COLS / 2;  // columns of h
          if (p.bias) {
            const bool bias_wide = reinterpret_cast<uintptr_t>(p.bias) % 16 == 0 && p.half % 8 == 0;
#pragma unroll
            for (int j = 0; j < COLS / 16; ++j) {
              const int c = c0 + 16 * (j % (H / 16));
              add16(*reinterpret_cast<float(*)[16]>(&acc[16 * j]), p.bias, p.bias_dtype,
                    (j >= H / 16 ? static_cast<size_t>(p.half) : 0) + c, p.N - c, bias_wide);
            }
          }
          act_all<H>(*reinterpret_cast<float(*)[H]>(&acc[0]), p.act);
#pragma unroll
          for (int i = 0; i < H; ++i) acc[i] *= acc[H + i];
          if (p.h_scale) {
            // the group's scale: the row's maximum over the quadrant's four warps
            float m = 0.0f;
            if (c0 + H <= p.N) {
#pragma unroll
              for (int i = 0; i < H; ++i) m = vmax(m, acc[i]);
            } else {
#pragma unroll
              for (int i = 0; i < H; ++i)
                if (c0 + i < p.N) m = vmax(m, acc[i]);
            }
            // two sets of maxima in turn: one barrier per tile
            float* maxima = rowmax + turn * (EPI_WARPS * 32);
            turn ^= 1;
            maxima[e * 32 + lane] = m;
            if (!quad_all(q, true)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int w = 0; w < QW; ++w) m = fmaxf(m, maxima[(q + 4 * w) * 32 + lane]);
            const GroupScale g(m);
            if (__any_sync(0xffffffffu, g.lift != 1.0f)) {
#pragma unroll
              for (int i = 0; i < H; ++i) acc[i] *= g.lift;
            }
            if (r0 + lane < p.M) {
              const size_t row = static_cast<size_t>(r0 + lane);
              uint8_t* to = static_cast<uint8_t*>(p.y) + row * p.ld_y + c0;
              uint32_t half[4];
#pragma unroll
              for (int j = 0; j < H / 16; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = codes4(&acc[16 * j + 4 * i], g);
                const int n = p.N - c0 - 16 * j;
                if (p.h_wide && c0 + H <= p.N) {  // a whole sector at once
                  if (j & 1) st_global_32(to + 16 * (j - 1), half, w);
#pragma unroll
                  for (int i = 0; i < 4; ++i) half[i] = w[i];
                } else if (n >= 16) {
                  reinterpret_cast<uint4*>(to)[j] = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                  for (int b = 0; b < 16; ++b)
                    if (b < n) to[16 * j + b] = static_cast<uint8_t>(w[b / 4] >> (8 * (b & 3)));
                }
              }
              if (h == 0) p.h_scale[row * ((p.N + 127) / 128) + c0 / 128] = g.s;
            }
          } else {
            pair_tile<true>(p, &tmY, acc, box, lane, r0, c0);
          }
        } else {
          pair_tile<false>(p, &tmY, acc, box, lane, r0, c0);
        }
      } else {
        // sums over the ring: every MMA has read it, and every load has landed
        float* part = reinterpret_cast<float*>(smem) + static_cast<size_t>(q * 32 + lane) * S::PITCH;
#pragma unroll
        for (int j = 0; j < COLS / 4; ++j) {
          const bool up = GATED && j >= COLS / 8;
          const int c = GATED ? (up ? BN / 2 - COLS / 2 : 0) + h * (COLS / 2) + j * 4 : h * COLS + j * 4;
          *reinterpret_cast<float4*>(part + c) = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        }
      }
    }
    if (CG == 2) {
      if (lane == 0) {
        bulk_wait_group0();
        // the last commit arrives in both blocks: the odd one stays until it has
        if (rank == 1 && warp == 4) mbar_wait_quiet(done, 0, 1000000000ull);
      }
      __syncwarp();
    }
    if constexpr (CG == 1) {
      // all of the tile's sums lie in shared memory
      if (p.splits > 1) cluster_sync_all();
      else asm volatile("bar.sync 1, %0;" ::"n"(EPI_WARPS * 32) : "memory");
      // this block's share of the rows, 4 columns (of the output) per thread
      int tr, tc;
      tile_at(p, first, tr, tc);
      const int rows = min(BM, p.M - tr * BM);
      const int per = (rows + p.splits - 1) / p.splits;
      const int begin = static_cast<int>(rank) * per, end = min(begin + per, rows);
      constexpr int LANES = OUT_COLS / 4 < 32 ? OUT_COLS / 4 : 32;  // threads of a row
      constexpr int PASSES = OUT_COLS / 4 / LANES;
      constexpr int GROUPS = EPI_WARPS * 32 / LANES;
      const int in_row = (static_cast<int>(threadIdx.x) - 128) % LANES;
      const uint32_t sums = smem_u32(smem);
      if (__all_sync(0xffffffffu, *abort_flag == 0)) {
        // whole warps leave the loop together where a row's maximum is shared
        for (int r = begin + (static_cast<int>(threadIdx.x) - 128) / LANES; r < end; r += GROUPS) {
          const int row = tr * BM + r;
#pragma unroll
          for (int i = 0; i < PASSES; ++i) {
            const int cc = (in_row + i * LANES) * 4, c = tc * OUT_COLS + cc, n = p.N - c;
            const uint32_t at = sums + (r * S::PITCH + cc) * 4;
            float v[4] = {}, u[4] = {};
            for (int k = 0; k < p.splits; ++k) {
              const uint32_t from = p.splits > 1 ? k : rank;
              const float4 a = ld_cluster_f32x4(at, from);
              v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
              if (GATED) {
                const float4 b = ld_cluster_f32x4(at + BN / 2 * 4, from);
                u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
              }
            }
            if (p.bias) {
              add4(v, p.bias, p.bias_dtype, c, n);
              if (GATED) add4(u, p.bias, p.bias_dtype, static_cast<size_t>(p.half) + c, n);
            }
            act_all<4>(v, p.act);
            const size_t to = static_cast<size_t>(row) * p.ld_y + c;
            if constexpr (GATED) {
              float m = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[k] *= u[k];
                if (k < n) m = vmax(m, v[k]);
              }
              if (OUT_COLS == 128 && p.h_scale) {
                m = warp_max(m);
                const GroupScale g(m);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] *= g.lift;
                const uint32_t w = codes4(v, g);
                uint8_t* h = static_cast<uint8_t*>(p.y) + to;
                if (n >= 4) {
                  *reinterpret_cast<uint32_t*>(h) = w;
                } else {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (k < n) h[k] = static_cast<uint8_t>(w >> (8 * k));
                }
                if (in_row == 0) p.h_scale[static_cast<size_t>(row) * ((p.N + 127) / 128) + tc] = g.s;
                continue;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] *= p.alpha;
              if (p.residual) add4(v, p.residual, p.out_dtype, to, n);
            }
            store4(p.y, p.out_dtype, to, v, n);
          }
        }
      }
      if (p.splits > 1) cluster_sync_all();  // no block leaves while another still reads its sums
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // neither block's barriers or tensor memory are in use any more
  if (warp == 2) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(BUFS * BN) : "memory");
    else tmem_dealloc(tmem, BUFS * BN);
  }
}

// Rows of codes, ld bytes apart, in boxes of 128 bytes x `rows`.
bool encode_codes(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, long long ld, uint32_t rows) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {BKB, rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int BN, bool GATED>
cudaError_t launch_shape(const Fp8Args& a, int splits, cudaStream_t s) {
  using Sh = Shape<CG, BN>;
  constexpr int OUT_COLS = GATED ? BN / 2 : BN;
  Fp8Params p{};
  p.M = a.M;
  p.N = a.N;
  p.nk = (a.K + BKB - 1) / BKB;
  p.nR = (a.M + CG * BM - 1) / (CG * BM);
  p.nC = (a.N + OUT_COLS - 1) / OUT_COLS;
  p.splits = splits;
  p.half = GATED ? a.N : 0;
  p.blocks = (a.N + 127) / 128;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.act = a.act;
  p.bias_dtype = a.bias_dtype;
  p.out_dtype = a.out_dtype;
  p.alpha = a.alpha;
  p.ld_y = a.ld_y;
  p.bias = a.bias;
  p.residual = a.residual;
  p.y = a.y;
  p.h_scale = a.h_scale;
  p.hdr = a.hdr;
  CUtensorMap ta, tb, ty;
  if (!encode_codes(&ta, a.x, a.K, a.M, a.ld_x, BM) ||
      !encode_codes(&tb, a.w, a.K, static_cast<uint64_t>(a.N) * (GATED ? 2 : 1), a.ld_w, CG == 2 ? BM : GATED ? BN / 2 : BN))
    return cudaErrorInvalidValue;
  ty = ta;
  p.y_tma = CG == 2 && !a.h_scale && storable(a.y, a.out_dtype, a.N, a.ld_y);
  if (p.y_tma && !encode_store(&ty, a.y, a.out_dtype, a.N, a.M, a.ld_y, GATED && a.out_dtype != MOE_DTYPE_F32 ? 64 : 128))
    return cudaErrorInvalidValue;
  static const cudaError_t attr = [] {
    cudaFuncAttributes f{};
    const cudaError_t e = cudaFuncGetAttributes(&f, linear_fp8_kernel<CG, BN, GATED>);
    if (e != cudaSuccess) return e;
    if (f.numRegs != LAUNCH_REGS) return cudaErrorInvalidConfiguration;  // the split of registers would not add up
    return cudaFuncSetAttribute(linear_fp8_kernel<CG, BN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Sh::SMEM));
  }();
  if (attr != cudaSuccess) return attr;
  p.h_wide = a.h_scale && reinterpret_cast<uintptr_t>(a.y) % 32 == 0 && a.ld_y % 32 == 0;
  p.sx_vec = p.nk % 4 == 0 && reinterpret_cast<uintptr_t>(a.x_scale) % 16 == 0 && p.nk % (4 * splits) == 0;
  const long long tiles = static_cast<long long>(p.nR) * p.nC;
  const int sms = num_sms();
  if (sms < 2) return cudaErrorNoDevice;
  const long long blocks = CG == 2 ? 2 * (tiles < sms / 2 ? tiles : sms / 2) : tiles * splits;
  cudaLaunchAttribute la[2];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = CG == 2 ? 2 : splits;
  la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
  la[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Sh::SMEM;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_fp8_kernel<CG, BN, GATED>, ta, tb, ty, p);
}

// About how long a launch takes (us), fitted to measurements on GB300 (weights in L2) of some 125 problems,
// 17 to 4096 rows, N and K of 256 to 8192, in every form: the form of the least estimate is on average 1%
// slower than the fastest one, 16% at most.
float pair_estimate(const Fp8Args& a) {
  const long long cols = a.gated ? 128 : 256;
  const long long tiles = (a.M + 255ll) / 256 * ((a.N + cols - 1) / cols);
  return 2.7f + (tiles + 75) / 76 * (0.52f * ((a.K + 127) / 128) + (a.h_scale ? 2.8f : 2.5f));
}
float single_estimate(const Fp8Args& a, int bn, int splits) {
  const long long cols = a.gated ? bn / 2 : bn;
  const long long blocks = (a.M + 127ll) / 128 * ((a.N + cols - 1) / cols) * splits;
  // a cluster's blocks lie in one group of SMs: clusters of 4 find some 144 of 152 SMs, of 8 some 120
  const int sms = splits == 8 ? 120 : splits == 4 ? 144 : 152;
  const int stages = ((a.K + 127) / 128 + splits - 1) / splits;
  const float wave = bn == 256 ? 9.0f + 0.434f * stages : bn == 128 ? 6.6f + 0.279f * stages : 5.5f + 0.269f * stages;
  float t = (blocks + sms - 1) / sms * wave - 2.5f + 1.3e-4f * (a.M < 128 ? a.M : 128) * bn / splits;
  if (splits > 1) t += 1.3f - 0.0054f * bn;
  for (int s = splits; s > 1; s /= 2) t += 0.58f;
  return t;
}

struct Choice {
  int bn, splits;  // bn 0: pairs
  float us;
};
Choice choose(const Fp8Args& a) {
  const int nk = (a.K + 127) / 128;
  Choice best{0, 1, pair_estimate(a)};
  for (int bn = a.h_scale ? 256 : a.gated ? 128 : 64; bn <= 256; bn *= 2)
    for (int splits = 1; splits <= MAX_SPLITS && splits <= nk; splits *= 2) {
      const float us = single_estimate(a, bn, splits);
      if (us < best.us) best = {bn, splits, us};
    }
  return best;
}

}  // namespace
}  // namespace f8

cudaError_t launch_linear_fp8(const Fp8Args& a, cudaStream_t s) {
  using namespace f8;
  stage_begin(a.gated ? "gated_fp8" : "linear_fp8", s);
  cudaError_t err;
  const bool few = takes_few(a);
  const Choice c = few ? Choice{} : choose(a);
  if (few) {
    err = launch_few(a, s);
  } else if (a.gated) {
    err = c.bn == 0 ? launch_shape<2, 256, true>(a, 1, s)
          : c.bn == 256 ? launch_shape<1, 256, true>(a, c.splits, s)
                        : launch_shape<1, 128, true>(a, c.splits, s);
  } else {
    err = c.bn == 0     ? launch_shape<2, 256, false>(a, 1, s)
          : c.bn == 256 ? launch_shape<1, 256, false>(a, c.splits, s)
          : c.bn == 128 ? launch_shape<1, 128, false>(a, c.splits, s)
                        : launch_shape<1, 64, false>(a, c.splits, s);
  }
  stage_end(s);
  return err;
}

}  // namespace moe
