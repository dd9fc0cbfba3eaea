// The linear layer's products at sizes that fill the GPU: out[r][c] in tiles of
// 256 x 256 by pairs of SMs (tcgen05.mma with cta_group::2, M = 256, N = 256).
//
// Each block of a pair (a cluster of two) loads 128 rows r and 128 columns c per
// stage, 32 KB instead of the 48 KB of a 128 x 256 tile on one SM for the same
// arithmetic, because the tensor cores of both read both halves of the column
// operand.  A 128 x 256 tile on one SM asks 96 bytes per clock and SM of the L2 at the full
// MMA rate; the pair asks 64.  The even block issues the MMAs for both; operand loads
// of both count on its barriers, and its commits arrive on the barriers of both.
//
// Persistent pairs walk over the tiles.  Rows r lie on the TMEM lanes, 128 per
// block, 2 x 256 accumulator columns, so that the epilogue of one tile
// overlaps the MMAs of the next.  Warps: 0 loads, 1 issues MMAs (even block), 2
// owns TMEM, 4-19 run the epilogue (four warps per 32 lanes, 64 columns each): 32
// columns at a time are loaded from TMEM, finished in fp32, rounded once, staged in
// shared memory as a 128-byte-swizzled box of 32 rows and stored by TMA, which
// clips the edges.  A tile's whole sum is one accumulator's, whatever the output's
// type (tensor memory holds two tiles), rounded in fp32 at every step of it.
//
// Bound by the tensor cores: 16384 x 8192 x 2048 bf16 takes 294 us, 1.87 PFLOP/s (a library
// product reaches 1.95 in short runs, 1.74 under the power limit).  With a GELU and its
// argument kept 400 us: 16 warps' worth of epilogue instructions beside the MMAs and a
// second output; a residual or an odd width (plain stores) cost similar shares.
#include "linear.cuh"

namespace moe {
namespace lin {
namespace {

constexpr int TILE = 256;       // rows and columns of a pair's tile
constexpr int HALF = 128;       // rows (and loaded columns) of one block
constexpr int STAGES = 5;
constexpr int OP_BYTES = HALF * BK * 2;
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int EPI_WARPS = 16;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
constexpr int BOX_BYTES = 32 * 128;            // 32 rows of 128 bytes
constexpr int NUM_BARS = 2 * STAGES + 4 + 1;
constexpr int EPI_COLS = TILE / (EPI_WARPS / 4);  // columns per epilogue warp
static_assert(EPI_COLS == 64, "an epilogue warp fills one box of 16-bit values");
// ring | one box per epilogue warp | barriers
constexpr int BOX_OFFSET = STAGES * STAGE_BYTES;
constexpr int BAR_OFFSET = BOX_OFFSET + EPI_WARPS * BOX_BYTES;
constexpr size_t SMEM_BYTES = 1024 + BAR_OFFSET + 256;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one block");

// One product of a launch.
struct PairProduct {
  int R, C, nk;
  int nR, nC;
  int a_mn, b_mn;  // operand rows / cols contiguous along r / c
};
// A launch computes one product, or two whose epilogues differ in their output only
// (the gradient's two), `prod[0]` the one with the longer sum.
struct PairParams {
  PairProduct prod[2];
  int tiles[2];
  int ratio;  // tiles of prod[1] that take about as long as one of prod[0]
  int type;
  int y_tma, z_tma;  // whether TMA can store the output (16-byte aligned rows)
  Epilogue ep;
  void* y[2];        // per product
  int reset_status;
  DeviceHeader* hdr;
};
struct PairMaps {
  CUtensorMap a, b, y;
};

// The i-th tile of a pair: (product, tile), false after its last.  Tiles of prod[0] go
// round the pairs first; pairs left without one in the last round take `ratio` tiles of
// prod[1] instead; the rest of prod[1] goes round again.  So the two products of a
// gradient, each of which would leave part of the GPU idle in its last round, share one.
__device__ __forceinline__ bool pair_item(const PairParams& p, int pair, int npairs, int i, int& prod, int& tile) {
  const int heavy = pair < p.tiles[0] ? (p.tiles[0] - pair - 1) / npairs + 1 : 0;
  prod = 0;
  tile = pair + i * npairs;
  if (i < heavy) return true;
  prod = 1;
  i -= heavy;
  const int last = p.tiles[0] % npairs;  // pairs with a tile of the last round
  int gap = (npairs - last) * p.ratio;
  if (pair >= last) {
    if (i < p.ratio) {
      tile = pair - last + i * (npairs - last);
      return tile < p.tiles[1];
    }
    i -= p.ratio;
  }
  if (gap > p.tiles[1]) gap = p.tiles[1];
  tile = gap + pair + i * npairs;
  return tile < p.tiles[1];
}

// ------------------------------------------------------------------ two-SM forms
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// A load into this block's shared memory that counts on a barrier of the pair's even block.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both blocks once the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// Tile t's first row and column: groups of 8 row tiles, column by column within a
// group, so that the pairs in flight share both operands in L2.
__device__ __forceinline__ void tile_origin(const PairProduct& p, int t, int& r0, int& c0) {
  constexpr int GR = 8;
  const int group = t / (GR * p.nC), in_group = t - group * (GR * p.nC);
  const int rows_here = min(GR, p.nR - group * GR);
  c0 = in_group / rows_here * TILE;
  r0 = (group * GR + in_group % rows_here) * TILE;
}

// 16 values (columns c.. of one row) into row `lane` of a swizzled box: 16-byte chunk j of a
// row sits at chunk j ^ (lane & 7).  `part`: which 16 of the box's columns.
__device__ __forceinline__ void put_box(uint8_t* box, int lane, int part, int dtype, const float (&v)[16]) {
  uint8_t* row = box + lane * 128;
  if (dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(row + (((part * 4 + j) ^ (lane & 7)) << 4)) =
          make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
      if (dtype == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 b = __floats2half2_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      *reinterpret_cast<uint4*>(row + (((part * 2 + j) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Columns c.. c + 31 of a box of fp32 values (32 rows from r0) to an array whose rows TMA
// cannot store: a row at a time, one lane per column, plus the residual's values.  Not
// inlined: its registers would be spilled from the paths that TMA stores.
template <typename T>
__device__ __forceinline__ void flush_box_as(const uint8_t* box, int lane, T* out, long long ld, const T* residual,
                                             int r0, int R, int c, int C) {
  const int rows = c + lane < C ? min(32, R - r0) : 0;
  const size_t at = static_cast<size_t>(r0) * ld + c + lane;
  out += at;
  if (residual) residual += at;
#pragma unroll 1
  for (int r = 0; r < rows; r += 16) {
    T u[16] = {};
    if (residual) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (r + i < rows) u[i] = residual[i * ld];
      residual += 16 * ld;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (r + i < rows) {
        float v = *reinterpret_cast<const float*>(box + (r + i) * 128 + (((lane >> 2) ^ ((r + i) & 7)) << 4) + (lane & 3) * 4);
        if (residual) v += as_float(u[i]);
        out[i * ld] = as_type<T>(v);
      }
    out += 16 * ld;
  }
  __syncwarp();  // the box may be written again
}
__device__ __noinline__ void flush_box(const uint8_t* box, int lane, void* out, int dtype, long long ld,
                                          const void* residual, int r0, int R, int c, int C) {
  if (dtype == MOE_DTYPE_F32)
    flush_box_as(box, lane, static_cast<float*>(out), ld, static_cast<const float*>(residual), r0, R, c, C);
  else if (dtype == MOE_DTYPE_BF16)
    flush_box_as(box, lane, static_cast<__nv_bfloat16*>(out), ld, static_cast<const __nv_bfloat16*>(residual), r0, R, c, C);
  else
    flush_box_as(box, lane, static_cast<__half*>(out), ld, static_cast<const __half*>(residual), r0, R, c, C);
}

// v[i] += p[at + i], 16 values of which `n` exist; `wide`: p + at is 16-byte aligned.
__device__ __forceinline__ void add16(float (&v)[16], const void* p, int dtype, size_t at, int n, bool wide) {
  if (n < 16 || !wide) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i] += load_as_f32(p, dtype, at + i);
  } else if (dtype == MOE_DTYPE_F32) {
    float4 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[4 * j] += f[j].x; v[4 * j + 1] += f[j].y; v[4 * j + 2] += f[j].z; v[4 * j + 3] += f[j].w;
    }
  } else {
    uint4 raw[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) raw[j] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at)[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = dtype == MOE_DTYPE_BF16
                             ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]))
                             : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[8 * j + 2 * i] += f.x;
        v[8 * j + 2 * i + 1] += f.y;
      }
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    linear_pair_kernel(const __grid_constant__ PairMaps m0, const __grid_constant__ PairMaps m1,
                       const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFFSET);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * STAGES), tempty0 = smem_u32(bars + 2 * STAGES + 2);
  const uint32_t mma_done = smem_u32(bars + 2 * STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      // the epilogue warps of both blocks, and the warps that fetch a residual ahead
      mbar_init(tempty0 + 8 * a, 2 * (EPI_WARPS + (p.ep.residual ? 1 : 0)));
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&m0.a);
    prefetch_tensormap(&m0.b);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2 * TILE)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other block's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dep_wait();
  dep_launch();
  // a wait that records a timeout lasts seconds: nothing of this launch is lost here
  if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) p.hdr->status = p.hdr->info = 0u;

  const int npairs = static_cast<int>(gridDim.x) >> 1, pair = static_cast<int>(blockIdx.x) >> 1;

  if (warp == 0) {
    // Like the MMA warp: uniform control, one lane issues, the next slot's barrier is
    // looked at ahead.
    const bool leader = elect_one();
    const uint32_t lead_full0 = map_rank(full0, 0), ring = smem_u32(smem);
    uint32_t stage = 0, phase = 1;
    int issued = 0;
    bool ok = true;
    bool ready = mbar_try_wait(empty0, phase);
    int prod, tile;
    for (int i = 0; ok && pair_item(p, pair, npairs, i, prod, tile); ++i) {
      const PairProduct& q = p.prod[prod];
      const CUtensorMap* ma = prod ? &m1.a : &m0.a;
      const CUtensorMap* mb = prod ? &m1.b : &m0.b;
      const bool a_mn = q.a_mn, b_mn = q.b_mn;
      int r0, c0;
      tile_origin(q, tile, r0, c0);
      r0 += rank * HALF;
      c0 += rank * HALF;
      const int nk = q.nk;
      for (int kb = 0; kb < nk; ++kb) {
        if (!ready && !mbar_wait(empty0 + 8 * stage, phase, abort_flag, p.hdr, 0x610000u)) {
          ok = false;
          break;
        }
        const uint32_t full = full0 + 8 * stage, bar = lead_full0 + 8 * stage;
        const uint32_t a = ring + stage * STAGE_BYTES, b = a + OP_BYTES;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (leader) {
          // the even block's barrier expects the bytes of both blocks
          if (rank == 0) mbar_arrive_expect_tx(full, 2 * STAGE_BYTES);
          const int k = kb * BK;
          if (a_mn) {
            tma_load_2d_pair(a, ma, r0, k, bar);
            tma_load_2d_pair(a + OP_BYTES / 2, ma, r0 + 64, k, bar);
          } else {
            tma_load_2d_pair(a, ma, k, r0, bar);
          }
          if (b_mn) {
            tma_load_2d_pair(b, mb, c0, k, bar);
            tma_load_2d_pair(b + OP_BYTES / 2, mb, c0 + 64, k, bar);
          } else {
            tma_load_2d_pair(b, mb, k, c0, bar);
          }
        }
        __syncwarp();
        ++issued;
        ready = mbar_try_wait(empty0 + 8 * stage, phase);
      }
    }
    if (!ok && rank == 0 && leader) {  // let the copies already issued land before shared memory is given up
      for (int i = 0; i < min(issued, STAGES); ++i) {
        stage = (stage + STAGES - 1) % STAGES;
        if (stage == STAGES - 1) phase ^= 1;
        mbar_wait_quiet(full0 + 8 * stage, phase ^ 1, 50000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // The whole warp walks the loop, so that addresses and descriptors stay in uniform
    // registers; one lane issues.  The next stage's barrier is looked at before this
    // stage's MMAs are issued: the look takes longer than an MMA.
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t ring = smem_u32(smem);
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      int prod, tile;
      for (int i = 0; ok && pair_item(p, pair, npairs, i, prod, tile); ++i) {
        const bool a_mn = p.prod[prod].a_mn, b_mn = p.prod[prod].b_mn;
        const int nk = p.prod[prod].nk;
        const uint32_t idesc =
            make_idesc(p.type, p.type, TILE, TILE) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        const OperandWalk wa(a_mn), wb(b_mn);
        if (!mbar_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, p.hdr, 0x620000u)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * TILE;
        bool ready = mbar_try_wait(full0 + 8 * stage, phase);
        for (int kb = 0; kb < nk; ++kb) {
          if (!ready && !mbar_wait(full0 + 8 * stage, phase, abort_flag, p.hdr, 0x630000u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = ring + stage * STAGE_BYTES, empty = empty0 + 8 * stage;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          ready = kb + 1 < nk && mbar_try_wait(full0 + 8 * stage, phase);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16_pair(d, wa.at(a, kk), wb.at(a + OP_BYTES, kk), idesc, (kb | kk) != 0);
            mma_commit_pair(empty);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) mma_commit_pair(tfull0 + 8 * acc);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (leader) {
        mma_commit_pair(mma_done);
        mbar_wait_quiet(mma_done, 0, 1000000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // The residual of a tile is fetched into L2 while the tile before it is finished, so
    // that the epilogue's loads do not wait for memory.  Its wait is by parity like the
    // epilogue's, so it too says when it has seen a tile, before which the accumulator is not
    // filled again: two completions it had not looked at would read as none.
    if (p.ep.residual) {
      const size_t es = p.ep.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
      const uint32_t lead_tempty0 = map_rank(tempty0, 0);
      uint32_t acc = 0, acc_phase = 0;
      int prod, tile;
      for (int i = 0; pair_item(p, pair, npairs, i, prod, tile); ++i) {
        int r0, c0;
        tile_origin(p.prod[prod], tile, r0, c0);
        r0 += rank * HALF;
        const size_t row_bytes = static_cast<size_t>(min(TILE, p.prod[prod].C - c0)) * es;
        for (int r = lane; r < min(HALF, p.prod[prod].R - r0); r += 32) {
          const uint8_t* row = static_cast<const uint8_t*>(p.ep.residual) + (static_cast<size_t>(r0 + r) * p.ep.ld_y + c0) * es;
          for (size_t b = 0; b < row_bytes; b += 128) prefetch_l2(row + b);
        }
        int good = 1;
        if (lane == 0) {
          good = mbar_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.hdr, 0x650000u);
          if (good) mbar_arrive_cluster(lead_tempty0 + 8 * acc);
        }
        if (!__shfl_sync(0xffffffffu, good, 0)) break;
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
  } else if (warp >= 4) {
    const int e = warp - 4, q = warp & 3, h = e >> 2;
    uint8_t* box = smem + BOX_OFFSET + e * BOX_BYTES;
    const uint32_t lead_tempty0 = map_rank(tempty0, 0);
    const Epilogue& ep = p.ep;
    const bool wide = ep.out_dtype == MOE_DTYPE_F32;
    const bool plain = p.y_tma && !wide && !ep.bias && !ep.residual && !ep.z && ep.act == MOE_ACT_NONE && ep.alpha == 1.0f;
    const bool bias_wide = reinterpret_cast<uintptr_t>(ep.bias) % 16 == 0;
    const bool residual_wide = reinterpret_cast<uintptr_t>(ep.residual) % 16 == 0;
    uint32_t acc = 0, acc_phase = 0;
    // the box may be written again once the store that read it has done so
    auto box_free = [&]() {
      if (lane == 0) bulk_wait_group_read0();
      __syncwarp();
    };
    int prod, tile;
    for (int i = 0; pair_item(p, pair, npairs, i, prod, tile); ++i) {
      const int R = p.prod[prod].R, C = p.prod[prod].C;
      const CUtensorMap* my = prod ? &m1.y : &m0.y;
      int r0, c0;
      tile_origin(p.prod[prod], tile, r0, c0);
      r0 += rank * HALF + q * 32;  // this warp's rows and columns
      c0 += h * EPI_COLS;
      int good = 1;
      if (lane == 0) good = mbar_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.hdr, 0x640000u);
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) break;
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE + h * EPI_COLS;
      const bool row_in = r0 + lane < R;
      // sum + bias of 16 columns from c0 + j * 16
      auto load_z = [&](int j, float(&v)[16]) {
        tmem_ld16(tb + j * 16, v);
        tmem_ld_wait_regs16(v);
        if (ep.bias) add16(v, ep.bias, ep.bias_dtype, c0 + j * 16, C - c0 - j * 16, bias_wide);  // same for every lane
      };
      auto store_box = [&](const CUtensorMap* map, int c) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (r0 < R && c < C) tma_store_2d(map, smem_u32(box), c, r0);
          bulk_commit_group();
        }
      };
      if (plain) {  // nothing to compute: all 64 columns at once, a short chain for short sums
        float v[2][32];
        tmem_ld32(tb, v[0]);
        tmem_ld32(tb + 32, v[1]);
        tmem_ld_wait_regs(v[0]);
        tmem_ld_wait_regs(v[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(lead_tempty0 + 8 * acc);
          bulk_wait_group_read0();
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) put_box(box, lane, j, ep.out_dtype, *reinterpret_cast<float(*)[16]>(&v[j >> 1][(j & 1) * 16]));
        store_box(my, c0);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
        continue;
      }
      // z goes out first: its store reads the box while the activation is computed (the
      // accumulator is read a second time instead of being kept)
      if (ep.z) {
        box_free();
#pragma unroll 2
        for (int j = 0; j < 4; ++j) {
          float v[16];
          load_z(j, v);
          if (p.z_tma) {
            put_box(box, lane, j, ep.z_dtype, v);
          } else {
            put_box(box, lane, j & 1, MOE_DTYPE_F32, v);
            if (j & 1) {
              __syncwarp();
              flush_box(box, lane, ep.z, ep.z_dtype, ep.ld_z, nullptr, r0, R, c0 + (j - 1) * 16, C);
            }
          }
        }
        if (p.z_tma) store_box(&tmZ, c0);
      }
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + j * 16;
        float v[16];
        load_z(j, v);
        if (j == 3) {  // this warp's accumulator columns are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8 * acc);
        }
        act_all<16>(v, ep.act);
        if (ep.alpha != 1.0f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= ep.alpha;
        }
        if (!p.y_tma) {
          if (j == 0) box_free();
          put_box(box, lane, j & 1, MOE_DTYPE_F32, v);
          if (j & 1) {
            __syncwarp();
            flush_box(box, lane, p.y[prod], ep.out_dtype, ep.ld_y, ep.residual, r0, R, c - 16, C);
          }
          continue;
        }
        if (ep.residual && row_in)  // its rows are aligned as y's, which TMA stores
          add16(v, ep.residual, ep.out_dtype, static_cast<size_t>(r0 + lane) * ep.ld_y + c, C - c, residual_wide);
        if (j == 0 || (wide && j == 2)) box_free();
        put_box(box, lane, wide ? j & 1 : j, ep.out_dtype, v);
        if (j == 3 || (wide && j == 1)) store_box(my, wide ? c - 16 : c0);
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0) {
      bulk_wait_group0();
      // the last commit arrives in both blocks: the odd one stays until it has
      if (rank == 1 && warp == 4) mbar_wait_quiet(mma_done, 0, 1000000000ull);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither block's barriers or tensor memory are in use any more
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * TILE) : "memory");
  }
}

// A store map: boxes of 32 rows of 128 bytes.
bool encode_store(CUtensorMap* map, void* base, int dtype, int cols, int rows, long long ld) {
  EncodeTiledFn fn = get_encode_tiled();
  if (!fn) return false;
  const uint32_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  const cuuint32_t box[2] = {128 / es, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = dtype == MOE_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, type, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool storable(const void* base, int dtype, long long ld) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld * (dtype == MOE_DTYPE_F32 ? 4 : 2) % 16 == 0;
}

bool encode_product(PairMaps* m, PairProduct* pp, const Product& q) {
  pp->R = q.R;
  pp->C = q.C;
  pp->nk = (q.K + BK - 1) / BK;
  pp->nR = (q.R + TILE - 1) / TILE;
  pp->nC = (q.C + TILE - 1) / TILE;
  pp->a_mn = q.rows_mn;
  pp->b_mn = q.cols_mn;
  return encode(&m->a, q.rows.base, q.type, q.rows.inner, q.rows.outer, q.rows.ld, 64, q.rows_mn ? 64 : HALF) &&
         encode(&m->b, q.cols.base, q.type, q.cols.inner, q.cols.outer, q.cols.ld, 64, q.cols_mn ? 64 : HALF) &&
         (!storable(q.ep.y, q.ep.out_dtype, q.ep.ld_y) ||
          encode_store(&m->y, q.ep.y, q.ep.out_dtype, q.C, q.R, q.ep.ld_y));
}

}  // namespace

// Measured on GB300: 4 us of launch, set-up and drain, 0.30 us per stage of a tile, and the
// epilogue of a tile, of which all but the last overlaps the next tile's stages: 3.5 us,
// and more with an activation, z, a residual, or rows that TMA cannot store.
float pair_estimate(const Product& q) {
  const long long tiles = static_cast<long long>((q.R + TILE - 1) / TILE) * ((q.C + TILE - 1) / TILE);
  const float stages = 0.30f * ((q.K + BK - 1) / BK);
  float epilogue = 3.5f;
  if (q.ep.act != MOE_ACT_NONE) epilogue += 1.0f;
  if (q.ep.residual) epilogue += 4.3f;
  if (!storable(q.ep.y, q.ep.out_dtype, q.ep.ld_y)) epilogue += 4.0f;
  if (q.ep.z) epilogue += storable(q.ep.z, q.ep.z_dtype, q.ep.ld_z) ? 1.5f : 5.5f;
  const long long waves = (tiles + 75) / 76;
  return 4.0f + stages + epilogue + (waves - 1) * (stages > epilogue ? stages : epilogue);
}

cudaError_t launch_pair(const Product& first, const Product* second, cudaStream_t s) {
  const int sms = num_sms();
  if (sms < 2) return cudaErrorNoDevice;
  const Product* q0 = &first;
  if (second && second->K > first.K) {
    q0 = second;
    second = &first;
  }
  PairParams p{};
  PairMaps m0{}, m1;
  CUtensorMap tz{};
  if (!encode_product(&m0, &p.prod[0], *q0)) return cudaErrorInvalidValue;
  p.tiles[0] = p.prod[0].nR * p.prod[0].nC;
  p.ratio = 1;
  m1 = m0;
  tz = m0.y;
  if (second) {
    if (!encode_product(&m1, &p.prod[1], *second)) return cudaErrorInvalidValue;
    p.tiles[1] = p.prod[1].nR * p.prod[1].nC;
    p.ratio = (p.prod[0].nk + p.prod[1].nk / 2) / p.prod[1].nk;
  }
  // two products are stored the same way
  p.y_tma = storable(q0->ep.y, q0->ep.out_dtype, q0->ep.ld_y) &&
            (!second || storable(second->ep.y, second->ep.out_dtype, second->ep.ld_y));
  p.z_tma = q0->ep.z && storable(q0->ep.z, q0->ep.z_dtype, q0->ep.ld_z);
  p.y[0] = q0->ep.y;
  p.y[1] = second ? second->ep.y : nullptr;
  if (p.z_tma && !encode_store(&tz, q0->ep.z, q0->ep.z_dtype, q0->C, q0->R, q0->ep.ld_z)) return cudaErrorInvalidValue;
  static const cudaError_t attr =
      cudaFuncSetAttribute(linear_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
  if (attr != cudaSuccess) return attr;
  p.type = q0->type;
  p.ep = q0->ep;
  p.reset_status = first.reset_status;
  p.hdr = q0->hdr;
  const int tiles = p.tiles[0] + p.tiles[1];
  const int pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch_dependent(linear_pair_kernel, dim3(2 * pairs), dim3(THREADS), SMEM_BYTES, s, m0, m1, tz, p);
}

}  // namespace lin
}  // namespace moe
