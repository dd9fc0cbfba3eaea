// Linear layer with bias, activation and residual in its epilogue (moe_linear) and
// its gradient (moe_linear_backward) on the 5th-generation tensor cores:
//   z = x W^T + b,   y = alpha act(z) + residual
//   dz = alpha dy act'(z),   db = sum_m dz,   dx = dz W,   dW = dz^T x
//
// One kernel computes all three products.  Its output is out[r][c] (row-major):
// operand A supplies the 128 columns c of a tile on the 128 TMEM lanes, operand B
// the BN rows r on the TMEM columns, so that the lanes of an epilogue warp hold
// neighbouring addresses of one output row and few rows (decode) cost a narrow
// BN instead of a mostly empty 128-row tile.
//   y : A = W  [N][K],  B = x  [M][K]; both contiguous along the sum (K-major)
//   dx: A = W  [N][K] contiguous along its columns (MN-major), B = dz [M][N] K-major
//   dW: A = x  [M][K] MN-major,                                B = dz [M][N] MN-major
// so no operand is ever transposed in memory.  All operands come by TMA in boxes of
// 128-byte rows with the 128-byte swizzle; edges are zero-filled by TMA.
//
// Few tiles and a long sum: `splits` blocks of one cluster share a tile, each takes
// a range of the sum, and after a cluster barrier each adds its share of the rows
// over all partials, read from the others' shared memory in rank order: no
// workspace, no atomics, the same result every time.
//
// What bounds it: some rows read the weights once (up to eight rows of small products
// go to linear_few.cu; 8 x 4096 x 4096: 7.3 us for 34 MB, 4.6 TB/s,
// 5 us at a copy's rate, the rest launch, ring fill and join); few columns read x once
// (16384 x 128 x 2048: 14.2 us, 4.7 TB/s).  Products that fill the GPU with tiles are
// bound by arithmetic and go to linear_pair.cu.  Which tiles and splits a product takes
// is the least of tile_estimate's times, which were fitted to measurements.
#include "linear.cuh"

namespace moe {
namespace lin {

constexpr int BM = 128;  // output columns per tile (TMEM lanes)
constexpr int THREADS = 128;
constexpr int MAX_SPLITS = 8;
constexpr int A_BYTES = BM * BK * 2;

constexpr int MAX_STAGES = 12;
__host__ __device__ constexpr int stage_bytes(int BN) { return A_BYTES + BN * BK * 2; }
// 1 KB to align the ring, 256 bytes of barriers before it
__host__ __device__ constexpr int smem_bytes(int BN, int stages) { return 1024 + 256 + stages * stage_bytes(BN); }
// Stages with `blocks` blocks on an SM (one loads while another stores): all that fit.
constexpr int stages_of(int BN, int blocks) {
  const int n = (228 * 1024 / blocks - 1024 - smem_bytes(BN, 0)) / stage_bytes(BN);
  return n > MAX_STAGES ? MAX_STAGES : n;
}

// One product of a launch.
struct TileProduct {
  int C, R;        // output columns and rows
  int nk;          // stages of the whole sum
  int nC, nR;      // tiles
  int splits;      // blocks per tile: a cluster's, or 1
  int a_mn, b_mn;  // operand columns / rows contiguous along c / r
  int half;        // gated: rows of the gate in the column operand
  Epilogue ep;
};
// A launch computes one product, or two side by side (a gradient's two, unless both fill the
// GPU): blocks from `first_blocks` on belong to the second.  A cluster's blocks share a tile of
// one product, or take one tile each.
struct Params {
  TileProduct prod[2];
  int first_blocks;
  int stages;      // of the ring
  int nacc;        // accumulators that a block's part of the sum is spread over
  uint32_t tmem_cols;
  int type;        // 0 = f16, 1 = bf16 operands
  int reset_status;
  DeviceHeader* hdr;
};
struct TileMaps {
  CUtensorMap a, b;
};

// fp32 at shared-memory address `addr` of block `rank` of the cluster
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// n values of one output column, rows r0.. of an array with ld elements between rows.
template <int CH>
__device__ __forceinline__ void store_rows(void* out, int dtype, size_t at, long long ld, int n, const float (&v)[CH]) {
  if (dtype == MOE_DTYPE_F32) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i < n) p[i * ld] = v[i];
  } else if (dtype == MOE_DTYPE_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i < n) p[i * ld] = __float2bfloat16_rn(v[i]);
  } else {
    __half* p = static_cast<__half*>(out) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i < n) p[i * ld] = __float2half_rn(v[i]);
  }
}

template <int CH>
__device__ __forceinline__ void add_rows(float (&v)[CH], const void* in, int dtype, size_t at, long long ld, int n) {
  float r[CH];
  if (dtype == MOE_DTYPE_F32) {
    const float* p = static_cast<const float*>(in) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = i < n ? p[i * ld] : 0.0f;
  } else if (dtype == MOE_DTYPE_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(in) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = i < n ? __bfloat162float(p[i * ld]) : 0.0f;
  } else {
    const __half* p = static_cast<const __half*>(in) + at;
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = i < n ? __half2float(p[i * ld]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] += r[i];
}

// The fused epilogue of n rows from r0 of output column c (one thread's values).
template <int CH>
__device__ __forceinline__ void finish(const TileProduct& p, float (&v)[CH], int r0, int n, int c) {
  if (c >= p.C || n <= 0) return;
  if (p.ep.bias) {
    const float b = load_as_f32(p.ep.bias, p.ep.bias_dtype, c);
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] += b;
  }
  if (p.ep.z) store_rows<CH>(p.ep.z, p.ep.z_dtype, static_cast<size_t>(r0) * p.ep.ld_z + c, p.ep.ld_z, n, v);
  act_all<CH>(v, p.ep.act);
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] *= p.ep.alpha;
  const size_t at = static_cast<size_t>(r0) * p.ep.ld_y + c;
  if (p.ep.residual) add_rows<CH>(v, p.ep.residual, p.ep.out_dtype, at, p.ep.ld_y, n);
  store_rows<CH>(p.ep.y, p.ep.out_dtype, at, p.ep.ld_y, n, v);
}

// The gated epilogue of n rows from r0 of output column c: sums of its gate and up columns.
template <int CH>
__device__ __forceinline__ void finish_gated(const TileProduct& p, float (&g)[CH], float (&u)[CH], int r0, int n, int c) {
  if (c >= p.C || n <= 0) return;
  if (p.ep.bias) {
    const float bg = load_as_f32(p.ep.bias, p.ep.bias_dtype, c), bu = load_as_f32(p.ep.bias, p.ep.bias_dtype, p.half + c);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      g[i] += bg;
      u[i] += bu;
    }
  }
  if (p.ep.z) {
    const size_t at = static_cast<size_t>(r0) * p.ep.ld_z + c;
    store_rows<CH>(p.ep.z, p.ep.z_dtype, at, p.ep.ld_z, n, g);
    store_rows<CH>(p.ep.z, p.ep.z_dtype, at + p.half, p.ep.ld_z, n, u);
  }
  act_all<CH>(g, p.ep.act);
#pragma unroll
  for (int i = 0; i < CH; ++i) g[i] *= u[i];
  store_rows<CH>(p.ep.y, p.ep.out_dtype, static_cast<size_t>(r0) * p.ep.ld_y + c, p.ep.ld_y, n, g);
}

template <int CH>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[CH]) {
  static_assert(CH == 16 || CH == 32, "16 or 32 columns");
  if constexpr (CH == 16) tmem_ld16(addr, v);
  else tmem_ld32(addr, v);
}

// Warp 0 loads, warp 1 issues the MMAs, then all four warps (one per 32 TMEM lanes)
// run the epilogue.  GATED: lanes 0-63 hold 64 gate columns, 64-127 the up columns beside
// them, which meet in shared memory.
template <int BN, bool GATED>
__global__ void __launch_bounds__(THREADS) linear_kernel(const __grid_constant__ TileMaps m0,
                                                         const __grid_constant__ TileMaps m1,
                                                         const __grid_constant__ Params p) {
  constexpr int STAGE = stage_bytes(BN);
  constexpr int CH = BN < 32 ? BN : 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * MAX_STAGES + 1];
  __shared__ uint32_t tmem_slot[1];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool second = static_cast<int>(blockIdx.x) >= p.first_blocks;
  const TileProduct& o = p.prod[second ? 1 : 0];
  const CUtensorMap* ma = second ? &m1.a : &m0.a;
  const CUtensorMap* mb = second ? &m1.b : &m0.b;
  const bool a_mn = o.a_mn, b_mn = BN >= 64 && o.b_mn;  // an MN-major box is 64 wide
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + MAX_STAGES), done = smem_u32(bars + 2 * MAX_STAGES);
  const int rank = o.splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = (static_cast<int>(blockIdx.x) - (second ? p.first_blocks : 0)) / o.splits;
  if (tile >= o.nC * o.nR) return;  // fills up a cluster of single tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(ma);
    prefetch_tensormap(mb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!GATED) {
    dep_wait();
    dep_launch();
  }

  // tiles: 16 row tiles side by side, then the next column tile, so that the blocks in
  // flight share both operands in L2
  constexpr int GR = 16;
  const int group = tile / (GR * o.nC), in_group = tile - group * (GR * o.nC);
  const int rows_here = min(GR, o.nR - group * GR);
  constexpr int BC = GATED ? BM / 2 : BM;  // output columns per tile
  const int c0 = in_group / rows_here * BC;
  const int r0 = (group * GR + in_group % rows_here) * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(o.nk) * rank / o.splits);
  const int kb1 = static_cast<int>(static_cast<long long>(o.nk) * (rank + 1) / o.splits);
  const int n = kb1 - kb0;                // at least 1: splits <= nk
  const int nacc = min(p.nacc, n);        // accumulators that this block fills
  if (GATED) {
    // few rows wait for the weights: they start on their way into L2 before the kernel before this
    // one has ended (nothing is read)
    if (BN <= 64 && warp == 0 && elect_one()) {
      for (int i = 0; i < min(n, 16); ++i) {
        tma_prefetch_2d(ma, (kb0 + i) * BK, c0);
        tma_prefetch_2d(ma, (kb0 + i) * BK, o.half + c0);
      }
    }
    __syncwarp();
    dep_wait();
    dep_launch();
  }
  // a wait that records a timeout lasts seconds: nothing of this launch is lost here
  if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) p.hdr->status = p.hdr->info = 0u;

  // Both roles: uniform control flow (addresses and descriptors stay in uniform
  // registers), one lane issues, the next barrier is looked at ahead.
  if (warp == 0) {
    const bool leader = elect_one();
    const uint32_t ring = smem_u32(smem);
    uint32_t stage = 0, phase = 1;
    int issued = 0;
    bool ready = true;  // the ring starts empty
    for (; issued < n; ++issued) {
      if (!ready && !mbar_wait(empty0 + 8 * stage, phase, abort_flag, p.hdr, 0x510000u)) break;
      const uint32_t full = full0 + 8 * stage, a = ring + stage * STAGE, b = a + A_BYTES;
      if (++stage == static_cast<uint32_t>(p.stages)) {
        stage = 0;
        phase ^= 1;
      }
      if (leader) {
        const int k = (kb0 + issued) * BK;
        mbar_arrive_expect_tx(full, STAGE);
        if (GATED) {
          tma_load_2d(a, ma, k, c0, full);
          tma_load_2d(a + A_BYTES / 2, ma, k, o.half + c0, full);
        } else if (a_mn) {
          tma_load_2d(a, ma, c0, k, full);
          tma_load_2d(a + A_BYTES / 2, ma, c0 + 64, k, full);
        } else {
          tma_load_2d(a, ma, k, c0, full);
        }
        if (b_mn) {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j) tma_load_2d(b + j * 8192, mb, r0 + j * 64, k, full);
        } else {
          tma_load_2d(b, mb, k, r0, full);
        }
      }
      __syncwarp();
      ready = mbar_try_wait(empty0 + 8 * stage, phase);
    }
    if (issued < n && leader)  // let the copies already issued land before shared memory is given up
      for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
        mbar_wait_quiet(full0 + 8 * (i % p.stages), (i / p.stages) & 1, 50000000ull);
  } else if (warp == 1) {
    const bool leader = elect_one();
    const uint32_t idesc = make_idesc(p.type, p.type, BM, BN) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
    const OperandWalk wa(a_mn), wb(b_mn);
    const uint32_t ring = smem_u32(smem);
    uint32_t stage = 0, phase = 0;
    int acc = -1;
    bool ready = mbar_try_wait(full0, 0);
    for (int i = 0; i < n; ++i) {
      if (!ready && !mbar_wait(full0 + 8 * stage, phase, abort_flag, p.hdr, 0x520000u)) break;
      tc_fence_after();
      const uint32_t a = ring + stage * STAGE, b = a + A_BYTES, empty = empty0 + 8 * stage;
      if (++stage == static_cast<uint32_t>(p.stages)) {
        stage = 0;
        phase ^= 1;
      }
      ready = i + 1 < n && mbar_try_wait(full0 + 8 * stage, phase);
      const int now = nacc == 1 ? 0 : i * nacc / n;
      const bool fresh = now != acc;
      acc = now;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16(tmem + acc * BN, wa.at(a, kk), wb.at(b, kk), idesc,
                  !(fresh && kk == 0));
        mma_commit(empty);
      }
      __syncwarp();
    }
    if (leader) mma_commit(done);
  } else if (!GATED && o.ep.residual) {
    // the residual's part of the tile comes into L2 while the product is computed
    const size_t es = o.ep.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
    const size_t bytes = static_cast<size_t>(min(BM, o.C - c0)) * es;
    const int share = BN / o.splits;
    for (int j = rank * share + (warp - 2) * 32 + lane; j < min((rank + 1) * share, o.R - r0); j += 64) {
      const uint8_t* row = static_cast<const uint8_t*>(o.ep.residual) + (static_cast<size_t>(r0 + j) * o.ep.ld_y + c0) * es;
      for (size_t b = 0; b < bytes; b += 128) prefetch_l2(row + b);
    }
  }
  __syncwarp();
  if (lane == 0) mbar_wait(done, 0, abort_flag, p.hdr, 0x530000u);
  __syncthreads();
  tc_fence_after();
  const bool good = *abort_flag == 0;
  const uint32_t quad = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const int cl = warp * 32 + lane;

  auto gather = [&](int j, float (&v)[CH]) {
    tmem_load<CH>(quad + j, v);
    tmem_ld_wait();
    for (int q = 1; q < nacc; ++q) {
      float u[CH];
      tmem_load<CH>(quad + q * BN + j, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < CH; ++i) v[i] += u[i];
    }
  };
  // Few output columns leave most lanes without one: the values then go through shared
  // memory too, and groups of `width` threads take rows in turn.
  const int cols = min(BC, o.C - c0);
  const int width = cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : BM;
  if (!GATED && o.splits == 1 && width == BM) {
    if (good) {
#pragma unroll 1
      for (int j = 0; j < BN; j += CH) {
        if (r0 + j >= o.R) break;
        float v[CH];
        gather(j, v);
        finish<CH>(o, v, r0 + j, min(CH, o.R - r0 - j), c0 + cl);
      }
    }
  } else {
    float* part = reinterpret_cast<float*>(smem);  // [BN][128], over the ring: every MMA has read it
    if (good) {
#pragma unroll 1
      for (int j = 0; j < BN; j += CH) {
        float v[CH];
        gather(j, v);
#pragma unroll
        for (int i = 0; i < CH; ++i) part[(j + i) * BM + cl] = v[i];
      }
    }
    if (o.splits > 1) cluster_sync_all();
    else __syncthreads();
    if (good) {
      // this block's share of the rows, this thread's group's of them, RB at a time: all
      // ranks' values of RB rows are on their way before the first is added
      const int groups = BM / width, own = static_cast<int>(threadIdx.x) / width;
      const int c = static_cast<int>(threadIdx.x) & (width - 1);
      const int per = BN / o.splits;
      const int per_group = (per + groups - 1) / groups;
      constexpr int RB = GATED ? 4 : 8;
      constexpr int PARTS = GATED ? 2 : 1;  // gate and up
      const uint32_t mine = smem_u32(part) + c * 4;
      const uint32_t first = o.splits > 1 ? 0u : cluster_rank();  // of the blocks that share the tile
      const int begin = rank * per + own * per_group;
      const int end = min(min(begin + per_group, (rank + 1) * per), o.R - r0);
      for (int j = begin; j < end; j += RB) {
        const int cnt = min(RB, end - j);
        float u[MAX_SPLITS][PARTS][RB];
#pragma unroll
        for (int q = 0; q < MAX_SPLITS; ++q)
          if (q < o.splits)
#pragma unroll
            for (int h = 0; h < PARTS; ++h)
#pragma unroll
              for (int i = 0; i < RB; ++i)
                if (i < cnt) u[q][h][i] = ld_cluster_f32(mine + (j + i) * (BM * 4) + h * (BC * 4), first + q);
        float v[PARTS][RB] = {};
#pragma unroll
        for (int q = 0; q < MAX_SPLITS; ++q)
          if (q < o.splits)
#pragma unroll
            for (int h = 0; h < PARTS; ++h)
#pragma unroll
              for (int i = 0; i < RB; ++i) v[h][i] += u[q][h][i];
        if constexpr (GATED) finish_gated<RB>(o, v[0], v[1], r0 + j, cnt, c0 + c);
        else finish<RB>(o, v[0], r0 + j, cnt, c0 + c);
      }
    }
    if (o.splits > 1) cluster_sync_all();  // no block leaves while another still reads its partial
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// Accumulators that a block spreads its part of the sum over.
inline int accumulators(const Product& q, int bn) { return q.ep.out_dtype != MOE_DTYPE_F32 ? 1 : bn <= 64 ? 4 : 2; }
// Output columns per tile.
inline int tile_cols(const Product& q) { return q.gated ? BM / 2 : BM; }

bool encode_product(TileMaps* m, TileProduct* t, const Product& q, int bn, int splits) {
  t->C = q.C;
  t->R = q.R;
  t->nk = (q.K + BK - 1) / BK;
  t->nC = (q.C + tile_cols(q) - 1) / tile_cols(q);
  t->nR = (q.R + bn - 1) / bn;
  t->half = q.gated ? q.C : 0;
  t->splits = splits;
  t->a_mn = q.cols_mn;
  t->b_mn = q.rows_mn;
  t->ep = q.ep;
  return encode(&m->a, q.cols.base, q.type, q.cols.inner, q.cols.outer, q.cols.ld, 64, q.cols_mn || q.gated ? 64 : BM) &&
         encode(&m->b, q.rows.base, q.type, q.rows.inner, q.rows.outer, q.rows.ld, 64, q.rows_mn ? 64 : bn);
}

struct Choice {
  int bn, splits;
  float us;
  int splits2;  // of the second product: 1, or as many as a cluster has blocks, like the first's
};

template <int BN, bool GATED>
cudaError_t launch_tile(const Product& q, const Product* second, const Choice& c, cudaStream_t s) {
  Params p{};
  TileMaps m0, m1;
  if (!encode_product(&m0, &p.prod[0], q, BN, c.splits)) return cudaErrorInvalidValue;
  m1 = m0;
  if (second && !encode_product(&m1, &p.prod[1], *second, BN, c.splits2)) return cudaErrorInvalidValue;
  static const cudaError_t attr = cudaFuncSetAttribute(
      linear_kernel<BN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(BN, stages_of(BN, 1)));
  if (attr != cudaSuccess) return attr;
  p.type = q.type;
  p.reset_status = q.reset_status;
  p.hdr = q.hdr;
  const int cluster = second && c.splits2 > c.splits ? c.splits2 : c.splits;
  auto blocks_of = [&](const TileProduct& t) {
    return (static_cast<long long>(t.nC) * t.nR * t.splits + cluster - 1) / cluster * cluster;
  };
  p.first_blocks = static_cast<int>(blocks_of(p.prod[0]));
  const long long blocks = p.first_blocks + (second ? blocks_of(p.prod[1]) : 0);
  // one block per SM where the grid leaves no second one: its ring takes all of shared
  // memory (not in large clusters, which then no longer find enough free SMs together)
  p.stages = stages_of(BN, BN == 256 || (blocks <= 152 && cluster <= 2) ? 1 : 2);
  // fp32 output: the tensor core's running sum rounds at every step, so its length is
  // kept short by spreading the sum over up to four accumulators (here; large products, which
  // go to linear_pair.cu, keep the whole sum in one: its two are the tiles in flight)
  p.nacc = accumulators(q, BN);
  int cols = 32;
  while (cols < BN * p.nacc) cols *= 2;
  p.tmem_cols = cols;
  cudaLaunchAttribute la[2];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = cluster;
  la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
  la[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes(BN, p.stages);
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_kernel<BN, GATED>, m0, m1, p);
}

// About how long a launch takes (us), for tiles of 128 x bn split over `splits` blocks.
// Measured on GB300: 2.2 us of launch, set-up and drain; a block's stage takes 0.17 us
// (bn = 16) to 0.20 us (128), 0.45 us at 256, or as long as the SM's blocks together need
// for their operands at 143 GB/s per SM; the epilogue, which nothing overlaps, 0.037 us per
// row, and more with an activation, z or a residual; each further wave 1.7 us; joining
// partials 1 us, 0.4 us per doubling and 0.02 us per row.  Within 20% of the measured times of some forty shapes
// (8 x 4096 x 4096 to 16384 x 2048 x 72), near enough to tell 17 us (16384 x 128 x
// 2048's weight gradient at bn = 64, 8 splits) from 54 us (128, 1).
float gated_estimate(const Product& q, int bn, int splits);
float tile_estimate(const Product& q, int bn, int splits) {
  if (q.gated) return gated_estimate(q, bn, splits);
  const long long nk = (q.K + BK - 1) / BK;
  const long long blocks = static_cast<long long>((q.C + BM - 1) / BM) * ((q.R + bn - 1) / bn) * splits;
  // a cluster's blocks lie in one group of SMs: clusters of 8 reach 128 of 152 SMs
  const int occupancy = bn == 256 ? 1 : 2, sms = splits == 8 ? 128 : 152;
  const long long waves = (blocks + sms * occupancy - 1) / (sms * occupancy);
  const int together = blocks > sms ? occupancy : 1;
  float stage = bn <= 32 ? 0.175f : bn <= 128 ? 0.20f : 0.45f;
  const float load = together * stage_bytes(bn) / 143000.0f;
  if (load > stage) stage = load;
  float t = waves * static_cast<float>((nk + splits - 1) / splits) * stage;
  const float memory = 2.0f * (static_cast<float>(q.R) + q.C) * q.K / 6.5e6f;
  if (memory > t) t = memory;
  // lanes without a column take rows instead
  const float lanes = q.C <= 16 ? 0.125f : q.C <= 32 ? 0.25f : q.C <= 64 ? 0.5f : 1.0f;
  const float row = 0.037f + (q.ep.act != MOE_ACT_NONE ? 0.009f : 0.0f) + (q.ep.z ? 0.012f : 0.0f) +
                    (q.ep.residual ? 0.05f : 0.0f);
  t += 2.2f + 1.7f * (waves - 1) + waves * row * lanes * (bn < q.R ? bn : q.R) / splits;
  for (int s = splits; s > 1; s /= 2) t += 0.4f;
  return splits > 1 ? t + 1.0f + 0.02f * bn : t;
}

// The same for gated products, fitted to 84 of them in every form (1 to 2048 rows, 256 to 8192 columns,
// sums of 768 to 4096; weights from memory up to 64 rows): the form of the least estimate is on average 1%
// slower than the fastest, 11% at most.
float gated_estimate(const Product& q, int bn, int splits) {
  const int i = bn <= 16 ? 0 : bn <= 32 ? 1 : bn <= 64 ? 2 : bn <= 128 ? 3 : 4;
  const float per_stage[5] = {0.126f, 0.138f, 0.19f, 0.277f, 0.446f};
  const int stages = ((q.K + BK - 1) / BK + splits - 1) / splits;
  // fp32 output: no accumulator sums more than 512 values (its rounding, 1.8e-9 of the sum per value, would
  // show); linear_pair.cu takes what finds no such form here
  if (q.ep.out_dtype == MOE_DTYPE_F32 && stages > 8 * accumulators(q, bn)) return 1e9f;
  const long long blocks = static_cast<long long>((q.C + BM / 2 - 1) / (BM / 2)) * ((q.R + bn - 1) / bn) * splits;
  const int occupancy = bn == 256 ? 1 : 2, sms = splits == 8 ? 120 : splits == 4 ? 144 : 152;
  const long long waves = (blocks + sms * occupancy - 1) / (sms * occupancy);
  float t = waves * stages * per_stage[i] * (occupancy == 2 && blocks > sms ? 1.44f : 1.0f);
  const float memory = 2.0f * (static_cast<float>(q.R) + 2.0f * q.C) * q.K / 6.43e6f;
  if (memory > t) t = memory;
  const float row = 0.064f + (q.ep.act != MOE_ACT_SILU && q.ep.act != MOE_ACT_NONE ? 0.005f : 0.0f) + (q.ep.z ? 0.024f : 0.0f);
  t += 4.8f + 4.5f * (waves - 1) + waves * row * (bn < q.R ? bn : q.R) / splits;
  return splits > 1 ? t - 0.24f + 0.016f * bn : t;
}

Choice choose_tile(const Product& q) {
  const long long nk = (q.K + BK - 1) / BK;
  Choice best{0, 1, 0.0f, 1};
  for (int bn = q.rows_mn ? 64 : 16; bn <= 256; bn *= 2) {
    for (int splits = 1; splits <= MAX_SPLITS && (splits == 1 || nk / splits >= 2); splits *= 2) {
      const float us = tile_estimate(q, bn, splits);
      if (best.bn == 0 || us < best.us) best = {bn, splits, us, 1};
    }
    if (bn >= q.R) break;
  }
  return best;
}

template <bool GATED>
cudaError_t launch_shape(const Product& q, const Product* second, const Choice& c, cudaStream_t s) {
  switch (c.bn) {
    case 16: return launch_tile<16, GATED>(q, second, c, s);
    case 32: return launch_tile<32, GATED>(q, second, c, s);
    case 64: return launch_tile<64, GATED>(q, second, c, s);
    case 128: return launch_tile<128, GATED>(q, second, c, s);
    default: return launch_tile<256, GATED>(q, second, c, s);
  }
}

// Two products in one launch of tiles of 128 x bn whose blocks all find a place at once: the
// longer of the two.  Sums of different lengths are split differently where each block has
// an SM to itself (4 x 3167 x 104's gradient: 12.2 us apart, 9.5 together; with two blocks on
// an SM that loses to two launches: 2048 x 1024 x 1024 20.5 us apart, 24.4 together).
Choice choose_both(const Product& q0, const Product& q1) {
  const Product* q[2] = {&q0, &q1};
  Choice best{0, 1, 0.0f, 1};
  for (int bn = 64; bn <= 128; bn *= 2)
    for (int cluster = 1; cluster <= MAX_SPLITS; cluster *= 2)
      for (int shared = cluster > 1 ? 1 : 0; shared < (cluster > 1 ? 4 : 1); ++shared) {  // one bit per product
        long long blocks[2];
        bool ok = true;
        for (int i = 0; i < 2; ++i) {
          const int splits = shared >> i & 1 ? cluster : 1;
          ok = ok && (splits == 1 || (q[i]->K + BK - 1) / BK / splits >= 2);
          blocks[i] = static_cast<long long>((q[i]->C + BM - 1) / BM) * ((q[i]->R + bn - 1) / bn) * splits;
          blocks[i] = (blocks[i] + cluster - 1) / cluster * cluster;
        }
        const bool equal = cluster == 1 || shared == 3;
        if (!ok || blocks[0] + blocks[1] > (equal ? 2 : 1) * (cluster == 8 ? 128 : 152)) continue;
        const float t0 = tile_estimate(q0, bn, shared & 1 ? cluster : 1);
        const float t1 = tile_estimate(q1, bn, shared & 2 ? cluster : 1);
        const float us = t0 > t1 ? t0 : t1;
        if (best.bn == 0 || us < best.us) best = {bn, shared & 1 ? cluster : 1, us, shared & 2 ? cluster : 1};
      }
  return best;
}

bool takes_pair(const Product& q, const Choice& c) { return pair_estimate(q) < c.us; }

cudaError_t launch_product(const Product& q, cudaStream_t s) {
  const Choice c = choose_tile(q);
  if (takes_pair(q, c)) return launch_pair(q, nullptr, s);
  return q.gated ? launch_shape<true>(q, nullptr, c, s) : launch_shape<false>(q, nullptr, c, s);
}

cudaError_t launch_gradient_products(const GradientProducts& g, cudaStream_t s) {
  Product q{};
  q.type = g.dtype == MOE_DTYPE_BF16 ? 1 : 0;
  q.C = g.K;
  q.cols_mn = true;
  q.ep = {MOE_ACT_NONE, MOE_DTYPE_F32, g.dtype, g.dtype, 1.0f, g.K, 0, nullptr, nullptr, nullptr, nullptr};
  q.reset_status = 1;
  q.hdr = g.hdr;
  q.rows = g.dz;
  Product dx = q, dw = q;
  dx.R = g.M;
  dx.K = g.N;
  dx.cols = {g.w, g.ld_w, g.K, g.N};
  dx.rows_mn = false;
  dx.ep.y = g.dx;
  dw.R = g.N;
  dw.K = g.M;
  dw.cols = {g.x, g.ld_x, g.K, g.M};
  dw.rows_mn = true;
  dw.ep.y = g.dw;
  if (g.dx && g.dw) {
    const Choice cx = choose_tile(dx), cw = choose_tile(dw), both = choose_both(dw, dx);
    const bool px = takes_pair(dx, cx), pw = takes_pair(dw, cw);
    const float apart = (px ? pair_estimate(dx) : cx.us) + (pw ? pair_estimate(dw) : cw.us);
    const bool large = (px && pw) || (g.pairs_may_mix && pair_estimate_both(dx, dw) < (both.bn && both.us < apart ? both.us : apart));
    if (large || (both.bn && both.us < apart)) {
      stage_begin("linear_dx_dw", s);
      const cudaError_t err = large ? launch_pair(dx, &dw, s) : launch_shape<false>(dw, &dx, both, s);
      stage_end(s);
      return err;
    }
  }
  cudaError_t err = cudaSuccess;
  if (g.dx) {
    stage_begin("linear_dx", s);
    err = launch_product(dx, s);
    stage_end(s);
    dw.reset_status = 0;
  }
  if (err == cudaSuccess && g.dw) {
    stage_begin("linear_dw", s);
    err = launch_product(dw, s);
    stage_end(s);
  }
  return err;
}

// ------------------------------------------------------------------ dz
// dz = alpha dy act'(z) in the operands' type, and per chunk of rows the fp32 sums
// of its unrounded columns.  Thread (x, y): eight columns of every 8th row, four rows'
// loads issued before the first is used (bound by memory: dy and z in, dz out).  DT, T:
// types of dy and of z and dz.  VEC: rows that 16-byte accesses fit, columns 8 x .. 8 x +
// 7; otherwise columns x + 32 i, so that a warp's accesses are neighbours.
struct DzArgs {
  int M, N, rows;  // rows per chunk
  int act;
  float alpha;
  long long ld_dy, ld_dz;
  const void* dy;
  const void* z;
  void* dz;
  float* partials;  // [chunks][N], null: not wanted
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(T (&v)[8], const void* p, size_t at, int n) {
  const T* q = static_cast<const T*>(p) + at;
  if (VEC) {
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      reinterpret_cast<uint4*>(v)[j] = __ldg(reinterpret_cast<const uint4*>(q) + j);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) v[i] = q[32 * i];
  }
}

template <typename DT, typename T, bool VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(DzArgs a) {
  __shared__ float s_sum[8][256 + 8];
  constexpr int AHEAD = 4;
  dep_wait();
  dep_launch();
  const int c = blockIdx.x * 256 + threadIdx.x * (VEC ? 8 : 1);  // first column
  const int n = a.N - c;                                         // columns from there on
  auto in = [&](int i) { return VEC || 32 * i < n; };
  const int m0 = blockIdx.y * a.rows, m1 = min(a.M, m0 + a.rows);
  float sum[8] = {};
  if (n > 0) {
    for (int mb = m0 + threadIdx.y; mb < m1; mb += 8 * AHEAD) {
      alignas(16) DT g[AHEAD][8];
      alignas(16) T z[AHEAD][8];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const int m = mb + 8 * q;
        if (m < m1) {
          load8<DT, VEC>(g[q], a.dy, static_cast<size_t>(m) * a.ld_dy + c, n);
          if (a.act != MOE_ACT_NONE) load8<T, VEC>(z[q], a.z, static_cast<size_t>(m) * a.N + c, n);
        }
      }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const int m = mb + 8 * q;
        if (m >= m1) break;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = in(i) ? a.alpha * as_float(g[q][i]) : 0.0f;
        auto times = [&](int act) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (in(i)) v[i] *= act_grad(as_float(z[q][i]), act);
        };
        switch (a.act) {
          case MOE_ACT_NONE: break;
          case MOE_ACT_RELU: times(MOE_ACT_RELU); break;
          case MOE_ACT_SILU: times(MOE_ACT_SILU); break;
          case MOE_ACT_GELU: times(MOE_ACT_GELU); break;
          default: times(MOE_ACT_GELU_TANH);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
        if (a.dz) {
          T* to = static_cast<T*>(a.dz) + static_cast<size_t>(m) * a.ld_dz + c;
          if (VEC) {
            alignas(16) T out[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = as_type<T>(v[i]);
            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(out);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (in(i)) to[32 * i] = as_type<T>(v[i]);
          }
        }
      }
    }
  }
  if (!a.partials) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_sum[threadIdx.y][VEC ? threadIdx.x * 8 + i : threadIdx.x + 32 * i] = sum[i];
  __syncthreads();
  const int col = threadIdx.y * 32 + threadIdx.x;
  if (blockIdx.x * 256 + col < a.N) {
    float v = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += s_sum[y][col];
    a.partials[static_cast<size_t>(blockIdx.y) * a.N + blockIdx.x * 256 + col] = v;
  }
}

template <typename DT, typename T>
cudaError_t launch_dz(const DzArgs& d, bool vec, int chunks, cudaStream_t s) {
  const dim3 grid((d.N + 255) / 256, chunks), block(32, 8);
  return vec ? launch_dependent(linear_dz_kernel<DT, T, true>, grid, block, 0, s, d)
             : launch_dependent(linear_dz_kernel<DT, T, false>, grid, block, 0, s, d);
}
template <typename T>
cudaError_t launch_dz(const DzArgs& d, int dy_dtype, bool vec, int chunks, cudaStream_t s) {
  if (dy_dtype == MOE_DTYPE_F32) return launch_dz<float, T>(d, vec, chunks, s);
  if (dy_dtype == MOE_DTYPE_BF16) return launch_dz<__nv_bfloat16, T>(d, vec, chunks, s);
  return launch_dz<__half, T>(d, vec, chunks, s);
}

}  // namespace lin

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  using namespace lin;
  Product q{};
  q.R = a.M;
  q.C = a.N;
  q.K = a.K;
  q.type = a.dtype == MOE_DTYPE_BF16 ? 1 : 0;
  q.rows = {a.x, a.ld_x, a.K, a.M};
  q.cols = {a.w, a.ld_w, a.K, a.N};
  q.ep = {a.act, a.bias_dtype, a.out_dtype, a.dtype, a.alpha, a.ld_y, a.N, a.bias, a.residual, a.y, a.z};
  q.reset_status = 1;
  q.hdr = a.hdr;
  stage_begin("linear", s);
  const cudaError_t err = takes_few(a) ? launch_few(a, s) : launch_product(q, s);
  stage_end(s);
  return err;
}

size_t linear_dz_bytes(int M, int N) { return static_cast<size_t>(M) * lin::dz_ld(N) * 2; }
size_t linear_partials_bytes(int M, int N) {
  const int rows = lin::dz_rows(M);
  return static_cast<size_t>((M + rows - 1) / rows) * N * sizeof(float);
}

bool linear_dz_is_dy(const LinearBackwardArgs& a) {
  return a.act == MOE_ACT_NONE && a.alpha == 1.0f && a.dy_dtype == a.dtype && a.ld_y % 8 == 0 &&
         reinterpret_cast<uintptr_t>(a.dy) % 16 == 0;
}

cudaError_t launch_linear_backward(const LinearBackwardArgs& a, cudaStream_t s) {
  using namespace lin;
  const bool direct = linear_dz_is_dy(a);
  const bool products = a.dx || a.dw;
  // the first product clears the status word; without one nobody else does
  cudaError_t err = products ? cudaSuccess : launch_reset_header(a.hdr, s);
  if (err != cudaSuccess) return err;
  if ((!direct && products) || a.dbias) {
    DzArgs d{};
    d.M = a.M;
    d.N = a.N;
    d.rows = dz_rows(a.M);
    d.act = a.act;
    d.alpha = a.alpha;
    d.ld_dy = a.ld_y;
    d.ld_dz = dz_ld(a.N);
    d.dy = a.dy;
    d.z = a.z;
    d.dz = direct || !products ? nullptr : a.dz;
    const int chunks = (a.M + d.rows - 1) / d.rows;
    d.partials = !a.dbias ? nullptr : chunks == 1 ? a.dbias : a.partials;
    const bool vec = a.N % 8 == 0 && a.ld_y % 8 == 0 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.z) % 16 == 0;
    stage_begin("linear_dz", s);
    err = a.dtype == MOE_DTYPE_BF16 ? launch_dz<__nv_bfloat16>(d, a.dy_dtype, vec, chunks, s)
                                    : launch_dz<__half>(d, a.dy_dtype, vec, chunks, s);
    stage_end(s);
    if (err == cudaSuccess && a.dbias && chunks > 1) err = launch_column_sums(a.partials, chunks, a.N, a.dbias, s);
  }
  if (err != cudaSuccess || !products) return err;
  const Operand dz = direct ? Operand{a.dy, a.ld_y, a.N, a.M} : Operand{a.dz, dz_ld(a.N), a.N, a.M};
  return launch_gradient_products({a.M, a.N, a.K, a.dtype, a.ld_x, a.ld_w, a.x, a.w, a.dx, a.dw, dz, false, a.hdr}, s);
}

}  // namespace moe
