// Product of two matrices in 4-bit microscaled codes:
//   out[i, j] = bias[j] + sum_k (a[i, k] 2^Ea[i, k/32]) (b[j, k] 2^Eb[j, k/32])
//
// Tile kernel.  A persistent block per SM computes tiles of 128 x BN (256, 128 or
// 64).  One warp brings slabs of 128 bytes (256 k's) of both operands into a ring of
// shared memory stages by TMA, and the slabs' scales (512 bytes for 128 rows x 128
// k's, in the order of the tensor cores' copy) by plain bulk copies; one elected thread
// copies the scales on into TMEM and issues four block-scaled tcgen05.mma (K = 64
// each) a slab.  Scaling and summing are the tensor core's, so nothing else touches a
// step; eight warps read the finished sums and store them.  Each stage has its own TMEM
// columns for its scales: they are written again only after the stage's products
// are done, which the refill of the stage waits for anyway.  One thread alone runs
// through all steps: with the warp meeting at each (8192^3, tiles of 64 columns) 478 us, 424 so.
//
// Pair kernel.  Two SMs compute a tile of 256 x 256, each with its half of the rows of a and of b
// in shared memory: 35 KB a block and step from L2 instead of 51.  131,072 x 1024 x 8192: 311 us in a graph
// (7.0 PFLOP/s at the clock that the power limit leaves), 339 by single SMs.
//
// Work is cut as in the 8-bit product: whole tiles in turn, or all steps split evenly
// over the SMs with a second launch that joins the pieces; make_plan4() has the rule.
//
// Row kernel (one row, or two by a small b): reads b once; plain CUDA cores.  A
// lane's 16 bytes are one scale block; its products of two codes are multiples of 1/4
// up to 36, so sums of eight are exact in float16 pairs.  Bound by latency: 1 x 1024 x 8192 3.3 us.
#include <algorithm>
#include <cmath>

#include "emb_tiles.cuh"

namespace emb {
namespace {

constexpr int kBK = 256;             // k's of a step: 128 bytes of a row
constexpr int kThreads = (kSumWarps + 2) * 32;  // then a TMA warp and an MMA warp
constexpr int kTmaWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
constexpr int kAfterLoads = 0;       // lost_warp: not a warp's wait, but the block is told when its last load is issued

struct Matmul4Args {
  const unsigned char *a, *b, *sa, *sb;
  const float* bias;
  void* out;
  float* partial;            // [slots][kBM * BN]
  long long lda, ldb, ldo;
  int m, n, k;
  int m_tiles, n_tiles, k_blocks;
  int s_blocks;              // scale tiles in a row of them: ceil(k / 128)
  long long steps;           // m_tiles * n_tiles * k_blocks
  long long per_cta;         // steps a block takes; 0: whole tiles, block-stride
  unsigned* flags;
  int lost_warp;             // the warp whose wait at step lost_step counts as run out; -1: none
  unsigned lost_step;
};

// D[128 x N] (+)= A B^T, 64 k's: e2m1 operands in shared memory, a power of two for 32 k's of a row in TMEM.
__device__ __forceinline__ void tc_mma4(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, unsigned sa,
                                        unsigned sb, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((unsigned)add)
      : "memory");
}
// Copies 512 bytes of scales (32 rows of 16 bytes) into four TMEM columns, once for each 32 lanes.
__device__ __forceinline__ void tc_copy_scales(unsigned d, unsigned long long desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(desc) : "memory");
}
// Shared memory descriptor of such a block: no swizzle, eight-row groups 128 bytes apart, version 1.
__device__ __forceinline__ unsigned long long scale_desc(unsigned addr) {
  return (unsigned long long)((addr >> 4) & 0x3FFF) | (8ull << 32) | (1ull << 46);
}
__device__ __forceinline__ void tc_mma4_pair(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, unsigned sa,
                                             unsigned sb, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((unsigned)add)
      : "memory");
}
__device__ __forceinline__ void tc_copy_scales_pair(unsigned d, unsigned long long desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(desc) : "memory");
}

// A step's copies of scales and products, `left` k's of it (a constant for a whole one).  ROWS: tiles
// of scales of 128 rows, a's and b's; a block of 128 k's has a's scales in four TMEM columns,
// and b's tiles side by side.
template <int ROWS, bool PAIR>
__device__ __forceinline__ void issue_step4(unsigned d, unsigned long long da, unsigned long long db, unsigned idesc, unsigned long long ds,
                                            unsigned ts, unsigned half_cols, bool add, int left) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h * 128 < left) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const unsigned to = ts + (j == 0 ? h * 4 : 8 + h * 4 * (ROWS - 1) + (j - 1) * 4);
        if (PAIR) tc_copy_scales_pair(to, ds + (j * 1024 + h * 512) / 16);
        else tc_copy_scales(to, ds + (j * 1024 + h * 512) / 16);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kBK / 64; ++j) {
    if (j * 64 < left) {
      const unsigned id = (j & 1) * 2u, h = j >> 1, sa = ts + h * 4, sb = ts + 8 + h * 4 * (ROWS - 1) + half_cols;
      if (PAIR) tc_mma4_pair(d, da + 2 * j, db + 2 * j, idesc | (id << 4) | (id << 29), sa, sb, add || j > 0);
      else tc_mma4(d, da + 2 * j, db + 2 * j, idesc | (id << 4) | (id << 29), sa, sb, add || j > 0);
    }
  }
}
__device__ __forceinline__ void bulk_load(unsigned dst, const void* src, unsigned bytes, unsigned bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// ------------------------------------------------------------------ tile kernel

template <int BN>
struct TileCfg4 {
  static constexpr int kSlabBytes = (kBM + BN) * 128;
  static constexpr int kRowBlocks = 1 + (BN + 127) / 128;       // scale tiles of 128 rows in a step: a's, b's
  static constexpr int kScaleBytes = kRowBlocks * 1024;         // of 256 k's
  static constexpr int kStages = (204 * 1024 + 4096) / (kSlabBytes + kScaleBytes);  // 4, 6 or 8
  static constexpr int kAccs = BN == 256 ? 1 : 2;
  static constexpr int kScaleCols = kRowBlocks * 8;             // TMEM columns of a stage's scales
  static constexpr int kUsedCols = kAccs * BN + kStages * kScaleCols;
  static constexpr int kCols = kUsedCols <= 256 ? 256 : 512;
  static constexpr int kStoreBytes = kSumWarps * 32 * 17 * 4;   // 32 rows x 16 columns a warp, for unaligned output
  static constexpr int kBytes = kStages * (kSlabBytes + kScaleBytes) + kStoreBytes + 1024;  // + room to align
  static_assert(kUsedCols <= 512 && kBytes <= 232448, "TMEM columns, shared memory");
};

template <int BN, typename OT, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) tile4_kernel(const __grid_constant__ CUtensorMap map_a,
                                                            const __grid_constant__ CUtensorMap map_b,
                                                            const __grid_constant__ Matmul4Args p) {
  using C = TileCfg4<BN>;
  constexpr int kHalf = BN / 2;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long bars[2 * C::kStages + 2 * C::kAccs];
  __shared__ unsigned tmem_slot;
  __shared__ int stop_flag;
  __shared__ unsigned issued[2];  // steps whose loads and products were issued
  volatile int* stop = &stop_flag;
  const unsigned smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // full: a stage's slabs and scales are there.  done: its products are, so it may be
  // filled again.  afull: a tile's sums are complete.  aempty: they have been read.
  const unsigned full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages, afull0 = done0 + 8 * C::kStages;
  const unsigned aempty0 = afull0 + 8 * C::kAccs;
  const unsigned scales0 = smem + C::kStages * C::kSlabBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, 1);
    }
    for (int t = 0; t < C::kAccs; ++t) {
      mbar_init(afull0 + 8 * t, 1);
      mbar_init(aempty0 + 8 * t, kSumWarps);
    }
    stop_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(C::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = tmem_slot, tscales = tmem + C::kAccs * BN;

  long long pos, end;
  my_range(p, &pos, &end, blockIdx.x);
  Unit u;

  if (warp == kTmaWarp) {
    unsigned it = 0;
    bool go = true;
    const int last_b = (p.n - 1) >> 7;  // b's last tile of scales
    while (go && next_unit(p, &pos, end, &u, gridDim.x)) {
      for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
        const unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
        go = __all_sync(0xffffffffu, p.lost_warp == kTmaWarp && p.lost_step == it ? give_up(stop, p.flags)
                                                                                 : mbar_wait(done0 + 8 * s, ph ^ 1, stop, p.flags));
        if (!go) break;
        if (elect_one()) {
          const unsigned dst = smem + s * C::kSlabBytes, sdst = scales0 + s * C::kScaleBytes, bar = full0 + 8 * s;
          const unsigned bytes = min(2, p.s_blocks - 2 * kb) * 512;
          mbar_expect_tx(bar, C::kSlabBytes + C::kRowBlocks * bytes);
          tma_load(dst, &map_a, kb * 128, u.tm * kBM, bar);
          tma_load(dst + kBM * 128, &map_b, kb * 128, u.tn * BN, bar);
          bulk_load(sdst, p.sa + ((long long)u.tm * p.s_blocks + 2 * kb) * 512, bytes, bar);
#pragma unroll
          for (int j = 0; j < C::kRowBlocks - 1; ++j) {  // past b's last rows: any scales do
            const int rb = min((u.tn * BN >> 7) + j, last_b);
            bulk_load(sdst + 1024 * (1 + j), p.sb + ((long long)rb * p.s_blocks + 2 * kb) * 512, bytes, bar);
          }
        }
        __syncwarp();
      }
    }
    if (p.lost_warp == kAfterLoads) give_up(stop, p.flags);
    issued[0] = it;
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // e2m1 x e2m1, power-of-two scales, both K-major, N = BN, M = 128
    constexpr unsigned idesc = (1u << 7) | (1u << 10) | ((BN >> 3) << 17) | (1u << 23) | ((kBM >> 4) << 24);
    unsigned it = 0, tile = 0;
    bool go = true;
    while (go && next_unit(p, &pos, end, &u, gridDim.x)) {
      const unsigned t = tile % C::kAccs, tph = (tile / C::kAccs) & 1;
      go = __all_sync(0xffffffffu, mbar_wait(aempty0 + 8 * t, tph ^ 1, stop, p.flags));
      if (!go) break;
      tc_fence_after();
      // a tile of 64 columns has the scales of half a block of 128 rows of b
      const unsigned half_cols = BN == 64 ? (u.tn & 1) * 2 : 0;
      // One thread for the whole unit: with the warp meeting at every step, a step took 50 to 100 cycles more.
      bool fine = true;
      unsigned did = 0;
      if (elect_one()) {
        unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++did) {
          fine = p.lost_warp == kMmaWarp && p.lost_step == it + did ? give_up(stop, p.flags) : mbar_wait(full0 + 8 * s, ph, stop, p.flags);
          if (!fine) break;
          tc_fence_after();
          const unsigned at = smem + s * C::kSlabBytes, ts = tscales + s * C::kScaleCols, d = tmem + t * BN;
          const unsigned long long da = smem_desc(at), db = smem_desc(at + kBM * 128), ds = scale_desc(scales0 + s * C::kScaleBytes);
          const int left = p.k - kb * kBK;
          if (left >= kBK) issue_step4<C::kRowBlocks, false>(d, da, db, idesc, ds, ts, half_cols, kb > u.kb0, kBK);
          else issue_step4<C::kRowBlocks, false>(d, da, db, idesc, ds, ts, half_cols, kb > u.kb0, left);
          tc_commit(done0 + 8 * s);
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
        if (fine) tc_commit(afull0 + 8 * t);
      }
      __syncwarp();
      it += __reduce_max_sync(0xffffffffu, did);
      go = __all_sync(0xffffffffu, fine);
      if (!go) break;
      ++tile;
    }
    issued[1] = it;
    __syncwarp();
  } else {  // TMEM lanes 32 (warp % 4).., columns group (warp / 4)
    const int half = warp >> 2, quarter = warp & 3;
    float* const stage = reinterpret_cast<float*>(raw + (smem - smem_u32(raw)) + C::kStages * (C::kSlabBytes + C::kScaleBytes)) + warp * 32 * 17;
    unsigned tile = 0;
    while (next_unit(p, &pos, end, &u, gridDim.x)) {
      const unsigned t = tile % C::kAccs, tph = (tile / C::kAccs) & 1;
      const int row = u.tm * kBM + quarter * 32 + lane;
      const int col0 = u.tn * BN + half * kHalf;
      if (!__all_sync(0xffffffffu, mbar_wait(afull0 + 8 * t, tph, stop, p.flags))) break;
      tc_fence_after();
      const unsigned taddr = tmem + ((unsigned)(quarter * 32) << 16) + t * BN + half * kHalf;
      unsigned v[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tc_load32(taddr + c, v + c);
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tc_wait32(v + c);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(aempty0 + 8 * t);  // all sums are in registers
      float acc[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) acc[c] = __uint_as_float(v[c]);
      store_unit<BN, OT, WIDE>(p, u, warp, lane, row, col0, acc, stage);
      ++tile;
    }
  }
  tc_fence_before();
  __syncthreads();
  // A wait ran out, of whichever warp: copies and products that no one has waited for
  // land before TMEM is freed and the block ends.
  if (*stop) {  // the same for the block: written before the barrier only
    const unsigned n = warp >= kSumWarps ? issued[warp - kSumWarps] : 0;
    if (warp == kTmaWarp)
      for (unsigned j = n - min(n, (unsigned)C::kStages); j < n; ++j) mbar_drain(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
    if (warp == kMmaWarp && n > 0) mbar_drain(done0 + 8 * ((n - 1) % C::kStages), ((n - 1) / C::kStages) & 1);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
  }
}

// ------------------------------------------------------------------ pairs of SMs

// A tile of 256 x 256 by two neighbouring SMs: each holds its 128 rows of a, half of b's rows
// (the tensor cores read both halves), all scales of those 256 and the sums of its own rows.  A step then
// takes 35 KB a block from L2 where a tile of 128 x 256 takes 51: at 512 cycles of products a
// step those are 29 TB/s for 152 SMs, more than L2 gives.
struct PairCfg4 {
  static constexpr int kSlabBytes = 2 * kBM * 128;
  static constexpr int kScaleBytes = 3 * 1024;
  static constexpr int kScaleCols = 24;
};
template <bool WIDE>
struct PairStages4 : PairCfg4 {
  static constexpr int kStages = WIDE ? 6 : 5;
  static constexpr int kStoreBytes = WIDE ? 0 : kSumWarps * 32 * 17 * 4;
  static constexpr int kBytes = kStages * (kSlabBytes + kScaleBytes) + kStoreBytes + 1024;
  static_assert(256 + kStages * kScaleCols <= 512 && kBytes <= 232448, "TMEM columns, shared memory");
};

template <typename OT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb, const __grid_constant__ Matmul4Args p) {
  using C = PairStages4<WIDE>;
  constexpr int BN = 256, kHalf = BN / 2;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long bars[2 * C::kStages + 2];
  __shared__ unsigned tmem_slot, stop_flag;
  __shared__ unsigned issued[2];  // steps whose loads and products were issued
  const unsigned smem = (smem_u32(raw) + 1023u) & ~1023u, stop = smem_u32(&stop_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const unsigned full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages, afull = done0 + 8 * C::kStages, aempty = afull + 8;
  const unsigned scales0 = smem + C::kStages * C::kSlabBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, 1);
    }
    mbar_init(afull, 1);
    mbar_init(aempty, 2 * kSumWarps);                          // of both blocks
    stop_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pair_sync();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  const unsigned tmem = tmem_slot, tscales = tmem + BN;

  long long pos, end;
  my_range(p, &pos, &end, pair);
  Unit u;

  if (warp == kTmaWarp) {
    unsigned it = 0;
    bool go = true;
    const int last_a = (p.m - 1) >> 7, last_b = (p.n - 1) >> 7;  // last tiles of scales: past them, any do
    while (go && next_unit(p, &pos, end, &u, pairs)) {
      const int ra = u.tm * 2 + rank;
      for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
        const unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
        go = __all_sync(0xffffffffu, p.lost_warp == kTmaWarp && p.lost_step == it ? pair_give_up(stop, p.flags)
                                                                                 : pair_wait(done0 + 8 * s, ph ^ 1, stop, p.flags));
        if (!go) break;
        if (elect_one()) {
          const unsigned dst = smem + s * C::kSlabBytes, sdst = scales0 + s * C::kScaleBytes, bar = peer_addr(full0 + 8 * s, 0);
          if (rank == 0) mbar_expect_tx(full0 + 8 * s, 2 * (C::kSlabBytes + C::kScaleBytes));
          tma_load_pair(dst, &map_a, kb * 128, ra * kBM, bar);
          tma_load_pair(dst + kBM * 128, &map_b, kb * 128, u.tn * BN + rank * kBM, bar);
          tma_load_pair(sdst, &map_sa, 0, min(ra, last_a) * p.s_blocks + 2 * kb, bar);
#pragma unroll
          for (int j = 0; j < 2; ++j) tma_load_pair(sdst + 1024 * (1 + j), &map_sb, 0, min(u.tn * 2 + j, last_b) * p.s_blocks + 2 * kb, bar);
        }
        __syncwarp();
      }
    }
    if (p.lost_warp == kAfterLoads) pair_give_up(stop, p.flags);
    issued[0] = it;
    __syncwarp();
  } else if (warp == kMmaWarp) {
    constexpr unsigned idesc = (1u << 7) | (1u << 10) | ((BN >> 3) << 17) | (1u << 23) | ((2 * kBM >> 4) << 24);
    unsigned it = 0, tile = 0;
    bool go = rank == 0;
    while (go && next_unit(p, &pos, end, &u, pairs)) {
      go = __all_sync(0xffffffffu, pair_wait(aempty, (tile & 1) ^ 1, stop, p.flags));
      if (!go) break;
      bool fine = true;
      unsigned did = 0;
      if (elect_one()) {
        unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++did) {
          fine = p.lost_warp == kMmaWarp && p.lost_step == it + did ? pair_give_up(stop, p.flags) : pair_wait(full0 + 8 * s, ph, stop, p.flags);
          if (!fine) break;
          tc_fence_after();
          const unsigned at = smem + s * C::kSlabBytes, ts = tscales + s * C::kScaleCols;
          const unsigned long long da = smem_desc(at), db = smem_desc(at + kBM * 128), ds = scale_desc(scales0 + s * C::kScaleBytes);
          const int left = p.k - kb * kBK;
          if (left >= kBK) issue_step4<3, true>(tmem, da, db, idesc, ds, ts, 0, kb > u.kb0, kBK);
          else issue_step4<3, true>(tmem, da, db, idesc, ds, ts, 0, kb > u.kb0, left);
          commit_both(done0 + 8 * s);
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
        if (fine) commit_both(afull);
      }
      __syncwarp();
      it += __reduce_max_sync(0xffffffffu, did);
      go = __all_sync(0xffffffffu, fine);
      if (!go) break;
      ++tile;
    }
    issued[1] = it;
    __syncwarp();
  } else {  // TMEM lanes 32 (warp % 4).., columns group (warp / 4)
    const int half = warp >> 2, quarter = warp & 3;
    float* const stage = reinterpret_cast<float*>(raw + (smem - smem_u32(raw)) + C::kStages * (C::kSlabBytes + C::kScaleBytes)) + warp * 32 * 17;
    unsigned tile = 0;
    while (next_unit(p, &pos, end, &u, pairs)) {
      const int row = (u.tm * 2 + rank) * kBM + quarter * 32 + lane;
      const int col0 = u.tn * BN + half * kHalf;
      if (!__all_sync(0xffffffffu, pair_wait(afull, tile & 1, stop, p.flags))) break;
      tc_fence_after();
      const unsigned taddr = tmem + ((unsigned)(quarter * 32) << 16) + half * kHalf;
      unsigned v[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tc_load32(taddr + c, v + c);
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tc_wait32(v + c);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(aempty, 0);                   // all sums are in registers
      float acc[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) acc[c] = __uint_as_float(v[c]);
      store_unit<BN, OT, WIDE, 2>(p, u, warp, lane, row, col0, acc, stage);
      ++tile;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (pair_stopped(stop)) {  // a wait ran out: what is in flight lands before the blocks end
    const unsigned n = warp >= kSumWarps ? issued[warp - kSumWarps] : 0;
    if (rank == 0 && warp == kTmaWarp)
      for (unsigned j = n - min(n, (unsigned)C::kStages); j < n; ++j) pair_drain(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
    if (rank == 0 && warp == kMmaWarp && n > 0) pair_drain(done0 + 8 * ((n - 1) % C::kStages), ((n - 1) / C::kStages) & 1);
    pair_settle();
  }
  __syncthreads();
  pair_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------------ row kernel

constexpr int kRowMax = 2;

// 32 codes as pairs of float16.
__device__ __forceinline__ void codes32(const uint4& q, __half2* o) {
  const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned h[4];
    asm("{\n.reg .b8 c0, c1, c2, c3;\n"
        "mov.b32 {c0, c1, c2, c3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, c1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, c3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w[i]));
#pragma unroll
    for (int j = 0; j < 4; ++j) o[4 * i + j] = *reinterpret_cast<__half2*>(&h[j]);
  }
}
// Clears the bytes from `keep` on (keep < 16).
__device__ __forceinline__ uint4 head_bytes(uint4 q, int keep) {
  unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = keep - 4 * i;
    w[i] = left >= 4 ? w[i] : left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// d 2^(ea - 127) 2^(eb - 127), in two steps of half the exponent each: neither leaves the
// range before the product does.  255 is NaN.
__device__ __forceinline__ float scaled(float d, int ea, int eb) {
  const int e = ea + eb - 254, h = e >> 1;
  const float v = d * __uint_as_float((unsigned)(h + 127) << 23) * __uint_as_float((unsigned)(e - h + 127) << 23);
  return max(ea, eb) == 255 ? __uint_as_float(0x7fc00000u) : v;
}
__device__ __forceinline__ const unsigned char* scale_ptr(const unsigned char* s, int s_blocks, int row, int block) {
  return s + ((long long)(row >> 7) * s_blocks + (block >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (block & 3);
}

// A block's eight warps take 8 / S groups of R rows of b, S warps to a group; a lane
// takes a scale block (16 bytes) every 32 S of them.
template <int M, int S, int R, typename OT>
__global__ void __launch_bounds__(256) row4_kernel(const __grid_constant__ Matmul4Args p) {
  constexpr int kGroups = 8 / S, kBatch = R == 1 ? 2 : 1;
  __shared__ float part[8][R][M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x * kGroups + warp / S) * R;
  const int blocks = (p.k + 31) >> 5, bytes = (p.k + 1) >> 1;
  float acc[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < M; ++i) acc[r][i] = 0.0f;
  for (int b0 = (warp % S) * 32 + lane; b0 < blocks; b0 += kBatch * S * 32) {
    uint4 qb[kBatch][R], qa[kBatch][M];
    int eb[kBatch][R], ea[kBatch][M];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int b = b0 + u * S * 32;
      const bool in = b < blocks;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int j = min(j0 + r, p.n - 1);  // past the last row: read again, not stored
        qb[u][r] = in ? __ldg(reinterpret_cast<const uint4*>(p.b + j * p.ldb + b * 16)) : make_uint4(0, 0, 0, 0);
        eb[u][r] = in ? __ldg(scale_ptr(p.sb, p.s_blocks, j, b)) : 0;
      }
#pragma unroll
      for (int i = 0; i < M; ++i) {
        qa[u][i] = in && i < p.m ? __ldg(reinterpret_cast<const uint4*>(p.a + i * p.lda + b * 16)) : make_uint4(0, 0, 0, 0);
        ea[u][i] = in && i < p.m ? __ldg(scale_ptr(p.sa, p.s_blocks, i, b)) : 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int left = bytes - (b0 + u * S * 32) * 16;
      if (left < 16) {  // the row's last piece: what lies past k does not count
#pragma unroll
        for (int r = 0; r < R; ++r) qb[u][r] = head_bytes(qb[u][r], max(left, 0));
#pragma unroll
        for (int i = 0; i < M; ++i) qa[u][i] = head_bytes(qa[u][i], max(left, 0));
      }
      __half2 x[M][16];
#pragma unroll
      for (int i = 0; i < M; ++i) codes32(qa[u][i], x[i]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        __half2 w[16];
        codes32(qb[u][r], w);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          __half2 d0 = __hmul2(x[i][0], w[0]), d1 = __hmul2(x[i][8], w[8]);
#pragma unroll
          for (int c = 1; c < 8; ++c) {  // up to 8 * 36, in quarters: exact
            d0 = __hfma2(x[i][c], w[c], d0);
            d1 = __hfma2(x[i][8 + c], w[8 + c], d1);
          }
          const float2 f0 = __half22float2(d0), f1 = __half22float2(d1);
          acc[r][i] += scaled((f0.x + f0.y) + (f1.x + f1.y), ea[u][i], eb[u][r]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < M; ++i) {
      for (int o = 16; o; o >>= 1) acc[r][i] += __shfl_xor_sync(0xffffffffu, acc[r][i], o);
      if (lane == 0) part[warp][r][i] = acc[r][i];
    }
  __syncthreads();
  if (threadIdx.x < kGroups * R * M) {
    const int g = threadIdx.x / (R * M), r = threadIdx.x / M % R, i = threadIdx.x % M;
    const int col = (blockIdx.x * kGroups + g) * R + r;
    if (col < p.n && i < p.m) {
      float v = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) v += part[g * S + s][r][i];
      ((OT*)p.out)[i * p.ldo + col] = from_f32<OT>(v + (p.bias ? __ldg(p.bias + col) : 0.0f));
    }
  }
}

// ------------------------------------------------------------------ host side

struct Plan4 {
  int bn = 0;             // columns of a tile; 0: row kernel
  bool pair = false;      // tiles of 256 x 256, by pairs
  int m_tiles = 0, n_tiles = 0, k_blocks = 0;
  long long per_cta = 0;  // steps a block, 0: whole tiles
  int grid = 0;
  size_t ws_bytes = 0;
};

Plan4 make_plan4(long long m, long long n, long long k) {
  Plan4 pl;
  if (m == 0 || n == 0 || k == 0) return pl;
  pl.k_blocks = (int)((k + kBK - 1) / kBK);
  if (m == 1 || (m == kRowMax && (double)n * k <= 8e7)) return pl;
  const int sms = sm_count();
  // The tile's width, or pairs' tiles, and whole tiles or even shares of the steps: whichever a model of
  // the time (us, fitted to 17 shapes from 64 x 1024 x 8192 to 131,072 x 1024 x 8192, each run in all four
  // ways) puts first.  It is within 7 % from 60 us on, but leaves out what every product takes (launch, the ring's
  // first loads, the last tile's way out: 3 to 12 us), so small ones take up to several times what it
  // says (64 x 1024 x 8192: 4.7 by it, 6.9 measured; 1813 x 1301 x 322: 2.1 and 12.6); there it only orders the ways.  A step takes 0.33, 0.245 or 0.23 at 256, 128 or 64 columns and 0.284
  // by pairs, a tile's end 1.4, 0.6, 0.5 and 2.6; sharing costs the second launch and 0.3 a megabyte
  // of partial tiles.  Measured: 131,072 x 1024 x 8192 311 by pairs and 339 at 256; x 1024 77 at 256 and 90 by
  // pairs; 1024 x 1664 x 16,384 19 whole at 128 and 22 at 256; 64 x 1024 x 8192 7.6 shared and 10.7 whole.
  double best = 0.0;
  const double step_us[4] = {0.33, 0.245, 0.23, 0.284}, end_us[4] = {1.4, 0.6, 0.5, 2.6};
  const bool fits = ((m + 127) / 128) * ((k + 127) / 128) < 0x7fffffffLL && ((n + 127) / 128) * ((k + 127) / 128) < 0x7fffffffLL;
  for (int w = 0; w < (fits ? 4 : 3); ++w) {
    const bool pair = w == 3;
    const int bn = pair ? 256 : 256 >> w, rows = pair ? 2 * kBM : kBM, workers = pair ? std::max(1, sms / 2) : sms;
    const long long mt = (m + rows - 1) / rows, nt = (n + bn - 1) / bn, tiles = mt * nt, steps = tiles * pl.k_blocks;
    const long long rounds = (tiles + workers - 1) / workers;
    const double whole = (double)rounds * (pl.k_blocks * step_us[w] + end_us[w]);
    const long long per = std::max<long long>((steps + workers - 1) / workers, 2);
    const long long grid = (steps + per - 1) / per;
    const double mb = (double)(grid + tiles) * std::min<long long>(m, rows) * bn * 4e-6;
    const double shared = per * step_us[w] + end_us[w] + 2.6 + 0.3 * mb;
    const bool share = pl.k_blocks > 1 && shared < whole;
    const double us = share ? shared : whole;
    if (w > 0 && us >= best) continue;
    best = us;
    pl.bn = bn;
    pl.pair = pair;
    pl.m_tiles = (int)mt;
    pl.n_tiles = (int)nt;
    pl.per_cta = share ? per : 0;
    pl.grid = (int)(share ? grid : std::min<long long>(tiles, workers));
    pl.ws_bytes = share ? (size_t)(grid + tiles) * rows * bn * sizeof(float) : 0;
  }
  return pl;
}

struct Maps4 {
  CUtensorMap a, b, sa, sb;  // sa, sb: pairs only
};

template <int BN, typename OT>
cudaError_t launch_tiles4(const Matmul4Args& p, const Plan4& pl, const Maps4& t, bool wide, cudaStream_t st) {
  auto* k = wide ? tile4_kernel<BN, OT, true> : tile4_kernel<BN, OT, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg4<BN>::kBytes);
  if (e != cudaSuccess) return e;
  k<<<pl.grid, kThreads, TileCfg4<BN>::kBytes, st>>>(t.a, t.b, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || pl.per_cta == 0) return e;
  join_kernel<BN, OT, Matmul4Args><<<pl.m_tiles * pl.n_tiles * (kBM * BN / 1024), 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename OT>
cudaError_t launch_pairs4(const Matmul4Args& p, const Plan4& pl, const Maps4& t, bool wide, cudaStream_t st) {
  auto* k = wide ? pair4_kernel<OT, true> : pair4_kernel<OT, false>;
  const int bytes = wide ? PairStages4<true>::kBytes : PairStages4<false>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  k<<<2 * pl.grid, kThreads, bytes, st>>>(t.a, t.b, t.sa, t.sb, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || pl.per_cta == 0) return e;
  join_kernel<256, OT, Matmul4Args, 2><<<pl.m_tiles * pl.n_tiles * 2 * (kBM * 256 / 1024), 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <int M, typename OT>
cudaError_t launch_rows4(const Matmul4Args& p, cudaStream_t st) {
  // Enough rows to give every SM 32 warps: four a warp.  Else one a warp, and four warps to a long one.
  if (p.n >= 128 * sm_count() / 2) row4_kernel<M, 1, 4, OT><<<(p.n + 31) / 32, 256, 0, st>>>(p);
  else if (p.k > 2048) row4_kernel<M, 4, 1, OT><<<(p.n + 1) / 2, 256, 0, st>>>(p);
  else row4_kernel<M, 1, 1, OT><<<(p.n + 7) / 8, 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename OT>
cudaError_t launch4(const Matmul4Args& p, const Plan4& pl, const Maps4& t, bool wide, cudaStream_t st) {
  if (p.k == 0) {
    bias_kernel<OT, Matmul4Args><<<(int)std::min<long long>(((long long)p.m * p.n + 255) / 256, 8LL * sm_count()), 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  if (pl.bn == 0) return p.m == 1 ? launch_rows4<1, OT>(p, st) : launch_rows4<2, OT>(p, st);
  if (pl.pair) return launch_pairs4<OT>(p, pl, t, wide, st);
  if (pl.bn == 64) return launch_tiles4<64, OT>(p, pl, t, wide, st);
  if (pl.bn == 128) return launch_tiles4<128, OT>(p, pl, t, wide, st);
  return launch_tiles4<256, OT>(p, pl, t, wide, st);
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_fp4_matmul_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  if (m < 0 || n < 0 || k < 0) return fail(EMB_ERR_INVALID_ARG, "negative m, n or k");
  if (m > 0x7fff0000LL || n > 0x7fff0000LL || k > 0x7fff0000LL) return fail(EMB_ERR_UNSUPPORTED, "m, n or k above 2^31 - 65536");
  const Plan4 pl = make_plan4(m, n, k);
  if (pl.bn && (long long)pl.m_tiles * pl.n_tiles > 0x7fffffffLL / 32)
    return fail(EMB_ERR_UNSUPPORTED, "m * n too large");
  *bytes = pl.ws_bytes;
  return EMB_OK;
}

extern "C" emb_status emb_fp4_matmul(const void* a_d, int64_t lda, const void* sa_d, const void* b_d, int64_t ldb,
                                     const void* sb_d, int64_t m, int64_t n, int64_t k, const float* bias_d, void* out_d,
                                     emb_ftype out_t, int64_t ldo, void* workspace_d, size_t ws_bytes, void* stream) {
  size_t need = 0;
  const emb_status rc = emb_fp4_matmul_workspace_size(m, n, k, &need);
  if (rc != EMB_OK) return rc;
  if (!good_ftype(out_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  const int64_t kb = (k + 1) / 2;
  if (lda < kb || ldb < kb || lda % 16 || ldb % 16) return fail(EMB_ERR_INVALID_ARG, "a row of codes must be a multiple of 16 bytes and hold k");
  if (lda >= (1LL << 39) || ldb >= (1LL << 39)) return fail(EMB_ERR_UNSUPPORTED, "rows of codes over 2^39 bytes apart");
  if (ldo < n) return fail(EMB_ERR_INVALID_ARG, "ldo below n");
  if (m == 0 || n == 0) return EMB_OK;
  if (!out_d || (k > 0 && (!a_d || !b_d || !sa_d || !sb_d))) return fail(EMB_ERR_INVALID_ARG, "a, b, a scale or out is NULL");
  if (!aligned_to(a_d, 16) || !aligned_to(b_d, 16) || !aligned_to(sa_d, 16) || !aligned_to(sb_d, 16))
    return fail(EMB_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  if (!aligned_to(bias_d, 4) || !aligned_to(out_d, ftype_bytes(out_t))) return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (need && (!workspace_d || ws_bytes < need))
    return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_fp4_matmul_workspace_size()");
  if (need && !aligned_to(workspace_d, 32)) return fail(EMB_ERR_WORKSPACE, "workspace must be 32-byte aligned");
  const Plan4 pl = make_plan4(m, n, k);
  int lost;
  unsigned lost_step;
  lost_wait(&lost, &lost_step);
  const int lost_warps[4] = {kTmaWarp, kMmaWarp, -1, kAfterLoads};
  Matmul4Args p{(const unsigned char*)a_d, (const unsigned char*)b_d, (const unsigned char*)sa_d, (const unsigned char*)sb_d,
                bias_d, out_d, (float*)workspace_d, lda, ldb, ldo, (int)m, (int)n, (int)k, pl.m_tiles, pl.n_tiles,
                pl.k_blocks, (int)((k + 127) / 128), (long long)pl.m_tiles * pl.n_tiles * pl.k_blocks, pl.per_cta, nullptr,
                lost < 0 ? -1 : lost_warps[lost], lost_step};
  Maps4 t{};
  if (pl.bn) {
    EMB_CUDA(op_flags(&p.flags));
    bool ok = make_map(&t.a, a_d, m, kb, lda, kBM) && make_map(&t.b, b_d, n, kb, ldb, pl.pair ? kBM : pl.bn);
    if (pl.pair)
      ok = ok && make_scale_map(&t.sa, sa_d, (m + 127) / 128 * p.s_blocks) && make_scale_map(&t.sb, sb_d, (n + 127) / 128 * p.s_blocks);
    if (!ok)
      return fail(EMB_ERR_CUDA, "cuTensorMapEncodeTiled failed or is not available");
  }
  const bool wide = aligned_to(out_d, 32) && (ldo * ftype_bytes(out_t)) % 32 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (out_t == EMB_T_F32) e = launch4<float>(p, pl, t, wide, st);
  else if (out_t == EMB_T_BF16) e = launch4<__nv_bfloat16>(p, pl, t, wide, st);
  else e = launch4<__half>(p, pl, t, wide, st);
  if (e != cudaSuccess) return cuda_fail(e, "emb_fp4_matmul launch");
  return EMB_OK;
}

extern "C" emb_status emb_debug_fp4_matmul_plan(int64_t m, int64_t n, int64_t k, int64_t* plan) {
  size_t bytes = 0;
  if (!plan) return fail(EMB_ERR_INVALID_ARG, "plan is NULL");
  const emb_status rc = emb_fp4_matmul_workspace_size(m, n, k, &bytes);
  if (rc != EMB_OK) return rc;
  const Plan4 pl = make_plan4(m, n, k);
  plan[0] = pl.bn;
  plan[1] = (int64_t)pl.m_tiles * pl.n_tiles;
  plan[2] = pl.grid;
  plan[3] = pl.per_cta;
  plan[4] = pl.pair ? 2 : 1;
  return EMB_OK;
}
