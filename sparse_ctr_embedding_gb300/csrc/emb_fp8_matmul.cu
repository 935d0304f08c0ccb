// Product of two 8-bit block-scaled matrices:
//   out[i, j] = bias[j] + sum_b sa[b, i] sb[b, j] sum_{k in b} a[i, k] b[j, k]
// over blocks b of 128 k's.
//
// Tile kernel.  A persistent block per SM computes tiles of 128 x BN (256, 128
// or 64).  One warp brings 128-byte-wide slabs of both operands into a ring of
// shared memory stages by TMA (128-byte swizzle; rows and columns past the edges
// arrive as zeros); one elected thread issues four tcgen05.mma (e4m3, K = 32
// each) a slab, which sum one scale block in TMEM; eight warps read that sum
// from TMEM and add it, times its scales, to float32 accumulators in registers;
// one warp fetches the scales.  Two TMEM accumulators alternate, so the tensor
// cores work on the next block while the last one is scaled.
//
// What bounds it (BN 256, cycles a block of 128 k's): the products take 512, the
// scaling 304 of TMEM reads and 256 of multiply-adds (512 where b's scales
// differ by column), and with two accumulators the chain products - arrival -
// reads - release takes half its length, about 850, a block.  Times in this file are
// of calls in a loop, unless they say apart (L2 flushed before each call); of a pair,
// both were taken in turn when the choice was made.  131,072 x 1024 x 8192: 770 us
// apart, 2850 TFLOP/s (at 19,456 x 1024 x 4096 the tensor pipe is active 0.59 of the
// time; a product without scales would be 512 of 512); in a loop the power limit
// lowers the clock: 890 to 970, by the operands' values.  8192^3: 431; by rows 597.
// Steps that led here, on the first of these, with pauses between the
// calls: scaling from a fixed register budget and scales loaded where they are used
// 1336; packed multiply-adds, registers split by role 1157; scales three steps ahead
// 972; a warp for the scales 950; the MMA's operands in uniform registers and one
// completion barrier a stage 789; stores of unaligned rows out of the loop's kernel
// 750.
//
// Work is cut into (tile, block) steps.  Whole tiles go to the SMs in turn, or
// all steps are split evenly over the SMs (a tile's blocks then come from several
// SMs: their float32 partial tiles go to the workspace and a second launch adds
// them in order): make_plan() has the rule.  The split depends on the sizes and
// the SM count alone.
//
// Row kernel (one row, or two by a small b): reads b once; plain CUDA cores.
// 1 x 1024 x 8192: 5.5 us from DRAM, 3.9 in a graph of such calls (b then in L2), of
// which 1.2 is the floor and the rest the latency of a launch, of one round of loads
// (codes and scales are asked for together) and of the sums over lanes and warps.
// 1 x 16,384 x 8192: 33 us, floor 20; the conversions of the codes bound it (issue
// active 0.78 of the time, DRAM 0.50).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "emb_dense.cuh"

namespace emb {
namespace {

__device__ unsigned g_op_flags;   // EMB_FLAG_OP_* bits since the last emb_check_op_flag
__device__ unsigned g_op_taken;   // what the last check read

constexpr int kBM = 128;             // rows of a tile
constexpr int kBK = EMB_FP8_BLOCK;   // k's of a step: one scale block, 128 bytes of a row
constexpr int kScaleWarps = 8;
constexpr int kThreads = (kScaleWarps + 4) * 32;  // then a TMA warp, an MMA warp, a warp for the scales, an idle one
// Registers: the scaling warps' accumulators need more than an even share, the other four warps little.
constexpr int kLaunchRegs = 168, kScaleRegs = 224, kOtherRegs = 56;
static_assert(kScaleWarps * 32 * kScaleRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kTmaWarp = kScaleWarps, kMmaWarp = kScaleWarps + 1, kFetchWarp = kScaleWarps + 2;
constexpr int kAhead = 8;            // steps whose scales are held or on their way
constexpr int kAfterLoads = 0;       // lost_warp: not a warp's wait, but the block is told when its last load is issued
constexpr unsigned kWaitLimit = 1u << 21;  // polls of one wait before the kernel gives up

struct MatmulArgs {
  const unsigned char *a, *b;
  const float *sa, *sb, *bias;
  void* out;
  float* partial;            // [slots][kBM * BN]
  long long lda, ldb, ldo;
  long long sa_row, sb_row;  // scales in a row of sa and sb
  int m, n, k;
  int a_shift, b_shift;      // row i's scale is at i >> shift
  int m_tiles, n_tiles, k_blocks;
  long long steps;           // m_tiles * n_tiles * k_blocks
  long long per_cta;         // steps a block takes; 0: whole tiles, block-stride
  int wide_out;              // rows of out are aligned to 32 bytes
  int lost_warp;             // the warp whose wait at step lost_step counts as run out; -1: none
  unsigned lost_step;
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ unsigned smem_u32(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// What a wait that ran out does: the block's other waits end too, and the host is told.
__device__ __forceinline__ bool give_up(volatile int* stop) {
  *stop = 1;
  atomicOr(&g_op_flags, EMB_FLAG_OP_TIMEOUT);
  return false;
}
// Waits for a barrier's phase; false when the limit ran out here or in another
// warp of the block (`stop`), after which the caller leaves its loops.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, volatile int* stop) {
  if (mbar_try(bar, parity)) return true;
  for (unsigned i = 0; i < kWaitLimit; ++i) {
    if (mbar_try(bar, parity)) return true;
    if (*stop) return false;
  }
  return give_up(stop);
}
// After a wait has run out: waits for a barrier of what is still in flight.
__device__ __forceinline__ void mbar_drain(unsigned bar, unsigned parity) {
  for (unsigned i = 0; i < kWaitLimit && !mbar_try(bar, parity); ++i) {}
}
// One lane of a converged warp.  A branch on it (and not on a lane number) lets
// the compiler keep what the lane issues in uniform registers: with the latter
// each tcgen05.mma took about 100 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  unsigned one;
  asm volatile(
      "{\n.reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void tma_load(unsigned dst, const CUtensorMap* map, int x, int y, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_commit(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D[128 x N] (+)= A B^T, 32 k's, e4m3 operands in shared memory.
__device__ __forceinline__ void tc_mma(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
      : "memory");
}
// Starts reading 32 columns of this warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void tc_load32(unsigned addr, unsigned* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_load16(unsigned addr, unsigned* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
// Waits for the loads above; the registers pass through so that no use of them moves before it.
__device__ __forceinline__ void tc_wait32(unsigned* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                 "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tc_wait16(unsigned* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}
template <int N>
__device__ __forceinline__ void tc_load(unsigned addr, unsigned* v) {
  if constexpr (N == 16) tc_load16(addr, v);
  else tc_load32(addr, v);
}
template <int N>
__device__ __forceinline__ void tc_wait(unsigned* v) {
  if constexpr (N == 16) tc_wait16(v);
  else tc_wait32(v);
}

// Two floats side by side, and their products and multiply-adds (one issue slot for two).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void fma2(f32x2 a, f32x2 b, float* c) {
  f32x2 r = pack2(c[0], c[1]);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(a), "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(c[0]), "=f"(c[1]) : "l"(r));
}

// Shared memory descriptor of a K-major operand: rows of 128 bytes, 128-byte
// swizzle (layout 2), eight-row groups 1024 bytes apart, descriptor version 1.
__device__ __forceinline__ unsigned long long smem_desc(unsigned addr) {
  return (unsigned long long)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// ------------------------------------------------------------------ tile kernel

template <int BN>
struct TileCfg {
  static constexpr int kStageBytes = (kBM + BN) * kBK;
  static constexpr int kStages = (196 * 1024) / kStageBytes;  // 4, 6 or 8
  static constexpr int kHalf = BN * 4 / kScaleWarps;          // columns of a scaling warp
  static constexpr int kSlot = kBM + BN;                      // scales of a step: rows, columns
  static constexpr int kScaleBytes = kAhead * kSlot * 4;
  static constexpr int kStoreBytes = kScaleWarps * 32 * 17 * 4;  // 32 rows x 16 columns a warp, for unaligned output
  static constexpr int kBytes = kStages * kStageBytes + kScaleBytes + kStoreBytes + 1024;  // + room to align
};

struct Unit {  // consecutive blocks of one tile
  int tm, tn, kb0, kb1;
  long long tile;
};

// Tiles in groups of 16 rows of tiles, column by column within a group: the
// blocks at work at one time then share few slabs of a and b in L2.
__device__ __forceinline__ void tile_at(const MatmulArgs& p, long long t, int* tm, int* tn) {
  constexpr int kGroup = 16;
  const long long per_group = (long long)kGroup * p.n_tiles;
  const int g = (int)(t / per_group);
  const int in = (int)(t - g * per_group);
  const int rows = min(kGroup, p.m_tiles - g * kGroup);
  *tm = g * kGroup + in % rows;
  *tn = in / rows;
}

// The block's next unit from its position: a tile number, or a step.
__device__ __forceinline__ bool next_unit(const MatmulArgs& p, long long* pos, long long end, Unit* u) {
  if (*pos >= end) return false;
  if (p.per_cta == 0) {
    u->tile = *pos;
    u->kb0 = 0;
    u->kb1 = p.k_blocks;
    *pos += gridDim.x;
  } else {
    u->tile = *pos / p.k_blocks;
    u->kb0 = (int)(*pos - u->tile * p.k_blocks);
    u->kb1 = (int)min((long long)p.k_blocks, u->kb0 + (end - *pos));
    *pos += u->kb1 - u->kb0;
  }
  tile_at(p, u->tile, &u->tm, &u->tn);
  return true;
}
// Where a test asked for a step's wait to run out (emb_debug_lose_op_wait): ends the
// unit before that step, and tells after it that the step is reached.  Not asked in
// the scaling warps, where even once a unit it cost products by rows 3 %.
__device__ __forceinline__ void cut_lost(const MatmulArgs& p, int role, unsigned it, Unit* u) {
  if (p.lost_warp == role) u->kb1 = u->kb0 + (int)min((unsigned)(u->kb1 - u->kb0), p.lost_step - it);
}
__device__ __forceinline__ bool at_lost(const MatmulArgs& p, int role, unsigned it) {
  return p.lost_warp == role && p.lost_step == it;
}
__device__ __forceinline__ void my_range(const MatmulArgs& p, long long* pos, long long* end) {
  if (p.per_cta == 0) {
    *pos = blockIdx.x;
    *end = (long long)p.m_tiles * p.n_tiles;
  } else {
    *pos = blockIdx.x * p.per_cta;
    *end = min(p.steps, *pos + p.per_cta);
  }
}

template <typename OT>
__device__ __forceinline__ void store32(OT* dst, const float* v) {  // 32 bytes
  if constexpr (sizeof(OT) == 4) {
    Raw8<float> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.set2(i, v[2 * i], v[2 * i + 1]);
    r.store((float*)dst);
  } else {
    Raw8<OT> lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo.set2(i, v[2 * i], v[2 * i + 1]);
      hi.set2(i, v[8 + 2 * i], v[8 + 2 * i + 1]);
    }
    const unsigned* a = reinterpret_cast<const unsigned*>(lo.v);
    const unsigned* b = reinterpret_cast<const unsigned*>(hi.v);
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]),
                 "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
                 : "memory");
  }
}

// BCOL: b's scales differ by column (else one per 128 columns: one a warp).
// WIDE: rows of out are aligned to 32 bytes.  (Both ways of storing in one kernel
// cost the main loop its registers: 131,072 x 1024 x 8192 900 us instead of 790, with
// pauses between the calls.)
template <int BN, typename OT, bool BCOL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ CUtensorMap map_a,
                                                           const __grid_constant__ CUtensorMap map_b,
                                                           const __grid_constant__ MatmulArgs p) {
  using C = TileCfg<BN>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long bars[2 * C::kStages + 2 + 2 * kAhead];
  __shared__ unsigned tmem_slot;
  __shared__ int stop_flag;
  __shared__ unsigned issued[3];  // steps whose loads, products and scales were issued
  volatile int* stop = &stop_flag;
  const unsigned smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // full: a stage's slabs are there.  done: its products are, so the stage may be
  // filled again and its sums be read.  tempty: a TMEM accumulator has been read.
  // sfull, sempty: the scales of a step.
  const unsigned full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages, tempty0 = done0 + 8 * C::kStages;
  const unsigned sfull0 = tempty0 + 16, sempty0 = sfull0 + 8 * kAhead;
  float* const ring = reinterpret_cast<float*>(raw + (smem - smem_u32(raw)) + C::kStages * C::kStageBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) mbar_init(tempty0 + 8 * t, kScaleWarps);
    for (int s = 0; s < kAhead; ++s) {
      mbar_init(sfull0 + 8 * s, 32);
      mbar_init(sempty0 + 8 * s, kScaleWarps);
    }
    stop_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(2 * BN) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = tmem_slot;

  long long pos, end;
  my_range(p, &pos, &end);
  Unit u;

  if (warp >= kScaleWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {  // TMA: both slabs of each step
      unsigned it = 0;
      bool go = true;
      while (go && next_unit(p, &pos, end, &u)) {
        cut_lost(p, kTmaWarp, it, &u);
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
          const unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
          go = __all_sync(0xffffffffu, mbar_wait(done0 + 8 * s, ph ^ 1, stop));
          if (!go) break;
          if (elect_one()) {
            const unsigned dst = smem + s * C::kStageBytes, bar = full0 + 8 * s;
            mbar_expect_tx(bar, C::kStageBytes);
            tma_load(dst, &map_a, kb * kBK, u.tm * kBM, bar);
            tma_load(dst + kBM * kBK, &map_b, kb * kBK, u.tn * BN, bar);
          }
          __syncwarp();
        }
        if (go && at_lost(p, kTmaWarp, it)) go = give_up(stop);
      }
      if (p.lost_warp == kAfterLoads) give_up(stop);
      issued[0] = it;
    }
    if (warp == kMmaWarp) {
      // f32 accumulator, e4m3 x e4m3, both K-major, N = BN, M = 128
      constexpr unsigned idesc = (1u << 4) | ((BN >> 3) << 17) | ((kBM >> 4) << 24);
      unsigned it = 0;
      bool go = true;
      while (go && next_unit(p, &pos, end, &u)) {
        cut_lost(p, kMmaWarp, it, &u);
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
          const unsigned s = it % C::kStages, ph = (it / C::kStages) & 1;
          const unsigned t = it & 1, tph = (it >> 1) & 1;
          const bool ready_t = mbar_try(tempty0 + 8 * t, tph ^ 1), ready_f = mbar_try(full0 + 8 * s, ph);
          go = (ready_t || mbar_wait(tempty0 + 8 * t, tph ^ 1, stop)) && (ready_f || mbar_wait(full0 + 8 * s, ph, stop));
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          tc_fence_after();
          const unsigned at = smem + s * C::kStageBytes;
          const unsigned long long da = smem_desc(at), db = smem_desc(at + kBM * kBK);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < kBK / 32; ++j) tc_mma(tmem + t * BN, da + 2 * j, db + 2 * j, idesc, j > 0);
            tc_commit(done0 + 8 * s);
          }
          __syncwarp();
        }
        if (go && at_lost(p, kMmaWarp, it)) go = give_up(stop);
      }
      issued[1] = it;
    }
    if (warp == kFetchWarp) {
      // The steps' scales, by 4-byte asynchronous copies (rows of scales have no
      // alignment), up to kAhead steps early: each is a new cache line.
      unsigned it = 0;
      bool go = true;
      while (go && next_unit(p, &pos, end, &u)) {
        cut_lost(p, kFetchWarp, it, &u);
        const float *sa[kBM / 32], *sb[BCOL ? BN / 32 : 1];
#pragma unroll
        for (int i = 0; i < kBM / 32; ++i)
          sa[i] = p.sa + u.kb0 * p.sa_row + (min(u.tm * kBM + i * 32 + lane, p.m - 1) >> p.a_shift);
#pragma unroll
        for (int i = 0; i < (BCOL ? BN / 32 : 1); ++i)
          sb[i] = p.sb + u.kb0 * p.sb_row + (min(u.tn * BN + (BCOL ? i * 32 + lane : lane * kBK), p.n - 1) >> p.b_shift);
        for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
          const unsigned slot = it % kAhead;
          go = __all_sync(0xffffffffu, mbar_wait(sempty0 + 8 * slot, ((it / kAhead) & 1) ^ 1, stop));
          if (!go) break;
          const unsigned at = smem_u32(ring + slot * C::kSlot + lane);
#pragma unroll
          for (int i = 0; i < kBM / 32; ++i, sa[i - 1] += p.sa_row)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 128 * i), "l"(sa[i]) : "memory");
          if (BCOL || lane < (BN + kBK - 1) / kBK) {
#pragma unroll
            for (int i = 0; i < (BCOL ? BN / 32 : 1); ++i, sb[i - 1] += p.sb_row)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 4 * kBM + 128 * i), "l"(sb[i]) : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sfull0 + 8 * slot) : "memory");
        }
        if (go && at_lost(p, kFetchWarp, it)) go = give_up(stop);
      }
      issued[2] = it;
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncwarp();
  } else {  // scaling warps: TMEM lanes 32 (warp % 4).., columns group (warp / 4)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kScaleRegs));
    const int half = warp >> 2, quarter = warp & 3;
    float* const stage = ring + kAhead * C::kSlot + warp * 32 * 17;
    unsigned it = 0;
    bool go = true;
    while (go && next_unit(p, &pos, end, &u)) {
      const int row = u.tm * kBM + quarter * 32 + lane;
      const int col0 = u.tn * BN + half * C::kHalf;
      float acc[C::kHalf];
#pragma unroll
      for (int c = 0; c < C::kHalf; ++c) acc[c] = 0.0f;
      for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
        const unsigned t = it & 1, slot = it % kAhead, stage = it % C::kStages, ph = (it / C::kStages) & 1;
        const float* sl = ring + slot * C::kSlot + quarter * 32 + lane;
        const float* sb = ring + slot * C::kSlot + kBM + (BCOL ? half * C::kHalf : half * C::kHalf / kBK);
        go = mbar_wait(sfull0 + 8 * slot, (it / kAhead) & 1, stop);
        float s = 0.0f;
        if (go) s = BCOL ? *sl : *sl * *sb;
        go = go && mbar_wait(done0 + 8 * stage, ph, stop);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        if (!BCOL) {  // all lanes have read their scales: the vote above orders no memory
          __syncwarp();
          if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
        }
        tc_fence_after();
        const unsigned taddr = tmem + ((unsigned)(quarter * 32) << 16) + t * BN + half * C::kHalf;
        // Columns in chunks: the next one, and its scales, are on their way while one is added.
        constexpr int kChunk = BCOL ? 16 : 32, kChunks = C::kHalf / kChunk;
        const f32x2 s2 = pack2(s, s);
        unsigned v[2][kChunk];
        float4 b[2][BCOL ? kChunk / 4 : 1];
        auto start = [&](int c) {
          if constexpr (BCOL) {
#pragma unroll
            for (int j = 0; j < kChunk / 4; ++j) b[c & 1][j] = *reinterpret_cast<const float4*>(sb + c * kChunk + 4 * j);
          }
          tc_load<kChunk>(taddr + c * kChunk, v[c & 1]);
        };
        start(0);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          tc_wait<kChunk>(v[c & 1]);
          if (c + 1 < kChunks) {
            start(c + 1);
          } else {  // all of this accumulator is in registers: the MMA may write it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty0 + 8 * t);
          }
          const unsigned* w = v[c & 1];
          float* o = acc + c * kChunk;
#pragma unroll
          for (int j = 0; j < kChunk; j += 2) {
            const f32x2 x = pack2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
            if constexpr (BCOL) {
              const float4& q = b[c & 1][j / 4];
              fma2(x, mul2(s2, j % 4 == 0 ? pack2(q.x, q.y) : pack2(q.z, q.w)), o + j);
            } else {
              fma2(x, s2, o + j);
            }
          }
        }
        if constexpr (BCOL) {
          __syncwarp();
          if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
        }
      }
      if (!go) break;
      if (u.kb0 == 0 && u.kb1 == p.k_blocks) {
        if constexpr (WIDE) {
          if (row < p.m) {
            OT* dst = (OT*)p.out + row * p.ldo + col0;
            constexpr int kVec = 32 / sizeof(OT);
#pragma unroll
            for (int c = 0; c < C::kHalf; c += kVec) {
              if (p.bias) {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                  if (col0 + c + j < p.n) acc[c + j] += __ldg(p.bias + col0 + c + j);
              }
              if (col0 + c + kVec <= p.n) {
                store32<OT>(dst + c, acc + c);
              } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                  if (col0 + c + j < p.n) dst[c + j] = from_f32<OT>(acc[c + j]);
              }
            }
          }
        } else {
          // through shared memory, so that a half warp stores 16 neighbours of a row
          // (10,046 x 1293 x 475 to f16: 155 us with a row to a lane, 61 so; 39 by now)
#pragma unroll
          for (int c = 0; c < C::kHalf; c += 16) {
            if (col0 + c >= p.n) break;  // the same for the warp
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = acc[c + j];
            __syncwarp();
            const int col = col0 + c + (lane & 15);
            const float bias = p.bias && col < p.n ? __ldg(p.bias + col) : 0.0f;
            OT* dst = (OT*)p.out + (row - lane) * p.ldo + col;
#pragma unroll 4
            for (int r = lane >> 4; r < 32; r += 2)
              if (row - lane + r < p.m && col < p.n) dst[r * p.ldo] = from_f32<OT>(stage[r * 17 + (lane & 15)] + bias);
          }
        }
      } else if (row < p.m) {  // part of a tile: slot (block + tile) is this piece's alone
        float* dst = p.partial + (long long)(blockIdx.x + u.tile) * kBM * BN + (warp * C::kHalf * 4 + lane) * 8;
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 8) store32<float>(dst + c * 32, acc + c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // A wait ran out, of whichever warp: those that issued copies or products may have
  // left their loops in good order, with some in flight that no one has waited for.
  // They land before TMEM is freed and the block ends.
  if (*stop) {  // the same for the block: written before the barrier only
    const unsigned n = warp < kScaleWarps + 3 && warp >= kScaleWarps ? issued[warp - kScaleWarps] : 0;
    if (warp == kTmaWarp)
      for (unsigned j = n - min(n, (unsigned)C::kStages); j < n; ++j) mbar_drain(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
    if (warp == kMmaWarp && n > 0) mbar_drain(done0 + 8 * ((n - 1) % C::kStages), ((n - 1) / C::kStages) & 1);
    if (warp == kFetchWarp)
      for (unsigned j = n - min(n, (unsigned)kAhead); j < n; ++j) mbar_drain(sfull0 + 8 * (j % kAhead), (j / kAhead) & 1);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN));
  }
}

// Adds the pieces of each tile that several blocks computed, in k order.  A piece
// lies as the scaling warps store it, whole kilobytes at a time: by warps, by 8
// columns, by rows (1664 x 452 x 30,584 to bf16: 52 us, and 56 with pieces laid
// out by rows).  One block takes 32 rows x 32 columns, four columns a thread.
template <int BN, typename OT>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ MatmulArgs p) {
  constexpr int kBlocks = kBM * BN / 1024, kHalf = TileCfg<BN>::kHalf, kWarpBlocks = kHalf / 32;
  const long long tile = blockIdx.x / kBlocks;
  const int q = (int)(blockIdx.x % kBlocks), warp = q / kWarpBlocks, x = threadIdx.x / 8, y = threadIdx.x % 8;
  const long long first = tile * p.k_blocks / p.per_cta, last = ((tile + 1) * p.k_blocks - 1) / p.per_cta;
  if (first == last) return;  // one block had it whole
  int tm, tn;
  tile_at(p, tile, &tm, &tn);
  const int row = tm * kBM + (warp & 3) * 32 + x, col = tn * BN + (warp >> 2) * kHalf + q % kWarpBlocks * 32 + y * 4;
  if (row >= p.m || col >= p.n) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* src = p.partial + (first + tile) * kBM * BN + q * 1024 + y / 2 * 256 + x * 8 + y % 2 * 4;
#pragma unroll 8
  for (long long b = first; b <= last; ++b, src += (long long)kBM * BN) {
    const float4 w = *reinterpret_cast<const float4*>(src);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < p.n) ((OT*)p.out)[row * p.ldo + col + j] = from_f32<OT>(o[j] + (p.bias ? __ldg(p.bias + col + j) : 0.0f));
}

// ------------------------------------------------------------------ row kernel

constexpr int kRowMax = 2;

// 16 codes as floats.
__device__ __forceinline__ void codes16(const uint4& q, float* o) {
  const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_f32((unsigned short)(w[i] & 0xffffu)), b = e4m3x2_to_f32((unsigned short)(w[i] >> 16));
    o[4 * i] = a.x;
    o[4 * i + 1] = a.y;
    o[4 * i + 2] = b.x;
    o[4 * i + 3] = b.y;
  }
}
// Clears the codes from `keep` on (keep < 16).
__device__ __forceinline__ uint4 head16(uint4 q, int keep) {
  unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = keep - 4 * i;
    w[i] = left >= 4 ? w[i] : left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A block's eight warps take 8 / S groups of R rows of b, S warps to a group; a
// lane takes 16 neighbouring k's (one scale block for eight lanes) every 512 S.
// R rows share a's codes and their conversion, half of the work otherwise; eight
// pieces of b are on their way at a time (four at R = 1).
template <int M, int S, int R, typename OT>
__global__ void __launch_bounds__(256) row_kernel(const __grid_constant__ MatmulArgs p) {
  constexpr int kGroups = 8 / S, kBatch = R == 1 ? 4 : 8 / R;
  __shared__ float part[8][R][M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x * kGroups + warp / S) * R;
  float acc[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < M; ++i) acc[r][i] = 0.0f;
  const unsigned char* b[R];
  const float* sb[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = min(j0 + r, p.n - 1);  // past the last row: read again, not stored
    b[r] = p.b + j * p.ldb;
    sb[r] = p.sb + (j >> p.b_shift);
  }
  for (int k0 = ((warp % S) * 32 + lane) * 16; k0 < p.k; k0 += kBatch * S * 512) {
    uint4 qb[kBatch][R], qa[kBatch][M];
    float s[kBatch][R], t[kBatch][M];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = k0 + u * S * 512;
      const bool in = k < p.k;
      const int kb = k / kBK;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        qb[u][r] = in ? __ldg(reinterpret_cast<const uint4*>(b[r] + k)) : make_uint4(0, 0, 0, 0);  // rows are multiples of 16 bytes
        s[u][r] = in ? __ldg(sb[r] + kb * p.sb_row) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < M; ++i) {
        qa[u][i] = in && i < p.m ? __ldg(reinterpret_cast<const uint4*>(p.a + i * p.lda + k)) : make_uint4(0, 0, 0, 0);
        t[u][i] = in && i < p.m ? __ldg(p.sa + kb * p.sa_row + (i >> p.a_shift)) : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int left = p.k - (k0 + u * S * 512);
      if (left < 16) {  // the row's last piece: what lies past k does not count
#pragma unroll
        for (int r = 0; r < R; ++r) qb[u][r] = head16(qb[u][r], max(left, 0));
#pragma unroll
        for (int i = 0; i < M; ++i) qa[u][i] = head16(qa[u][i], max(left, 0));
      }
      float x[M][16];
#pragma unroll
      for (int i = 0; i < M; ++i) codes16(qa[u][i], x[i]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float w[16];
        codes16(qb[u][r], w);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          float d = 0.0f;
#pragma unroll
          for (int c = 0; c < 16; ++c) d = fmaf(x[i][c], w[c], d);
          acc[r][i] = fmaf(d, s[u][r] * t[u][i], acc[r][i]);
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

// out = bias: a product over no k's.
template <typename OT>
__global__ void __launch_bounds__(256) bias_kernel(const __grid_constant__ MatmulArgs p) {
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < (long long)p.m * p.n; e += (long long)gridDim.x * 256) {
    const long long i = e / p.n, j = e - i * p.n;
    ((OT*)p.out)[i * p.ldo + j] = from_f32<OT>(p.bias ? p.bias[j] : 0.0f);
  }
}

// Reads and clears the flag word in one step: a kernel of another stream may raise a bit at any time.
__global__ void take_flags_kernel() { g_op_taken = atomicExch(&g_op_flags, 0u); }

// ------------------------------------------------------------------ host side

std::atomic<int> g_lost_warp{-1};  // emb_debug_lose_op_wait
std::atomic<unsigned> g_lost_step{0};

struct Plan {
  int bn = 0;             // 0: row kernel
  int m_tiles = 0, n_tiles = 0, k_blocks = 0;
  long long per_cta = 0;  // steps a block, 0: whole tiles
  int grid = 0;
  size_t ws_bytes = 0;
};

Plan make_plan(long long m, long long n, long long k) {
  Plan pl;
  if (m == 0 || n == 0 || k == 0) return pl;
  pl.k_blocks = (int)((k + kBK - 1) / kBK);
  // 1 x 16,384 x 8192: 37 us by rows, 45 by tiles; 2 x 8192 x 8192 29 and 23, 2 x 4096 x 8192 18 and 21.
  // The bound for two rows lies between the last two sizes (6.7e7 and 3.4e7 codes); others were not measured.
  if (m == 1 || (m == kRowMax && (double)n * k <= 4e7)) return pl;
  const int sms = sm_count();
  const long long mt = (m + kBM - 1) / kBM;
  // The tile's width, and whole tiles or even shares of the steps: whichever a
  // model of the time (us, fitted to 20 shapes from 64 x 1024 x 8192 to 30,584 x
  // 452 x 692, within 30 % of each) puts first.  A step of 256, 128 or 64
  // columns takes 0.48, 0.33 or 0.29, a tile's end 3.3, 2 or 2; sharing costs the
  // second launch and 0.42 a megabyte of partial tiles.  Measured: 9853 x 448 x
  // 2560 30 whole and 41 shared at 256; 1024 x 1664 x 16,384 64 and 46; 1024 x
  // 8192 x 131,072 by rows 1250 and 1470.  One set of constants serves both kinds of
  // scales: the size of the workspace does not depend on the kind.  By rows a step
  // takes up to 1.4 times as long (8192^3 597 us, 431), which lengthens both sides.
  double best = 0.0;
  const double step_us[3] = {0.48, 0.33, 0.29}, end_us[3] = {3.3, 2.0, 2.0};
  for (int w = 0; w < 3; ++w) {
    const int bn = 256 >> w;
    const long long nt = (n + bn - 1) / bn, tiles = mt * nt, steps = tiles * pl.k_blocks;
    const long long rounds = (tiles + sms - 1) / sms;
    const double whole = (double)rounds * (pl.k_blocks * step_us[w] + end_us[w]);
    const long long per = std::max<long long>((steps + sms - 1) / sms, 2);
    const long long grid = (steps + per - 1) / per;
    const double mb = (double)(grid + tiles) * std::min<long long>(m, kBM) * bn * 4e-6;
    // blocks at different k's share no slabs: from DRAM a step then takes half as long again
    const double far = (double)(m + n) * k > 64e6 ? 1.5 : 1.0;
    const double shared = per * step_us[w] * far + end_us[w] + 4.0 + 0.42 * mb;
    const bool share = pl.k_blocks > 1 && shared < whole;
    const double us = share ? shared : whole;
    if (w > 0 && us >= best) continue;
    best = us;
    pl.bn = bn;
    pl.n_tiles = (int)nt;
    pl.per_cta = share ? per : 0;
    pl.grid = (int)(share ? grid : std::min<long long>(tiles, sms));
    pl.ws_bytes = share ? (size_t)(grid + tiles) * kBM * bn * sizeof(float) : 0;
  }
  pl.m_tiles = (int)mt;
  return pl;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeTiled)f;
  }();
  return fn;
}

// Slabs of 128 k's by `box_rows` rows of a code matrix; what lies outside is read as zeros.
bool make_map(CUtensorMap* map, const void* base, long long rows, long long k, long long ld, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename OT>
cudaError_t launch_tiles(const MatmulArgs& p, const Plan& pl, const CUtensorMap& ma, const CUtensorMap& mb, cudaStream_t st) {
  auto* k = p.wide_out ? (p.b_shift ? tile_kernel<BN, OT, false, true> : tile_kernel<BN, OT, true, true>)
                       : (p.b_shift ? tile_kernel<BN, OT, false, false> : tile_kernel<BN, OT, true, false>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<BN>::kBytes);
  if (e != cudaSuccess) return e;
  k<<<pl.grid, kThreads, TileCfg<BN>::kBytes, st>>>(ma, mb, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || pl.per_cta == 0) return e;
  join_kernel<BN, OT><<<pl.m_tiles * pl.n_tiles * (kBM * BN / 1024), 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <int M, typename OT>
cudaError_t launch_rows(const MatmulArgs& p, cudaStream_t st) {
  // Enough rows to give every SM 32 warps: four a warp.  Else one a warp, and four warps to a long one.
  if (p.n >= 128 * sm_count() / 2) row_kernel<M, 1, 4, OT><<<(p.n + 31) / 32, 256, 0, st>>>(p);
  else if (p.k > 1024) row_kernel<M, 4, 1, OT><<<(p.n + 1) / 2, 256, 0, st>>>(p);
  else row_kernel<M, 1, 1, OT><<<(p.n + 7) / 8, 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename OT>
cudaError_t launch(const MatmulArgs& p, const Plan& pl, const CUtensorMap& ma, const CUtensorMap& mb, cudaStream_t st) {
  if (p.k == 0) {
    bias_kernel<OT><<<(int)std::min<long long>(((long long)p.m * p.n + 255) / 256, 8LL * sm_count()), 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  if (pl.bn == 0) {
    return p.m == 1 ? launch_rows<1, OT>(p, st) : launch_rows<2, OT>(p, st);
  }
  if (pl.bn == 64) return launch_tiles<64, OT>(p, pl, ma, mb, st);
  if (pl.bn == 128) return launch_tiles<128, OT>(p, pl, ma, mb, st);
  return launch_tiles<256, OT>(p, pl, ma, mb, st);
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  if (m < 0 || n < 0 || k < 0) return fail(EMB_ERR_INVALID_ARG, "negative m, n or k");
  if (m > 0x7fff0000LL || n > 0x7fff0000LL || k > 0x7fff0000LL) return fail(EMB_ERR_UNSUPPORTED, "m, n or k above 2^31 - 65536");
  const Plan pl = make_plan(m, n, k);
  if (pl.bn && (long long)pl.m_tiles * pl.n_tiles > 0x7fffffffLL / 32)
    return fail(EMB_ERR_UNSUPPORTED, "m * n too large");
  *bytes = pl.ws_bytes;
  return EMB_OK;
}

extern "C" emb_status emb_fp8_matmul(const void* a_d, int64_t lda, const float* sa_d, int32_t a_block_rows,
                                     const void* b_d, int64_t ldb, const float* sb_d, int32_t b_block_rows, int64_t m,
                                     int64_t n, int64_t k, const float* bias_d, void* out_d, emb_ftype out_t, int64_t ldo,
                                     void* workspace_d, size_t ws_bytes, void* stream) {
  size_t need = 0;
  const emb_status rc = emb_fp8_matmul_workspace_size(m, n, k, &need);
  if (rc != EMB_OK) return rc;
  if (!good_ftype(out_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  if ((a_block_rows != 1 && a_block_rows != EMB_FP8_BLOCK) || (b_block_rows != 1 && b_block_rows != EMB_FP8_BLOCK))
    return fail(EMB_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (lda < k || ldb < k || lda % 16 || ldb % 16) return fail(EMB_ERR_INVALID_ARG, "a row of codes must be a multiple of 16 bytes and hold k");
  if (lda >= (1LL << 39) || ldb >= (1LL << 39)) return fail(EMB_ERR_UNSUPPORTED, "rows of codes over 2^39 bytes apart");
  if (ldo < n) return fail(EMB_ERR_INVALID_ARG, "ldo below n");
  if (m == 0 || n == 0) return EMB_OK;
  if (!out_d || (k > 0 && (!a_d || !b_d || !sa_d || !sb_d))) return fail(EMB_ERR_INVALID_ARG, "a, b, a scale or out is NULL");
  if (!aligned_to(a_d, 16) || !aligned_to(b_d, 16)) return fail(EMB_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (!aligned_to(sa_d, 4) || !aligned_to(sb_d, 4) || !aligned_to(bias_d, 4) || !aligned_to(out_d, ftype_bytes(out_t)))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (need && (!workspace_d || ws_bytes < need))
    return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_fp8_matmul_workspace_size()");
  if (need && !aligned_to(workspace_d, 32)) return fail(EMB_ERR_WORKSPACE, "workspace must be 32-byte aligned");
  const Plan pl = make_plan(m, n, k);
  const int as = a_block_rows == 1 ? 0 : 7, bs = b_block_rows == 1 ? 0 : 7;
  const size_t ob = ftype_bytes(out_t);
  const MatmulArgs p{(const unsigned char*)a_d, (const unsigned char*)b_d, sa_d, sb_d, bias_d, out_d, (float*)workspace_d,
                     lda, ldb, ldo, as ? (m + 127) / 128 : m, bs ? (n + 127) / 128 : n, (int)m, (int)n, (int)k, as, bs,
                     pl.m_tiles, pl.n_tiles, pl.k_blocks, (long long)pl.m_tiles * pl.n_tiles * pl.k_blocks, pl.per_cta,
                     aligned_to(out_d, 32) && (ldo * ob) % 32 == 0, g_lost_warp.load(), g_lost_step.load()};
  CUtensorMap ma{}, mb{};
  if (pl.bn && (!make_map(&ma, a_d, m, k, lda, kBM) || !make_map(&mb, b_d, n, k, ldb, pl.bn)))
    return fail(EMB_ERR_CUDA, "cuTensorMapEncodeTiled failed or is not available");
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (out_t == EMB_T_F32) e = launch<float>(p, pl, ma, mb, st);
  else if (out_t == EMB_T_BF16) e = launch<__nv_bfloat16>(p, pl, ma, mb, st);
  else e = launch<__half>(p, pl, ma, mb, st);
  if (e != cudaSuccess) return cuda_fail(e, "emb_fp8_matmul launch");
  return EMB_OK;
}

extern "C" emb_status emb_debug_lose_op_wait(int32_t role, int64_t step) {
  if (role < -1 || role > 3 || step < 0 || step > 0x7fffffffLL) return fail(EMB_ERR_INVALID_ARG, "role must be -1 to 3, step 0 to 2^31 - 1");
  const int warps[4] = {kTmaWarp, kMmaWarp, kFetchWarp, kAfterLoads};
  g_lost_step.store((unsigned)step);
  g_lost_warp.store(role < 0 ? -1 : warps[role]);
  return EMB_OK;
}

extern "C" emb_status emb_debug_fp8_matmul_plan(int64_t m, int64_t n, int64_t k, int64_t* plan) {
  size_t bytes = 0;
  if (!plan) return fail(EMB_ERR_INVALID_ARG, "plan is NULL");
  const emb_status rc = emb_fp8_matmul_workspace_size(m, n, k, &bytes);
  if (rc != EMB_OK) return rc;
  const Plan pl = make_plan(m, n, k);
  plan[0] = pl.bn;
  plan[1] = (int64_t)pl.m_tiles * pl.n_tiles;
  plan[2] = pl.grid;
  plan[3] = pl.per_cta;
  return EMB_OK;
}

extern "C" emb_status emb_check_op_flag(void* stream, uint32_t* flags_out) {
  static std::mutex one_check;  // g_op_taken holds one check's bits at a time
  const std::lock_guard<std::mutex> hold(one_check);
  cudaStream_t st = (cudaStream_t)stream;
  unsigned f = 0;
  take_flags_kernel<<<1, 1, 0, st>>>();
  EMB_CUDA(cudaGetLastError());
  EMB_CUDA(cudaMemcpyFromSymbolAsync(&f, g_op_taken, sizeof f, 0, cudaMemcpyDeviceToHost, st));
  EMB_CUDA(cudaStreamSynchronize(st));
  if (flags_out) *flags_out = f;
  if (f) return fail(EMB_ERR_DEVICE_FLAG, "a dense operator's bounded wait ran out: its output is not valid");
  return EMB_OK;
}
