// PTX of the tensor-core operators (emb_fp8_matmul.cu, emb_fp4_matmul.cu, emb_muon.cu):
// mbarriers with bounded waits, TMA loads, TMEM reads, operand descriptors, 32-byte stores.
#pragma once

#include <cuda.h>

#include "emb_dense.cuh"

namespace emb {

// The flag word of the current device that emb_check_op_flag reads (emb_fp8_matmul.cu).
cudaError_t op_flags(unsigned** word);
// What emb_debug_lose_op_wait asked for (emb_fp8_matmul.cu).
void lost_wait(int* role, unsigned* step);

constexpr unsigned kWaitLimit = 1u << 21;  // polls of one wait before the kernel gives up

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
// What a wait that ran out does: the block's other waits end too, and the host is told
// (`flags`: the word that emb_check_op_flag reads).
__device__ __forceinline__ bool give_up(volatile int* stop, unsigned* flags) {
  *stop = 1;
  atomicOr(flags, EMB_FLAG_OP_TIMEOUT);
  return false;
}
// Waits for a barrier's phase; false when the limit ran out here or in another
// warp of the block (`stop`), after which the caller leaves its loops.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, volatile int* stop, unsigned* flags) {
  if (mbar_try(bar, parity)) return true;
  for (unsigned i = 0; i < kWaitLimit; ++i) {
    if (mbar_try(bar, parity)) return true;
    if (*stop) return false;
  }
  return give_up(stop, flags);
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

// Shared memory descriptor of a K-major operand: rows of 128 bytes, 128-byte
// swizzle (layout 2), eight-row groups 1024 bytes apart, descriptor version 1.
__device__ __forceinline__ unsigned long long smem_desc(unsigned addr) {
  return (unsigned long long)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// ------------------------------------------------------------------ pairs of SMs (clusters of two blocks)
//
// A pair's MMAs are issued by its first block ("leader"); loads of both signal its barriers,
// completions go to both.  A wait that runs out raises `stop` (a word at the same place of both
// blocks' shared memory) in both.

__device__ __forceinline__ unsigned peer_addr(unsigned addr, unsigned rank) {
  unsigned r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ bool pair_give_up(unsigned stop, unsigned* flags) {
  for (unsigned r = 0; r < 2; ++r)
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(peer_addr(stop, r)) : "memory");
  atomicOr(flags, EMB_FLAG_OP_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool pair_stopped(unsigned stop) {
  unsigned v;
  asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(stop) : "memory");
  return v != 0;
}
__device__ __forceinline__ bool pair_try(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool pair_wait(unsigned bar, unsigned parity, unsigned stop, unsigned* flags) {
  if (pair_try(bar, parity)) return true;
  for (unsigned i = 0; i < kWaitLimit; ++i) {
    if (pair_try(bar, parity)) return true;
    if (pair_stopped(stop)) return false;
  }
  return pair_give_up(stop, flags);
}
__device__ __forceinline__ void pair_arrive(unsigned bar, unsigned rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, rank)) : "memory");
}
// After a wait has run out: waits for a barrier of what is still in flight.  Where the other block
// gave up first the barrier may never complete, so a millisecond at most (for each barrier; a ring has up to six):
// loads take microseconds.
__device__ __forceinline__ void pair_drain(unsigned bar, unsigned parity) {
  const long long from = clock64();
  while (!mbar_try(bar, parity) && clock64() - from < 2000000) {}
}
// ... and lets loads of the other block land that the leader no longer expects.
__device__ __forceinline__ void pair_settle() {
  for (int i = 0; i < 200; ++i) __nanosleep(1000);
}
// A TMA load that signals the leader's barrier (`bar`: its address in the cluster).
__device__ __forceinline__ void tma_load_pair(unsigned dst, const CUtensorMap* map, int x, int y, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void commit_both(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"((unsigned short)3)
               : "memory");
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

}  // namespace emb
