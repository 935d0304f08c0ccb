// Muon: momentum, orthogonalised by Newton-Schulz steps, as the update of matrices.
//   m = beta m + (1 - beta) g;  u = (1 - beta) g + beta m (Nesterov) or m;  X = u / (|u| + 1e-7)
//   five times:  A = X X^T;  B = b A + c A^2;  X = a X + B X        (X with its short side first)
//   p = p (1 - lr wd) - lr scale X
//
// Launches, each over all matrices of a call: the momentum with the sum of u's
// squares; X; then three a step, "gram" (A), "square" (B) and "apply" (X), the last of
// which writes the weights.  Everything between lies in the workspace.
//
// Products.  Operands are float16 with float32 sums on tcgen05.  X, A and B are kept
// times 2^12: singular values stay below about 1.25, so entries stay below 2^14, and
// entries down to 2^-26 keep their 11 bits.  "half" keeps one float16 of each: 2^-11
// a rounding, an eighth of what bfloat16 loses in the same step at the same rate.  "split"
// keeps two, the second what the first one lost (22 bits together), and takes three
// products of the four: float32's accuracy at a third of the rate.
//
// Layout.  A matrix lies in the workspace as the tensor cores read it from shared
// memory: tiles of 128 rows x 64 columns, a row 128 bytes, its 16-byte pieces swizzled,
// zeros past the edges.  A tile is 16 KB in one piece, so loads are plain bulk copies
// without a tensor map, whatever the matrix's shape.  The same tiles serve X^T: for X
// on the right of B its 64 x 64 halves are read as the operand whose columns are
// contiguous.  A and A^2 are symmetric: only tiles on and below the diagonal are
// computed, and written twice.
//
// Work is cut into items, a tile of 128 x 128 or a part of its k's where there are
// fewer tiles than SMs; a part's float32 sums go to the workspace, and the block that
// completes a tile adds them in k order (results do not depend on which block that is).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "emb_tc.cuh"

namespace emb {
namespace {

constexpr int kMaxMats = 128;       // matrices of one launch: bounded by the kernel's parameters
constexpr int kTileRows = 128, kSlab = 64;
constexpr int kTileBytes = kTileRows * kSlab * 2;   // 16 KB
constexpr int kBN = 128;
constexpr int kChunk = 8192;        // elements of a block in the momentum kernel
constexpr int kSteps = 5;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 4096.0f, kInvScale = 1.0f / 4096.0f;
constexpr int kSumWarps = 8, kThreads = (kSumWarps + 2) * 32, kLoadWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
constexpr int kAfterLoads = 0;
constexpr int kWhole = 1 << 30;     // per: tiles are not shared out

enum Phase { kGram = 0, kSquare = 1, kApply = 2 };

struct Mat {
  void* p;
  float* m;
  const void* g;
  long long x, a, b;        // tiles in the workspace: X (two buffers of x_tiles), A, B
  int rows, cols;           // of the parameter
  int s, l;                 // short and long side
  int sb, lb;               // blocks of 128 along each
  int first[5];             // of this matrix among all: items of the three phases, chunks, tiles of X
  int param_t, grad_t;
  float scale;
};

struct MuonArgs {
  unsigned char* ws;        // tiles
  float* partial;           // [slots][128 * kBN]
  unsigned* count;          // [slots]: parts of a tile that are there
  unsigned* done;           // [mats]: chunks of a matrix whose squares are summed
  float* squares;           // [chunks]
  float* inv_norm;          // [mats]
  unsigned* failed;         // a wait of this step ran out
  unsigned* flags;
  const float* grad_scale;
  int mats, planes;
  int per[3];               // k slabs of an item, by phase
  int total[5];             // items of the three phases, chunks, tiles of X
  float beta, decay, lr;
  int nesterov;
  int lost_warp;
  unsigned lost_step;
  Mat mat[kMaxMats];
};

__device__ __forceinline__ float load_f32(const void* p, int t, long long i) {
  if (t == EMB_T_F32) return ((const float*)p)[i];
  if (t == EMB_T_BF16) return to_f32<__nv_bfloat16>(((const __nv_bfloat16*)p)[i]);
  return to_f32<__half>(((const __half*)p)[i]);
}
__device__ __forceinline__ void store_f32(void* p, int t, long long i, float v) {
  if (t == EMB_T_F32) ((float*)p)[i] = v;
  else if (t == EMB_T_BF16) ((__nv_bfloat16*)p)[i] = from_f32<__nv_bfloat16>(v);
  else ((__half*)p)[i] = from_f32<__half>(v);
}
// The matrix that number `at` of a list belongs to.
__device__ __forceinline__ int mat_of(const MuonArgs& a, int list, int at) {
  int lo = 0, hi = a.mats - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.mat[mid].first[list] <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ float update_of(const MuonArgs& a, float g, float m) {
  return a.nesterov ? (1.0f - a.beta) * g + a.beta * m : m;
}

// ------------------------------------------------------------------ momentum and norm

__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ float part[8];
  __shared__ bool last;
  const int i = mat_of(a, 3, blockIdx.x);
  const Mat& t = a.mat[i];
  const long long n = (long long)t.rows * t.cols, at = (long long)(blockIdx.x - t.first[3]) * kChunk;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float sum = 0.0f;
#pragma unroll 4
  for (long long e = at + threadIdx.x; e < min(n, at + kChunk); e += 256) {
    const float g = load_f32(t.g, t.grad_t, e) * gs;
    const float m = a.beta * t.m[e] + (1.0f - a.beta) * g;
    t.m[e] = m;
    const float u = update_of(a, g, m);
    sum += u * u;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  const int chunks = (int)((n + kChunk - 1) / kChunk);
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int w = 0; w < 8; ++w) v += part[w];
    a.squares[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(a.done + i, 1u) + 1u == (unsigned)chunks;
  }
  __syncthreads();
  if (!last) return;
  // The matrix's last block adds the sums of all, in their order.
  __threadfence();
  __shared__ double whole[256];
  double d = 0.0;
  for (int c = threadIdx.x; c < chunks; c += 256) d += (double)__ldcg(a.squares + t.first[3] + c);
  whole[threadIdx.x] = d;
  __syncthreads();
  for (int o = 128; o; o >>= 1) {
    if (threadIdx.x < o) whole[threadIdx.x] += whole[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    // a sum that is not finite makes the whole matrix NaN
    const float norm = (float)sqrt(whole[0]) + 1e-7f;
    a.inv_norm[i] = norm <= kFltMax ? 1.0f / norm : __uint_as_float(0x7fc00000u);
  }
}

// ------------------------------------------------------------------ X

struct Pair {
  __half hi, lo;
};
__device__ __forceinline__ Pair split(float v) {
  const __half h = __float2half_rn(v);
  return {h, __float2half_rn(v - __half2float(h))};
}
// Eight neighbouring values as float16, and what that lost.
__device__ __forceinline__ void pack8(const float* v, bool two, uint4* hi, uint4* lo) {
  unsigned h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 x = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
    h[j] = *reinterpret_cast<const unsigned*>(&x);
    if (two) {
      const float2 f = __half22float2(x);
      const __half2 y = __floats2half2_rn(v[2 * j] - f.x, v[2 * j + 1] - f.y);
      l[j] = *reinterpret_cast<const unsigned*>(&y);
    }
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  if (two) *lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
  const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}
// Where piece c (eight columns) of row r lies in a tile.
__device__ __forceinline__ int piece_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// One tile of X a block: 128 rows x 64 columns, from the momentum and the gradient.
__global__ void __launch_bounds__(256) fill_kernel(const __grid_constant__ MuonArgs a) {
  const int i = mat_of(a, 4, blockIdx.x);
  const Mat& t = a.mat[i];
  const int tile = blockIdx.x - t.first[4], slabs = t.lb * 2, rb = tile / slabs, slab = tile - rb * slabs;
  const float inv = a.inv_norm[i] * kScale, gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const bool tall = t.rows > t.cols;
  unsigned char* dst = a.ws + t.x + (long long)tile * kTileBytes;
  const long long plane = (long long)t.sb * slabs * kTileBytes;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = k * 256 + threadIdx.x;
    const int r = tall ? at & 127 : at >> 3, c = tall ? at >> 7 : at & 7;  // neighbouring lanes: neighbours in memory
    const int row = rb * kTileRows + r, col = slab * kSlab + c * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (row < t.s && col + j < t.l) {
        const long long e = tall ? (long long)(col + j) * t.cols + row : (long long)row * t.cols + col + j;
        v[j] = update_of(a, load_f32(t.g, t.grad_t, e) * gs, t.m[e]) * inv;
      }
    }
    uint4 hi, lo;
    pack8(v, a.planes == 2, &hi, &lo);
    *reinterpret_cast<uint4*>(dst + piece_at(r, c)) = hi;
    if (a.planes == 2) *reinterpret_cast<uint4*>(dst + plane + piece_at(r, c)) = lo;
  }
}

// ------------------------------------------------------------------ products

// D[128 x 128] (+)= A B, 16 k's of float16.
__device__ __forceinline__ void tc_mma16(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
      : "memory");
}
__device__ __forceinline__ void bulk_load(unsigned dst, const void* src, unsigned bytes, unsigned bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
// Shared memory descriptor of an operand whose 64 contiguous elements run along its
// columns: 128-byte swizzle, blocks of 64 columns 8 KB apart, groups of eight k's 1024 bytes apart.
__device__ __forceinline__ unsigned long long column_desc(unsigned addr) {
  return (unsigned long long)((addr >> 4) & 0x3FFF) | (512ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <int PLANES>
struct MuonCfg {
  static constexpr int kStageBytes = PLANES * 2 * kTileBytes;   // 32 or 64 KB
  static constexpr int kStages = 192 * 1024 / kStageBytes;      // 6 or 3
  static constexpr int kBytes = kStages * kStageBytes + 1024;
  // Slabs that are summed in TMEM.  The tensor cores cut a sum's last bits where they add,
  // which for the squares on A's diagonal all goes one way: "split" adds the sums of four
  // slabs (48 additions) in registers, rounded to nearest (1024 x 4096: an update's error
  // 1.3e-5 with whole sums).
  static constexpr int kDrain = PLANES == 2 ? 4 : 1 << 30;
};

struct Item {
  int mat, i, j, k0, k1, part, parts, slot;
};
template <int PHASE>
__device__ __forceinline__ void item_at(const MuonArgs& a, int at, Item* it) {
  it->mat = mat_of(a, PHASE, at);
  const Mat& t = a.mat[it->mat];
  const int slabs = ((PHASE == kGram ? t.l : t.s) + kSlab - 1) / kSlab;
  it->parts = (slabs + a.per[PHASE] - 1) / a.per[PHASE];
  const int local = at - t.first[PHASE], tile = local / it->parts;
  it->part = local - tile * it->parts;
  it->slot = at - it->part;                                     // the tile's first
  // even shares: none is much shorter than the others
  it->k0 = (int)((long long)slabs * it->part / it->parts);
  it->k1 = (int)((long long)slabs * (it->part + 1) / it->parts);
  if (PHASE == kApply) {
    it->j = tile / t.sb;
    it->i = tile - it->j * t.sb;
  } else {  // the tiles on and below the diagonal, row by row
    int i = (int)((sqrtf(8.0f * tile + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > tile) --i;
    while ((i + 1) * (i + 2) / 2 <= tile) ++i;
    it->i = i;
    it->j = tile - i * (i + 1) / 2;
  }
}
__device__ __forceinline__ bool muon_give_up(volatile int* stop, const MuonArgs& a) {
  atomicOr(a.failed, 1u);
  return give_up(stop, a.flags);
}
__device__ __forceinline__ bool muon_wait(unsigned bar, unsigned parity, volatile int* stop, const MuonArgs& a) {
  if (mbar_wait(bar, parity, stop, a.flags)) return true;
  atomicOr(a.failed, 1u);
  return false;
}

// Whether `go` holds in all warps that hold sums.
__device__ __forceinline__ bool sums_go(bool go) {
  unsigned all;
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "setp.ne.b32 p, %1, 0;\n"
      "barrier.cta.red.and.pred q, 2, %2, p;\n"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((unsigned)go), "n"(kSumWarps * 32)
      : "memory");
  return all != 0;
}

// step: from 0.  X is read from buffer step & 1 and written to the other one.
template <int PHASE, int PLANES>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ MuonArgs a, int step) {
  using C = MuonCfg<PLANES>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long bars[2 * C::kStages + 4];
  __shared__ unsigned tmem_slot;
  __shared__ int stop_flag, complete;
  __shared__ unsigned issued[2];
  volatile int* stop = &stop_flag;
  const unsigned smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages, afull0 = done0 + 8 * C::kStages, aempty0 = afull0 + 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(afull0 + 8 * t, 1);
      mbar_init(aempty0 + 8 * t, kSumWarps);
    }
    stop_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(2 * kBN) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = tmem_slot;
  const int total = a.total[PHASE];
  Item it;

  if (warp == kLoadWarp) {
    unsigned n = 0;
    bool go = true;
    for (int at = blockIdx.x; go && at < total; at += gridDim.x) {
      item_at<PHASE>(a, at, &it);
      const Mat& t = a.mat[it.mat];
      const int xs = t.lb * 2, as = t.sb * 2;                           // slabs of a row of tiles of X; of A and B
      const long long xplane = (long long)t.sb * xs * kTileBytes, aplane = (long long)t.sb * as * kTileBytes;
      const unsigned char* x = a.ws + t.x + (step & 1) * PLANES * xplane;
      const unsigned char* left = PHASE == kGram ? x : a.ws + (PHASE == kSquare ? t.a : t.b);
      const unsigned char* right = PHASE == kSquare ? left : x;
      const long long lplane = PHASE == kGram ? xplane : aplane, rplane = PHASE == kSquare ? aplane : xplane;
      const int ls = PHASE == kGram ? xs : as;
      for (int k = it.k0; k < it.k1; ++k, ++n) {
        const unsigned s = n % C::kStages, ph = (n / C::kStages) & 1;
        go = __all_sync(0xffffffffu, a.lost_warp == kLoadWarp && a.lost_step == n ? muon_give_up(stop, a) : muon_wait(done0 + 8 * s, ph ^ 1, stop, a));
        if (!go) break;
        if (elect_one()) {
          const unsigned dst = smem + s * C::kStageBytes, bar = full0 + 8 * s;
          mbar_expect_tx(bar, C::kStageBytes);
#pragma unroll
          for (int q = 0; q < PLANES; ++q) {
            bulk_load(dst + q * kTileBytes, left + q * lplane + ((long long)it.i * ls + k) * kTileBytes, kTileBytes, bar);
            const unsigned to = dst + (PLANES + q) * kTileBytes;
            if (PHASE == kApply) {  // 64 rows of X by two blocks of 64 columns
              const unsigned char* from = right + q * rplane + ((long long)(k >> 1) * xs + it.j * 2) * kTileBytes + (k & 1) * (kTileBytes / 2);
              bulk_load(to, from, kTileBytes / 2, bar);
              bulk_load(to + kTileBytes / 2, from + kTileBytes, kTileBytes / 2, bar);
            } else {
              bulk_load(to, right + q * rplane + ((long long)it.j * ls + k) * kTileBytes, kTileBytes, bar);
            }
          }
        }
        __syncwarp();
      }
    }
    if (a.lost_warp == kAfterLoads) muon_give_up(stop, a);
    issued[0] = n;
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // float32 sums, float16 operands, M = N = 128; the right operand of "apply" has its columns contiguous
    constexpr unsigned idesc = (1u << 4) | ((kBN >> 3) << 17) | ((kTileRows >> 4) << 24) | (PHASE == kApply ? 1u << 16 : 0u);
    unsigned n = 0, tile = 0;
    bool go = true;
    for (int at = blockIdx.x; go && at < total; at += gridDim.x) {
      item_at<PHASE>(a, at, &it);
      for (int k = it.k0; k < it.k1; ++k, ++n) {
        const bool first = (k - it.k0) % C::kDrain == 0, last = k + 1 == it.k1 || (k + 1 - it.k0) % C::kDrain == 0;
        const unsigned t = tile & 1, tph = (tile >> 1) & 1;
        if (first) {
          go = __all_sync(0xffffffffu, muon_wait(aempty0 + 8 * t, tph ^ 1, stop, a));
          if (!go) break;
        }
        tile += last;
        const unsigned s = n % C::kStages, ph = (n / C::kStages) & 1;
        go = __all_sync(0xffffffffu, a.lost_warp == kMmaWarp && a.lost_step == n ? muon_give_up(stop, a) : muon_wait(full0 + 8 * s, ph, stop, a));
        if (!go) break;
        tc_fence_after();
        const unsigned from = smem + s * C::kStageBytes;
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < (PLANES == 2 ? 3 : 1); ++q) {  // hi hi, hi lo, lo hi
            const unsigned long long da = smem_desc(from + (q == 2 ? kTileBytes : 0));
            const unsigned bat = from + (PLANES + (q == 1 ? 1 : 0)) * kTileBytes;
            const unsigned long long db = PHASE == kApply ? column_desc(bat) : smem_desc(bat);
#pragma unroll
            for (int j = 0; j < kSlab / 16; ++j)
              tc_mma16(tmem + t * kBN, da + 2 * j, db + (PHASE == kApply ? 128 : 2) * j, idesc, !first || q > 0 || j > 0);
          }
          tc_commit(done0 + 8 * s);
          if (last) tc_commit(afull0 + 8 * t);
        }
        __syncwarp();
      }
    }
    issued[1] = n;
    __syncwarp();
  } else {
    const int half = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;  // a row a lane, 64 columns: one slab
    unsigned tile = 0;
    for (int at = blockIdx.x; at < total; at += gridDim.x) {
      item_at<PHASE>(a, at, &it);
      const Mat& t = a.mat[it.mat];
      float acc[kSlab];
      bool go = true;
      for (int k = it.k0; k < it.k1; k += min(C::kDrain, it.k1 - k), ++tile) {
        const unsigned tt = tile & 1, tph = (tile >> 1) & 1;
        go = __all_sync(0xffffffffu, muon_wait(afull0 + 8 * tt, tph, stop, a));
        if (!go) break;
        tc_fence_after();
        const unsigned taddr = tmem + ((unsigned)(quarter * 32) << 16) + tt * kBN + half * kSlab;
        unsigned v[kSlab];
        tc_load32(taddr, v);
        tc_load32(taddr + 32, v + 32);
        tc_wait32(v);
        tc_wait32(v + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(aempty0 + 8 * tt);
        const bool more = k > it.k0;
#pragma unroll
        for (int c = 0; c < kSlab; ++c) acc[c] = more ? acc[c] + __uint_as_float(v[c]) : __uint_as_float(v[c]);
      }
      // All eight warps go on or none: they meet at barriers below.
      if (!sums_go(go)) break;
      if (it.parts > 1) {
        float* part = a.partial + (long long)at * kTileRows * kBN + warp * 2048 + lane * 8;
#pragma unroll
        for (int c = 0; c < kSlab; c += 8) store32<float>(part + c * 32, acc + c);
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
        if (threadIdx.x == 0) {
          complete = atomicAdd(a.count + it.slot, 1u) + 1u == (unsigned)it.parts;
          if (complete) a.count[it.slot] = 0;                 // for the next launch
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
        const bool mine = complete;
        asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
        if (!mine) continue;
        __threadfence();
#pragma unroll
        for (int c = 0; c < kSlab; ++c) acc[c] = 0.0f;
        const float* src = a.partial + (long long)it.slot * kTileRows * kBN + warp * 2048 + lane * 8;
        for (int q = 0; q < it.parts; ++q, src += kTileRows * kBN) {
#pragma unroll
          for (int c = 0; c < kSlab; c += 4) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(src + (c / 8) * 256 + (c & 4)));
            acc[c] += w.x;
            acc[c + 1] += w.y;
            acc[c + 2] += w.z;
            acc[c + 3] += w.w;
          }
        }
      }
      const int xs = t.lb * 2, as = t.sb * 2;
      const long long xplane = (long long)t.sb * xs * kTileBytes, aplane = (long long)t.sb * as * kTileBytes;
      const long long here = ((long long)it.i * (PHASE == kApply ? xs : as) + it.j * 2 + half) * kTileBytes;
      const unsigned char* old = PHASE == kApply ? a.ws + t.x + (step & 1) * PLANES * xplane + here : a.ws + t.a + here;
      unsigned char* out = PHASE == kApply ? a.ws + t.x + (~step & 1) * PLANES * xplane + here : a.ws + (PHASE == kGram ? t.a : t.b) + here;
      const long long plane = PHASE == kApply ? xplane : aplane;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float* o = acc + 8 * c;
        if (PHASE == kGram) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= kInvScale;
        } else {
          float w[8];
          unpack8(*reinterpret_cast<const uint4*>(old + piece_at(r, c)), w);
          if (PLANES == 2) {
            float lo[8];
            unpack8(*reinterpret_cast<const uint4*>(old + plane + piece_at(r, c)), lo);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] += lo[j];
          }
          constexpr float kOld = PHASE == kSquare ? kB : kA, kNew = PHASE == kSquare ? kC * kInvScale : kInvScale;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = kOld * w[j] + kNew * o[j];
        }
      }
      if (PHASE == kApply && step == kSteps - 1) {
        const int row = it.i * kTileRows + r, col0 = it.j * kBN + half * kSlab;
        const bool tall = t.rows > t.cols;
        const float rate = a.lr * t.scale * kInvScale;
        if (row < t.s && *(volatile unsigned*)a.failed == 0) {
#pragma unroll
          for (int c = 0; c < kSlab; ++c) {
            if (col0 + c < t.l) {
              const long long e = tall ? (long long)(col0 + c) * t.cols + row : (long long)row * t.cols + col0 + c;
              store_f32(t.p, t.param_t, e, load_f32(t.p, t.param_t, e) * a.decay - rate * acc[c]);
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 hi, lo;
          pack8(acc + 8 * c, PLANES == 2, &hi, &lo);
          *reinterpret_cast<uint4*>(out + piece_at(r, c)) = hi;
          if (PLANES == 2) *reinterpret_cast<uint4*>(out + plane + piece_at(r, c)) = lo;
        }
        if (PHASE != kApply && it.i != it.j) {  // the same values above the diagonal
          const int col = (quarter & 1) * 32 + lane;
          unsigned char* up = a.ws + (PHASE == kGram ? t.a : t.b) + ((long long)it.j * as + it.i * 2 + (quarter >> 1)) * kTileBytes + (col & 7) * 2;
#pragma unroll
          for (int c = 0; c < kSlab; ++c) {
            const Pair w = split(acc[c]);
            *reinterpret_cast<__half*>(up + piece_at(half * kSlab + c, col >> 3)) = w.hi;
            if (PLANES == 2) *reinterpret_cast<__half*>(up + plane + piece_at(half * kSlab + c, col >> 3)) = w.lo;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*stop) {  // a wait ran out: what is in flight lands before the block ends
    const unsigned n = warp >= kSumWarps ? issued[warp - kSumWarps] : 0;
    if (warp == kLoadWarp)
      for (unsigned j = n - min(n, (unsigned)C::kStages); j < n; ++j) mbar_drain(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
    if (warp == kMmaWarp && n > 0) mbar_drain(done0 + 8 * ((n - 1) % C::kStages), ((n - 1) / C::kStages) & 1);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kBN));
  }
}

// ------------------------------------------------------------------ host side

struct MuonPlan {
  size_t bytes = 0;
  size_t partial = 0, count = 0, done = 0, squares = 0, inv_norm = 0, failed = 0;  // offsets
  size_t zero_from = 0, zero_bytes = 0;
};

// Lays out one launch group; false where a list's numbers pass 31 bits.
bool plan_group(const emb_muon_tensor* t, int n, int planes, MuonArgs* a, MuonPlan* pl) {
  long long tiles = 0, chunks = 0, xtiles = 0, steps[3] = {}, ntiles[3] = {};
  a->mats = 0;
  a->planes = planes;
  for (int i = 0; i < n; ++i) {
    if (t[i].rows == 0 || t[i].cols == 0) continue;
    Mat& m = a->mat[a->mats++];
    m.p = t[i].param_d;
    m.m = t[i].m_d;
    m.rows = (int)t[i].rows;
    m.cols = (int)t[i].cols;
    m.s = std::min(m.rows, m.cols);
    m.l = std::max(m.rows, m.cols);
    m.sb = (m.s + 127) / 128;
    m.lb = (m.l + 127) / 128;
    m.param_t = t[i].param_t;
    m.grad_t = t[i].grad_t;
    m.scale = t[i].scale;
    const long long x = 2LL * m.sb * m.lb, q = 2LL * m.sb * m.sb;
    m.x = tiles * kTileBytes;
    m.a = (tiles + 2 * planes * x) * kTileBytes;
    m.b = m.a + planes * q * kTileBytes;
    tiles += planes * (2 * x + 2 * q);
    m.first[3] = (int)chunks;
    m.first[4] = (int)xtiles;
    chunks += ((long long)m.rows * m.cols + kChunk - 1) / kChunk;
    xtiles += x;
    const long long tri = (long long)m.sb * (m.sb + 1) / 2, full = (long long)m.sb * m.lb;
    const int sl = (m.l + kSlab - 1) / kSlab, ss = (m.s + kSlab - 1) / kSlab;
    ntiles[kGram] += tri;
    ntiles[kSquare] += tri;
    ntiles[kApply] += full;
    steps[kGram] += tri * sl;
    steps[kSquare] += tri * ss;
    steps[kApply] += full * ss;
    if (chunks > 0x7fffffffLL || xtiles > 0x7fffffffLL || ntiles[kApply] > 0x3fffffffLL) return false;
  }
  const int sms = sm_count();
  long long slots = 0;
  a->total[3] = (int)chunks;
  a->total[4] = (int)xtiles;
  for (int ph = 0; ph < 3; ++ph) {
    // Where there are fewer tiles than SMs a tile's k's are shared out, four slabs a part at least.
    a->per[ph] = ntiles[ph] >= sms ? kWhole : (int)std::max<long long>(4, (steps[ph] + sms - 1) / sms);
    long long items = 0;
    for (int i = 0; i < a->mats; ++i) {
      Mat& m = a->mat[i];
      const long long k = ((ph == kGram ? m.l : m.s) + kSlab - 1) / kSlab, parts = a->per[ph] == kWhole ? 1 : (k + a->per[ph] - 1) / a->per[ph];
      m.first[ph] = (int)items;
      items += parts * (ph == kApply ? (long long)m.sb * m.lb : (long long)m.sb * (m.sb + 1) / 2);
    }
    a->total[ph] = (int)items;
    if (a->per[ph] != kWhole) slots = std::max(slots, items);
  }
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl->partial = (size_t)tiles * kTileBytes;
  pl->count = pl->partial + (size_t)slots * kTileRows * kBN * 4;
  pl->done = pl->count + up((size_t)slots * 4);
  pl->failed = pl->done + up((size_t)kMaxMats * 4);
  pl->inv_norm = pl->failed + 256;
  pl->squares = pl->inv_norm + up((size_t)kMaxMats * 4);
  pl->bytes = pl->squares + up((size_t)chunks * 4);
  pl->zero_from = pl->count;
  pl->zero_bytes = pl->inv_norm - pl->count;
  return true;
}

template <int PHASE, int PLANES>
cudaError_t launch_product(const MuonArgs& a, int step, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(product_kernel<PHASE, PLANES>, cudaFuncAttributeMaxDynamicSharedMemorySize, MuonCfg<PLANES>::kBytes);
  if (e != cudaSuccess) return e;
  product_kernel<PHASE, PLANES><<<std::min(a.total[PHASE], sm_count()), kThreads, MuonCfg<PLANES>::kBytes, st>>>(a, step);
  return cudaGetLastError();
}

template <int PLANES>
cudaError_t launch_steps(const MuonArgs& a, cudaStream_t st) {
  for (int step = 0; step < kSteps; ++step) {
    cudaError_t e = launch_product<kGram, PLANES>(a, step, st);
    if (e == cudaSuccess) e = launch_product<kSquare, PLANES>(a, step, st);
    if (e == cudaSuccess) e = launch_product<kApply, PLANES>(a, step, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

emb_status check_tensors(const emb_muon_tensor* t, int32_t n, emb_muon_products products) {
  if (n < 0 || (n > 0 && !t)) return fail(EMB_ERR_INVALID_ARG, "tensors is NULL or their number negative");
  if (products != EMB_MUON_HALF && products != EMB_MUON_SPLIT) return fail(EMB_ERR_INVALID_ARG, "bad products");
  for (int i = 0; i < n; ++i) {
    if (t[i].rows < 0 || t[i].cols < 0) return fail(EMB_ERR_INVALID_ARG, "negative rows or cols");
    if (t[i].rows > EMB_MUON_MAX_DIM || t[i].cols > EMB_MUON_MAX_DIM) return fail(EMB_ERR_UNSUPPORTED, "a side above EMB_MUON_MAX_DIM");
    if (!good_ftype(t[i].param_t) || !good_ftype(t[i].grad_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
    if (!std::isfinite(t[i].scale)) return fail(EMB_ERR_INVALID_ARG, "scale must be finite");
  }
  return EMB_OK;
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_muon_workspace_size(const emb_muon_tensor* tensors, int32_t n_tensors, emb_muon_products products,
                                              size_t* bytes) {
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  const emb_status rc = check_tensors(tensors, n_tensors, products);
  if (rc != EMB_OK) return rc;
  size_t most = 0;
  for (int at = 0; at < n_tensors; at += kMaxMats) {
    MuonArgs a;
    MuonPlan pl;
    if (!plan_group(tensors + at, std::min(kMaxMats, n_tensors - at), products == EMB_MUON_SPLIT ? 2 : 1, &a, &pl))
      return fail(EMB_ERR_UNSUPPORTED, "matrices too large for one call");
    if (a.mats) most = std::max(most, pl.bytes);
  }
  *bytes = most;
  return EMB_OK;
}

extern "C" emb_status emb_muon_step(const emb_muon_tensor* tensors, const void* const* grads, int32_t n_tensors,
                                    const emb_muon_params* params, void* workspace_d, size_t ws_bytes, void* stream) {
  if (!params) return fail(EMB_ERR_INVALID_ARG, "params is NULL");
  const emb_muon_params& o = *params;
  if (!(o.lr >= 0.0 && o.lr <= 1e30) || !(o.weight_decay >= 0.0 && o.weight_decay <= 1e30) || !(o.momentum >= 0.0 && o.momentum < 1.0))
    return fail(EMB_ERR_INVALID_ARG, "lr and weight_decay must be >= 0, 0 <= momentum < 1");
  size_t need = 0;
  emb_status rc = emb_muon_workspace_size(tensors, n_tensors, o.products, &need);
  if (rc != EMB_OK) return rc;
  if (need == 0) return EMB_OK;
  if (!grads) return fail(EMB_ERR_INVALID_ARG, "grads is NULL");
  for (int i = 0; i < n_tensors; ++i) {
    const emb_muon_tensor& t = tensors[i];
    if (t.rows == 0 || t.cols == 0) continue;
    if (!t.param_d || !t.m_d || !grads[i]) return fail(EMB_ERR_INVALID_ARG, "a parameter, momentum or gradient is NULL");
    if (!aligned_to(t.param_d, ftype_bytes(t.param_t)) || !aligned_to(t.m_d, 4) || !aligned_to(grads[i], ftype_bytes(t.grad_t)))
      return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  }
  if (!aligned_to(o.grad_scale_d, 4)) return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (!workspace_d || ws_bytes < need) return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_muon_workspace_size()");
  if (!aligned_to(workspace_d, 256)) return fail(EMB_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  cudaStream_t st = (cudaStream_t)stream;
  int lost;
  unsigned lost_step, *flags = nullptr;
  lost_wait(&lost, &lost_step);
  EMB_CUDA(op_flags(&flags));
  const int lost_warps[4] = {kLoadWarp, kMmaWarp, -1, kAfterLoads};
  for (int at = 0; at < n_tensors; at += kMaxMats) {
    MuonArgs a;
    MuonPlan pl;
    const int n = std::min(kMaxMats, n_tensors - at);
    plan_group(tensors + at, n, o.products == EMB_MUON_SPLIT ? 2 : 1, &a, &pl);
    if (a.mats == 0) continue;
    for (int i = 0, j = 0; i < n; ++i)
      if (tensors[at + i].rows && tensors[at + i].cols) a.mat[j++].g = grads[at + i];
    unsigned char* ws = (unsigned char*)workspace_d;
    a.ws = ws;
    a.partial = (float*)(ws + pl.partial);
    a.count = (unsigned*)(ws + pl.count);
    a.done = (unsigned*)(ws + pl.done);
    a.failed = (unsigned*)(ws + pl.failed);
    a.inv_norm = (float*)(ws + pl.inv_norm);
    a.squares = (float*)(ws + pl.squares);
    a.flags = flags;
    a.grad_scale = o.grad_scale_d;
    a.beta = (float)o.momentum;
    a.decay = (float)(1.0 - o.lr * o.weight_decay);
    a.lr = (float)o.lr;
    a.nesterov = o.nesterov != 0;
    a.lost_warp = lost < 0 ? -1 : lost_warps[lost];
    a.lost_step = lost_step;
    EMB_CUDA(cudaMemsetAsync(ws + pl.zero_from, 0, pl.zero_bytes, st));
    momentum_kernel<<<a.total[3], 256, 0, st>>>(a);
    EMB_CUDA(cudaGetLastError());
    fill_kernel<<<a.total[4], 256, 0, st>>>(a);
    EMB_CUDA(cudaGetLastError());
    const cudaError_t e = a.planes == 2 ? launch_steps<2>(a, st) : launch_steps<1>(a, st);
    if (e != cudaSuccess) return cuda_fail(e, "emb_muon_step launch");
  }
  return EMB_OK;
}
