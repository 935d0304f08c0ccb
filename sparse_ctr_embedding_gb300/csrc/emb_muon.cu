// Muon: momentum, orthogonalised by Newton-Schulz steps, as the update of matrices.
//   m = beta m + (1 - beta) g;  u = (1 - beta) g + beta m (Nesterov) or m;  X = u / (|u| + 1e-7)
//   five times:  A = X X^T;  B = b A + c A^2;  X = a X + B X        (X with its short side first)
//   p = p (1 - lr wd) - lr scale X
//
// Launches, each over all matrices of a call: the momentum with the sum of u's
// squares; X; then all products in one, three phases a step, "gram" (A), "square" (B) and
// "apply" (X), the last of which writes the weights.  Everything between lies in the workspace.
//
// Products.  Operands are float16 with float32 sums on tcgen05.  X, A and B are kept
// times 2^12: singular values stay below about 1.25, so entries stay below 2^14, and
// entries down to 2^-26 keep their 11 bits.  "half" keeps one float16 of each: 2^-11
// a rounding, an eighth of what bfloat16 loses in the same step at the same rate.  "split"
// keeps two, the second what the first one lost (22 bits together), and takes three
// products of the four: about float32's accuracy at a third of the rate (an update's error 2e-6 to
// 7e-6, where float32 products have 2e-6 to 5e-6: 256 x 512 to 4096 x 4096, 1024 x 8192 among them).
//
// Layout.  A matrix lies in the workspace as the tensor cores read it from shared
// memory: tiles of 128 rows x 64 columns, a row 128 bytes, its 16-byte pieces swizzled,
// zeros past the edges.  A tile is 16 KB in one piece, so one tensor map of plain rows of 128
// bytes serves all matrices, whatever their shapes.  The same tiles serve X^T: for X
// on the right of B its 64 x 64 halves are read as the operand whose columns are
// contiguous.  A and A^2 are symmetric: only tiles on and below the diagonal are
// computed, and written twice.
//
// Work is cut into items, a tile of 256 x 256 for a pair of SMs or a part of its k's where there
// are fewer tiles than pairs; a part's float32 sums go to the workspace, and its block then adds
// all parts' sums, in k order, for its share of the tile.
//
// Bound by the tensor cores where matrices are large (4096 x 4096 and four smaller ones, 2.0 TFLOP: 1390 us, 0.74 of
// the rate of a large library product), else by the way from one phase to the next: three
// matrices up to 256 x 512 take 157 us, ten a phase.  "split", 1024 x 8192 and three smaller: 647; it spills 876 bytes
// a thread ("half" 72), the sums' warps with 224 registers.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "emb_tiles.cuh"

namespace emb {
namespace {

constexpr int kMaxMats = 128;       // matrices of one launch: bounded by the kernel's parameters
constexpr int kTileRows = 128, kSlab = 64;
constexpr int kTileBytes = kTileRows * kSlab * 2;   // 16 KB
constexpr int kBN = 256;            // rows and columns of a pair's tile
constexpr int kCols = 128;          // columns of a warp that holds sums
constexpr int kChunk = 8192;        // elements of a block in the momentum kernel
constexpr int kSteps = 5;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 4096.0f, kInvScale = 1.0f / 4096.0f;
constexpr int kThreads = (kSumWarps + 4) * 32, kLoadWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
// Registers: the sums need more than an even share, the other four warps (two of them idle) little.
constexpr int kLaunchRegs = 168, kSumRegs = 224, kOtherRegs = 56;
static_assert(kSumWarps * 32 * kSumRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kAfterLoads = 0;

enum Phase { kGram = 0, kSquare = 1, kApply = 2 };

struct Mat {
  void* p;
  float* m;
  const void* g;
  long long x, a, b;        // tiles in the workspace: X (two buffers of x_tiles), A, B
  int rows, cols;           // of the parameter
  int s, l;                 // short and long side
  int sb, lb;               // tiles of 256 along each
  int parts[3];             // of a tile, by phase
  int first[5];             // of this matrix among all: items of the three phases, chunks, tiles of X
  int param_t, grad_t;
  int wide;                 // rows of the parameter are aligned to four elements
  int vec;                  // momentum and gradient are aligned to eight
  float scale;
};

struct MuonArgs {
  unsigned char* ws;        // tiles
  float* partial;           // [slots][2][128 * kBN]: a slot an item, a half a block of its pair
  unsigned* count;          // [slots][2]: parts of a tile that are there, over all steps; at its first slot
  unsigned* ready;          // [mats]: shares of tiles that are complete, over all steps
  unsigned* done;           // [mats]: chunks of a matrix whose squares are summed
  float* squares;           // [chunks]
  float* inv_norm;          // [mats]
  unsigned* failed;         // a wait of this step ran out
  unsigned* flags;
  const float* grad_scale;
  int mats, planes;
  int slot0[3], slots;      // first slot, by phase; slots of items, after which the blocks' own lie
  int total[5];             // items of the three phases, chunks, tiles of X
  float beta, omb, decay, lr;   // omb: 1 - beta, rounded once (from the rounded beta it is 1.3e-5 of itself off at 0.999)
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
__device__ __forceinline__ void load8_f32(const void* p, int t, long long i, float* o) {
  auto from = [&](auto* q) {
    Raw8<std::remove_const_t<std::remove_pointer_t<decltype(q)>>> r;
    r.load(q + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = r.get(j);
  };
  if (t == EMB_T_F32) from((const float*)p);
  else if (t == EMB_T_BF16) from((const __nv_bfloat16*)p);
  else from((const __half*)p);
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
  return a.nesterov ? a.omb * g + a.beta * m : m;
}

// ------------------------------------------------------------------ momentum and norm

// This block's elements [at, end): the momentum, and the sum of its updates' squares over this thread's.
template <typename G>
__device__ __forceinline__ float momentum_of(const MuonArgs& a, const Mat& t, long long at, long long end, float gs) {
  float sum = 0.0f;
  const G* g = (const G*)t.g;
  if (t.vec) {
    long long e = at + threadIdx.x * 8LL;
    constexpr int kBatch = 2;
    for (; e + (kBatch - 1) * 2048 + 8 <= end; e += kBatch * 2048) {  // all loads before any store
      Raw8<G> gr[kBatch];
      Raw8<float> m[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        gr[q].load(g + e + q * 2048);
        m[q].load(t.m + e + q * 2048);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = gr[q].get(j) * gs;
          m[q].v[j] = a.beta * m[q].v[j] + a.omb * x;
          const float u = update_of(a, x, m[q].v[j]);
          sum += u * u;
        }
        m[q].store(t.m + e + q * 2048);
      }
    }
    for (; e < end; e += 2048) {
      for (long long i = e; i < min(end, e + 8); ++i) {
        const float x = to_f32<G>(g[i]) * gs, m = a.beta * t.m[i] + a.omb * x, u = update_of(a, x, m);
        t.m[i] = m;
        sum += u * u;
      }
    }
    return sum;
  }
#pragma unroll 4
  for (long long i = at + threadIdx.x; i < end; i += 256) {
    const float x = to_f32<G>(g[i]) * gs, m = a.beta * t.m[i] + a.omb * x, u = update_of(a, x, m);
    t.m[i] = m;
    sum += u * u;
  }
  return sum;
}

// Bound by memory: gradient and momentum in, momentum out (52.6M elements: 65 us, 100 with an element an access).
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ float part[8];
  __shared__ bool last;
  const int i = mat_of(a, 3, blockIdx.x);
  const Mat& t = a.mat[i];
  const long long n = (long long)t.rows * t.cols, at = (long long)(blockIdx.x - t.first[3]) * kChunk, end = min(n, at + kChunk);
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float sum = t.grad_t == EMB_T_F32    ? momentum_of<float>(a, t, at, end, gs)
              : t.grad_t == EMB_T_BF16 ? momentum_of<__nv_bfloat16>(a, t, at, end, gs)
                                       : momentum_of<__half>(a, t, at, end, gs);
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

// One tile of X a block: 128 rows x 64 columns, from the momentum and the gradient (52.6M elements: 75 us, eight
// an access; 84 by single ones).
__global__ void __launch_bounds__(256) fill_kernel(const __grid_constant__ MuonArgs a) {
  const int i = mat_of(a, 4, blockIdx.x);
  const Mat& t = a.mat[i];
  const int tile = blockIdx.x - t.first[4], slabs = t.lb * 4, rb = tile / slabs, slab = tile - rb * slabs;
  const float inv = a.inv_norm[i] * kScale, gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const bool tall = t.rows > t.cols;
  unsigned char* dst = a.ws + t.x + (long long)tile * kTileBytes;
  const long long plane = 2LL * t.sb * slabs * kTileBytes;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = k * 256 + threadIdx.x;
    const int r = tall ? at & 127 : at >> 3, c = tall ? at >> 7 : at & 7;  // neighbouring lanes: neighbours in memory
    const int row = rb * kTileRows + r, col = slab * kSlab + c * 8;
    float v[8];
    if (t.vec && !tall && t.cols % 8 == 0 && row < t.s && col < t.l) {  // eight elements an access
      const long long e = (long long)row * t.cols + col;
      float g[8];
      load8_f32(t.g, t.grad_t, e, g);
      Raw8<float> m;
      m.load(t.m + e);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = update_of(a, g[j] * gs, m.v[j]) * inv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (row < t.s && col + j < t.l) {
          const long long e = tall ? (long long)(col + j) * t.cols + row : (long long)row * t.cols + col + j;
          v[j] = update_of(a, load_f32(t.g, t.grad_t, e) * gs, t.m[e]) * inv;
        }
      }
    }
    uint4 hi, lo;
    pack8(v, a.planes == 2, &hi, &lo);
    *reinterpret_cast<uint4*>(dst + piece_at(r, c)) = hi;
    if (a.planes == 2) *reinterpret_cast<uint4*>(dst + plane + piece_at(r, c)) = lo;
  }
}

// ------------------------------------------------------------------ products

// Two neighbouring SMs (a cluster of two blocks) work on a tile of 256 x 256 together: each
// holds its 128 rows of the left operand, half of the right one, and the sums of its rows.
// A pair's MMAs are issued by its first block ("leader").

// D[256 x 256] (+)= A B, 16 k's of float16.
__device__ __forceinline__ void tc_mma16(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add)
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
  static constexpr int kBytes = kStages * kStageBytes + kSumWarps * 4096 + 1024;  // + a unit a warp, room to align
  static_assert(kBytes <= 232448, "shared memory");
  // Slabs that are summed in TMEM.  The tensor cores cut a sum's last bits where they add,
  // which for the squares on A's diagonal all goes one way: "split" adds the sums of four
  // slabs (48 additions) in registers, rounded to nearest (1024 x 4096: an update's error
  // 1.3e-5 with whole sums).
  static constexpr int kDrain = PLANES == 2 ? 4 : 1 << 30;
};

struct Item {
  int mat, phase, step, i, j, k0, k1, part, parts, at;
};
// Item number `seq` of all steps' phases, one after the other.
__device__ __forceinline__ void item_at(const MuonArgs& a, int seq, Item* it) {
  const int whole = a.total[0] + a.total[1] + a.total[2];
  it->step = seq / whole;
  int at = seq - it->step * whole;
  it->phase = at < a.total[0] ? kGram : at < a.total[0] + a.total[1] ? kSquare : kApply;
  if (it->phase >= kSquare) at -= a.total[0];
  if (it->phase == kApply) at -= a.total[1];
  it->mat = mat_of(a, it->phase, at);
  const Mat& t = a.mat[it->mat];
  const int slabs = ((it->phase == kGram ? t.l : t.s) + kSlab - 1) / kSlab;
  it->parts = t.parts[it->phase];
  const int local = at - t.first[it->phase], tile = local / it->parts, part = local - tile * it->parts;
  it->part = part;
  it->at = a.slot0[it->phase] + at;
  // even shares: none is much shorter than the others
  it->k0 = (int)((long long)slabs * part / it->parts);
  it->k1 = (int)((long long)slabs * (part + 1) / it->parts);
  if (it->phase == kApply) {
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
// Shares of this matrix's tiles (one for each block of an item's pair) that are complete before an
// item of this step and phase may begin.
__device__ __forceinline__ unsigned tiles_before(const Mat& t, const Item& it) {
  const int tri = t.sb * (t.sb + 1) / 2, n0 = tri * t.parts[0], n1 = tri * t.parts[1], n2 = t.sb * t.lb * t.parts[2];
  return 2u * (unsigned)(it.step * (n0 + n1 + n2) + (it.phase > 0 ? n0 : 0) + (it.phase > 1 ? n1 : 0));
}

// What a wait that ran out does: the pair's other waits end, the weights stay, the host is told.
__device__ __forceinline__ bool muon_give_up(unsigned stop, const MuonArgs& a) {
  atomicOr(a.failed, 1u);
  return pair_give_up(stop, a.flags);
}
// A phase of a large matrix takes a second: the limit on polls is longer than the other products'.
constexpr unsigned kMuonLimit = 1u << 27;
__device__ __forceinline__ bool muon_wait(unsigned bar, unsigned parity, unsigned stop, const MuonArgs& a) {
  if (pair_try(bar, parity)) return true;
  for (unsigned i = 0; i < kMuonLimit; ++i) {
    if (pair_try(bar, parity)) return true;
    if (pair_stopped(stop)) return false;
  }
  return muon_give_up(stop, a);
}
// Waits until the tiles that an item reads are complete.
__device__ __forceinline__ bool tiles_wait(const unsigned* count, unsigned need, unsigned stop, const MuonArgs& a) {
  for (unsigned i = 0; i < (1u << 22); ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    if (v >= need) return true;
    if ((i & 15) == 15 && (pair_stopped(stop) || *(volatile unsigned*)a.failed)) return muon_give_up(stop, a);
  }
  return muon_give_up(stop, a);
}
__device__ __forceinline__ void tma_load2(unsigned dst, const CUtensorMap* map, long long at, unsigned bar) {
  tma_load_pair(dst, map, 0, (int)(at >> 7), bar);
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
__device__ __forceinline__ void sums_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory"); }

// p = p decay - rate x for a unit: this lane's row `row` of X, 32 columns from `col` on.  Where the
// parameter's rows are X's, a row of it is made of eight lanes' accesses, through
// shared memory; else a lane's neighbours are the others' and each column is one access.
template <typename T>
__device__ __forceinline__ void update_unit(T* p, const Mat& t, int row, int col, bool tall, float decay, float rate, const float* x,
                                            unsigned char* stage) {
  const int lane = threadIdx.x & 31;
  if (tall) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      T v[16];
      T* q = p + (long long)(col + h) * t.cols + row;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (row < t.s && col + h + j < t.l) v[j] = q[(long long)j * t.cols];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (row < t.s && col + h + j < t.l) q[(long long)j * t.cols] = from_f32<T>(to_f32<T>(v[j]) * decay - rate * x[h + j]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
  __syncwarp();
  const int r0 = row - lane, c4 = col + (lane & 7) * 4;
#pragma unroll
  for (int h = 0; h < 8; h += 4) {
    __align__(16) T v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = r0 + (h + i) * 4 + (lane >> 3);
      const T* q = p + (long long)rr * t.cols + c4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (rr < t.s && c4 + j < t.l && !t.wide) v[i][j] = q[j];
      if (t.wide && rr < t.s && c4 < t.l) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(v[i]) = *reinterpret_cast<const uint4*>(q);
        else *reinterpret_cast<uint2*>(v[i]) = *reinterpret_cast<const uint2*>(q);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = (h + i) * 4 + (lane >> 3), rr = r0 + lr;
      const float4 y = *reinterpret_cast<const float4*>(stage + lr * 128 + (((lane & 7) ^ (lr & 7)) << 4));
      const float z[4] = {y.x, y.y, y.z, y.w};
      T* q = p + (long long)rr * t.cols + c4;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = from_f32<T>(to_f32<T>(v[i][j]) * decay - rate * z[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (rr < t.s && c4 + j < t.l && !t.wide) q[j] = v[i][j];
      if (t.wide && rr < t.s && c4 < t.l) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(v[i]);
        else *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(v[i]);
      }
    }
  }
}

// All five steps.  An item begins when the tiles that it reads are complete (a.ready: tiles
// of a matrix that are, over all steps); its pair then loads, multiplies and writes like any
// other product, so small matrices go on while large ones are at work.  Items are dealt
// in order and all blocks are resident (a cooperative launch), so what an item waits for
// is at work or done.  X of step t lies in buffer t & 1.
template <int PLANES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ MuonArgs a) {
  using C = MuonCfg<PLANES>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long bars[2 * C::kStages + 4];
  __shared__ unsigned tmem_slot, stop_flag;
  __shared__ unsigned issued[2];
  const unsigned smem = (smem_u32(raw) + 1023u) & ~1023u, stop = smem_u32(&stop_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rank = blockIdx.x & 1;                        // in the pair; 0 leads
  const unsigned full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages, afull0 = done0 + 8 * C::kStages, aempty0 = afull0 + 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(done0 + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(afull0 + 8 * t, 1);
      mbar_init(aempty0 + 8 * t, 2 * kSumWarps);               // of both blocks
    }
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
  const unsigned tmem = tmem_slot;
  const int total = kSteps * (a.total[0] + a.total[1] + a.total[2]), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  Item it;

  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      unsigned n = 0;
      bool go = true;
      for (int at = pair; go && at < total; at += pairs) {
        item_at(a, at, &it);
        const Mat& t = a.mat[it.mat];
        const long long xs = t.lb * 4, as = t.sb * 4;                     // slabs of a row of tiles of X; of A and B
        const long long xplane = t.sb * 2 * xs * kTileBytes, aplane = t.sb * 2 * as * kTileBytes;
        const bool apply = it.phase == kApply, gram = it.phase == kGram;
        const long long x = t.x + (it.step & 1) * PLANES * xplane;
        const long long left = gram ? x : apply ? t.b : t.a, right = it.phase == kSquare ? t.a : x;
        const long long lplane = gram ? xplane : aplane, rplane = it.phase == kSquare ? aplane : xplane, ls = gram ? xs : as;
        go = __all_sync(0xffffffffu, tiles_wait(a.ready + it.mat, tiles_before(t, it), stop, a));
        if (!go) break;
        asm volatile("fence.proxy.async;" ::: "memory");                  // plain stores of other blocks, read by TMA
        for (int k = it.k0; k < it.k1; ++k, ++n) {
          const unsigned s = n % C::kStages, ph = (n / C::kStages) & 1;
          go = __all_sync(0xffffffffu, a.lost_warp == kLoadWarp && a.lost_step == n ? muon_give_up(stop, a) : muon_wait(done0 + 8 * s, ph ^ 1, stop, a));
          if (!go) break;
          if (elect_one()) {
            const unsigned dst = smem + s * C::kStageBytes, bar = peer_addr(full0 + 8 * s, 0);
            if (rank == 0) mbar_expect_tx(full0 + 8 * s, 2 * C::kStageBytes);
#pragma unroll
            for (int q = 0; q < PLANES; ++q) {
              tma_load2(dst + q * kTileBytes, &map, left + q * lplane + ((it.i * 2 + rank) * ls + k) * kTileBytes, bar);
              tma_load2(dst + q * kTileBytes + kTileBytes / 2, &map, left + q * lplane + ((it.i * 2 + rank) * ls + k) * kTileBytes + kTileBytes / 2, bar);
              const unsigned to = dst + (PLANES + q) * kTileBytes;
              // the half of the right operand: 128 rows of its tile, or 64 rows of X by two blocks of 64 columns
              const long long from = right + q * rplane + (apply ? ((k >> 1) * xs + it.j * 4 + rank * 2) * kTileBytes + (k & 1) * (kTileBytes / 2)
                                                                 : ((it.j * 2 + rank) * ls + k) * kTileBytes);
              tma_load2(to, &map, from, bar);
              tma_load2(to + kTileBytes / 2, &map, from + (apply ? kTileBytes : kTileBytes / 2), bar);
            }
          }
          __syncwarp();
        }
      }
      if (a.lost_warp == kAfterLoads) muon_give_up(stop, a);
      issued[0] = n;
    } else if (warp == kMmaWarp && rank == 0) {
      // float32 sums, float16 operands, M = N = 256
      constexpr unsigned idesc0 = (1u << 4) | ((256 >> 3) << 17) | ((256 >> 4) << 24);
      // One thread for all: with the warp meeting at every slab, a slab took 50 to 100 cycles more.
      unsigned n = 0, tile = 0;
      if (elect_one()) {
        bool go = true;
        unsigned s = 0, ph = 0;
        for (int at = pair; go && at < total; at += pairs) {
          item_at(a, at, &it);
          const bool apply = it.phase == kApply;                          // its right operand has its columns contiguous
          const unsigned idesc = idesc0 | (apply ? 1u << 16 : 0u), badvance = apply ? 128 : 2;
          for (int k = it.k0; k < it.k1; ++k, ++n) {
            const bool first = (k - it.k0) % C::kDrain == 0, last = k + 1 == it.k1 || (k + 1 - it.k0) % C::kDrain == 0;
            const unsigned t = tile & 1, tph = (tile >> 1) & 1;
            if (first) {
              go = muon_wait(aempty0 + 8 * t, tph ^ 1, stop, a);
              if (!go) break;
            }
            tile += last;
            go = a.lost_warp == kMmaWarp && a.lost_step == n ? muon_give_up(stop, a) : muon_wait(full0 + 8 * s, ph, stop, a);
            if (!go) break;
            tc_fence_after();
            const unsigned from = smem + s * C::kStageBytes;
#pragma unroll
            for (int q = 0; q < (PLANES == 2 ? 3 : 1); ++q) {  // hi hi, hi lo, lo hi
              const unsigned long long da = smem_desc(from + (q == 2 ? kTileBytes : 0));
              const unsigned bat = from + (PLANES + (q == 1 ? 1 : 0)) * kTileBytes;
              const unsigned long long db = apply ? column_desc(bat) : smem_desc(bat);
#pragma unroll
              for (int j = 0; j < kSlab / 16; ++j) tc_mma16(tmem + t * kBN, da + 2 * j, db + badvance * j, idesc, !first || q > 0 || j > 0);
            }
            commit_both(done0 + 8 * s);
            if (last) commit_both(afull0 + 8 * t);
            if (++s == C::kStages) s = 0, ph ^= 1;
          }
        }
      }
      __syncwarp();
      n = __reduce_max_sync(0xffffffffu, n);
      issued[1] = n;
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int half = warp >> 2, quarter = warp & 3;            // TMEM: a row a lane, 128 columns a warp
    constexpr int kPiece = 32, kPieces = kCols / kPiece;
    unsigned char* const stage = raw + (smem - smem_u32(raw)) + C::kStages * C::kStageBytes + warp * 4096;
    unsigned tile = 0;
    auto release = [&](unsigned which) {                       // an accumulator that has been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive(aempty0 + 8 * which, 0);
    };
    for (int at = pair; at < total; at += pairs) {
      item_at(a, at, &it);
      const Mat& t = a.mat[it.mat];
      const long long tile_floats = kTileRows * kBN;
      // Where this thread's 128 sums go if they leave: an item's slot, or ("split") the block's own.
      float* const part = a.partial + ((long long)(it.parts > 1 ? it.at : a.slots + pair) * 2 + rank) * tile_floats + warp * 4096 + lane * 8;
      const bool apply = it.phase == kApply, gram = it.phase == kGram, finish = apply && it.step == kSteps - 1;
      const long long xs = t.lb * 4, as = t.sb * 4;
      const long long xplane = t.sb * 2 * xs * kTileBytes, aplane = t.sb * 2 * as * kTileBytes, plane = apply ? xplane : aplane;
      const int rb = it.i * 2 + rank;                          // this block's rows: a block of 128
      const int row_end = (t.s + 63) & ~63, col_end = ((apply ? t.l : t.s) + 63) & ~63;
      const long long here0 = (rb * (apply ? xs : as) + it.j * 4) * kTileBytes;
      const unsigned char* old0 = a.ws + (apply ? t.x + (it.step & 1) * PLANES * xplane : t.a) + here0;
      unsigned char* out0 = a.ws + (apply ? t.x + (~it.step & 1) * PLANES * xplane : gram ? t.a : t.b) + here0;
      // Unit w * 4 + b is the piece of 32 rows x 32 columns that warp w has b-th.  In memory its rows are
      // 64 of a line's 128 bytes; a lane reads and writes 16 of those, four lanes a row, and
      // the rows meet their owners' registers in shared memory (a row a lane: 32 lines an access).
      auto unit_row = [](int u) { return (u >> 2 & 3) * 32; };
      auto unit_col = [](int u) { return (u >> 4) * 128 + (u & 3) * 32; };
      auto unit_in = [&](int u) { return rb * kTileRows + unit_row(u) < row_end && it.j * kBN + unit_col(u) < col_end; };
      auto line_at = [&](int u, int i) {                       // this lane's i-th access
        const int rr = unit_row(u) + i * 8 + (lane >> 2), cc = unit_col(u);
        return (long long)(cc >> 6) * kTileBytes + piece_at(rr, (cc >> 5 & 1) * 4 + (lane & 3));
      };
      uint4 old[PLANES == 1 ? kPieces : PLANES][4];            // "half": of all units of this warp; "split": both parts of one
      auto fetch = [&](int u, int q, int pl) {
#pragma unroll
        for (int i = 0; i < 4; ++i) old[q][i] = __ldcg(reinterpret_cast<const uint4*>(old0 + pl * plane + line_at(u, i)));
      };
      bool go = true;
      unsigned taddr = 0;
      // "half": the old values are on their way while the products run
      const bool early = PLANES == 1 && !gram && it.parts == 1;
      if constexpr (PLANES == 1) {
        if (early) {
          go = __all_sync(0xffffffffu, tiles_wait(a.ready + it.mat, tiles_before(t, it), stop, a));
#pragma unroll
          for (int b = 0; b < kPieces; ++b)
            if (go && unit_in(warp * 4 + b)) fetch(warp * 4 + b, b, 0);
        }
        go = go && __all_sync(0xffffffffu, muon_wait(afull0 + 8 * (tile & 1), (tile >> 1) & 1, stop, a));
        tc_fence_after();
        taddr = tmem + ((unsigned)(quarter * 32) << 16) + (tile & 1) * kBN + half * kCols;
      } else {
        float acc[kCols];                                      // the sums of the drained accumulators
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
        for (int k = it.k0; k < it.k1; k += min(C::kDrain, it.k1 - k), ++tile) {
          const unsigned tt = tile & 1, tph = (tile >> 1) & 1;
          go = __all_sync(0xffffffffu, muon_wait(afull0 + 8 * tt, tph, stop, a));
          if (!go) break;
          tc_fence_after();
          taddr = tmem + ((unsigned)(quarter * 32) << 16) + tt * kBN + half * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            unsigned v[32];
            tc_load32(taddr + c, v);
            tc_wait32(v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c + j] += __uint_as_float(v[j]);
          }
          release(tt);
        }
        // They leave the registers (L2 has them): what follows needs those.
#pragma unroll
        for (int c = 0; c < kCols; c += 8) store32<float>(part + c * 32, acc + c);
      }
      // All eight warps go on or none: they meet at barriers below.
      if (!sums_go(go)) break;
      const float* joined = PLANES == 2 ? part - warp * 4096 : nullptr;
      int u0 = warp * 4, u1 = u0 + 4, du = 1;                  // this warp's units
      if (it.parts > 1) {
        if constexpr (PLANES == 1) {
#pragma unroll 1
          for (int b = 0; b < kPieces; ++b) {
            unsigned v[kPiece];
            tc_load32(taddr + b * kPiece, v);
            tc_wait32(v);
#pragma unroll
            for (int c = 0; c < kPiece; c += 8) store32<float>(part + (b * kPiece + c) * 32, reinterpret_cast<const float*>(v) + c);
          }
          release(tile++ & 1);
        }
        // The parts' blocks join a share of the tile each, when all of them are there: they were
        // dealt side by side, so none waits long (one block joining all: 6 parts of "split" 14 to 19 us).
        unsigned* const count = a.count + (it.at - it.part) * 2 + rank;
        sums_sync();
        if (threadIdx.x == 0)                                  // the barrier's writes go out with this thread's
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
        go = __all_sync(0xffffffffu, tiles_wait(count, (unsigned)(it.parts * (it.step + 1)), stop, a));
        if (!sums_go(go)) break;
        joined = a.partial + ((long long)(it.at - it.part) * 2 + rank) * tile_floats + lane * 8;
        u0 = 32 * it.part / it.parts + warp;
        u1 = 32 * (it.part + 1) / it.parts;
        du = kSumWarps;
      }
      const bool keep = finish && *(volatile unsigned*)a.failed != 0;
      const bool tall = t.rows > t.cols;
      const float kold = apply ? kA : gram ? 0.0f : kB, knew = it.phase == kSquare ? kC * kInvScale : kInvScale;
      const float rate = a.lr * t.scale * kInvScale;
      // Rows and columns past the edge's multiple of 64 are never read as k's and need no values.
#pragma unroll 1
      for (int u = u0; u < u1; u += du) {
        if (!unit_in(u)) continue;                             // the same for the warp
        if (!gram && !early) {
#pragma unroll
          for (int q = 0; q < PLANES; ++q) fetch(u, q, q);
        }
        float o[kPiece];
        if (joined) {
#pragma unroll
          for (int j = 0; j < kPiece; ++j) o[j] = 0.0f;
          const float* src = joined + (u >> 2) * 4096 + (u & 3) * kPiece * 32;
          const int parts = it.parts;
#pragma unroll 3
          for (int q = 0; q < parts; ++q, src += 2 * tile_floats) {
#pragma unroll
            for (int c = 0; c < kPiece; c += 4) {
              const float4 w = __ldcg(reinterpret_cast<const float4*>(src + (c / 8) * 256 + (c & 4)));
              o[c] += w.x;
              o[c + 1] += w.y;
              o[c + 2] += w.z;
              o[c + 3] += w.w;
            }
          }
        } else if constexpr (PLANES == 1) {
          unsigned v[kPiece];
          tc_load32(taddr + (u & 3) * kPiece, v);
          tc_wait32(v);
#pragma unroll
          for (int j = 0; j < kPiece; ++j) o[j] = __uint_as_float(v[j]);
        }
        // A row of a unit in shared memory: 64 bytes, its 16-byte pieces swizzled so that neither way meets a bank twice.
        auto mine = [&](int c) { return stage + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4); };
        auto theirs = [&](int i) { return stage + (i * 8 + (lane >> 2)) * 64 + (((lane & 3) ^ (lane >> 3 & 3)) << 4); };
        if (gram) {
#pragma unroll
          for (int j = 0; j < kPiece; ++j) o[j] *= kInvScale;
        } else {
          float w[kPiece];
#pragma unroll
          for (int q = 0; q < PLANES; ++q) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(theirs(i)) = old[q][i];
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float l[8];
              unpack8(*reinterpret_cast<const uint4*>(mine(c)), l);
#pragma unroll
              for (int j = 0; j < 8; ++j) w[8 * c + j] = q ? w[8 * c + j] + l[j] : l[j];
            }
          }
#pragma unroll
          for (int j = 0; j < kPiece; ++j) o[j] = kold * w[j] + knew * o[j];
          if constexpr (PLANES == 1) {                         // the next unit's move up
#pragma unroll
            for (int q = 0; q + 1 < kPieces; ++q)
#pragma unroll
              for (int c = 0; c < 4; ++c) old[q][c] = old[q + 1][c];
          }
        }
        const int row = unit_row(u) + lane, col = unit_col(u);
        if (!finish) {
#pragma unroll
          for (int q = 0; q < PLANES; ++q) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint4 hi, lo;
              pack8(o + 8 * c, q == 1, &hi, &lo);
              *reinterpret_cast<uint4*>(mine(c)) = q ? lo : hi;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(out0 + q * plane + line_at(u, i)) = *reinterpret_cast<const uint4*>(theirs(i));
          }
          if (!apply && it.i != it.j) {  // the same values above the diagonal: a lane's column there is its row
            const int c0 = row & 63;
            unsigned char* up = a.ws + (gram ? t.a : t.b) + ((long long)(it.j * 2 + (col >> 7)) * as + rb * 2 + (row >> 6)) * kTileBytes;
#pragma unroll
            for (int c = 0; c < kPiece; c += 2) {  // rows c and c + 1 between neighbours: two columns each
              const bool odd = lane & 1;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? o[c] : o[c + 1], 1);
              const float x = odd ? got : o[c], y = odd ? o[c + 1] : got;
              const __half2 hi = __floats2half2_rn(x, y);
              const int at = piece_at((col & 127) + c + odd, c0 >> 3) + (c0 & 6) * 2;
              *reinterpret_cast<__half2*>(up + at) = hi;
              if (PLANES == 2) {
                const float2 f = __half22float2(hi);
                *reinterpret_cast<__half2*>(up + plane + at) = __floats2half2_rn(x - f.x, y - f.y);
              }
            }
          }
        } else if (!keep) {
          const int prow = rb * kTileRows + row, pcol = it.j * kBN + col;
          if (t.param_t == EMB_T_F32) update_unit((float*)t.p, t, prow, pcol, tall, a.decay, rate, o, stage);
          else if (t.param_t == EMB_T_BF16) update_unit((__nv_bfloat16*)t.p, t, prow, pcol, tall, a.decay, rate, o, stage);
          else update_unit((__half*)t.p, t, prow, pcol, tall, a.decay, rate, o, stage);
        }
      }
      if (PLANES == 1 && it.parts == 1) release(tile++ & 1);
      // This block's share of the tile is there.
      sums_sync();
      if (threadIdx.x == 0)                                    // other blocks read it by TMA
        asm volatile("fence.proxy.async;\nred.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.ready + it.mat) : "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (pair_stopped(stop)) {  // a wait ran out: what is in flight lands before the blocks end
    const unsigned n = warp >= kSumWarps && warp < kSumWarps + 2 ? issued[warp - kSumWarps] : 0;
    if (rank == 0 && warp == kLoadWarp)
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

// ------------------------------------------------------------------ host side

struct MuonPlan {
  size_t bytes = 0;
  size_t partial = 0, count = 0, done = 0, ready = 0, squares = 0, inv_norm = 0, failed = 0;  // offsets
  size_t zero_from = 0, zero_bytes = 0;
};

// Pairs of SMs that can be at work at one time.
int pair_count() {
  static std::atomic<int> of[64];   // by device, 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return std::max(1, sm_count() / 2);
  }
  int n = of[dev].load();
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sm_count() & ~1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = MuonCfg<1>::kBytes;
    if (cudaFuncSetAttribute(product_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, MuonCfg<1>::kBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, product_kernel<1>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = std::max(1, sm_count() / 4);
    }
    of[dev].store(n);
  }
  return n;
}

// Lays out one launch group; false where a list's numbers pass 31 bits.
bool plan_group(const emb_muon_tensor* t, int n, int planes, MuonArgs* a, MuonPlan* pl) {
  long long tiles = 0, chunks = 0, xtiles = 0, ntiles[3] = {}, steps[3] = {};
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
    m.sb = (m.s + 255) / 256;
    m.lb = (m.l + 255) / 256;
    m.wide = m.rows <= m.cols && m.cols % 4 == 0 && aligned_to(m.p, 4 * ftype_bytes(t[i].param_t));
    m.param_t = t[i].param_t;
    m.grad_t = t[i].grad_t;
    m.scale = t[i].scale;
    const long long x = 8LL * m.sb * m.lb, q = 8LL * m.sb * m.sb;   // tiles of 128 x 64
    m.x = tiles * kTileBytes;
    m.a = (tiles + 2 * planes * x) * kTileBytes;
    m.b = m.a + planes * q * kTileBytes;
    tiles += planes * (2 * x + 2 * q);
    m.first[3] = (int)chunks;
    m.first[4] = (int)xtiles;
    chunks += ((long long)m.rows * m.cols + kChunk - 1) / kChunk;
    xtiles += x;
    const long long tri = (long long)m.sb * (m.sb + 1) / 2, full = (long long)m.sb * m.lb;
    ntiles[kGram] += tri;
    ntiles[kSquare] += tri;
    ntiles[kApply] += full;
    steps[kGram] += tri * ((m.l + kSlab - 1) / kSlab);
    steps[kSquare] += tri * ((m.s + kSlab - 1) / kSlab);
    steps[kApply] += full * ((m.s + kSlab - 1) / kSlab);
    if (chunks > 0x7fffffffLL || xtiles > 0x7fffffffLL || ntiles[kApply] > 0x3fffffffLL) return false;
  }
  const int pairs = pair_count();
  bool shared[3] = {};
  long long slots = 0;
  a->total[3] = (int)chunks;
  a->total[4] = (int)xtiles;
  for (int ph = 0; ph < 3; ++ph) {
    // Where there are fewer tiles than pairs a tile's k's may be shared out: a slab takes 0.27 us ("split"
    // 0.8), and a part that is written, counted and read by the last one about 3 and 1.2 for each.
    long long items = 0;
    a->slot0[ph] = (int)slots;
    for (int i = 0; i < a->mats; ++i) {
      Mat& m = a->mat[i];
      const long long k = ((ph == kGram ? m.l : m.s) + kSlab - 1) / kSlab, tiles = ph == kApply ? (long long)m.sb * m.lb : (long long)m.sb * (m.sb + 1) / 2;
      int best = 1;
      double best_us = 0.0;
      // pairs that this matrix's share of the phase's slabs would keep at work
      const double share = (double)pairs * tiles * k / steps[ph];
      for (int parts = 1; parts <= 16 && parts <= k && (parts == 1 || tiles * parts <= share + 0.5); ++parts) {
        const double us = (double)((k + parts - 1) / parts) * (planes == 2 ? 0.8 : 0.27) + (parts > 1 ? 3.0 + 1.2 * parts : 0.0);
        if (parts == 1 || us < best_us) best = parts, best_us = us;
      }
      m.parts[ph] = best;
      m.first[ph] = (int)items;
      items += tiles * best;
      if (best > 1) shared[ph] = true;
    }
    a->total[ph] = (int)items;
    if (shared[ph]) slots += items;
  }
  if (((long long)a->total[0] + a->total[1] + a->total[2]) * kSteps > 0x7fffffffLL - 4096) return false;
  a->slots = (int)slots;
  if (planes == 2) slots += pairs;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl->partial = (size_t)tiles * kTileBytes;
  pl->count = pl->partial + (size_t)slots * 2 * kTileRows * kBN * 4;
  pl->done = pl->count + up((size_t)slots * 8);
  pl->ready = pl->done + up((size_t)kMaxMats * 4);
  pl->failed = pl->ready + up((size_t)kMaxMats * 4);
  pl->inv_norm = pl->failed + 256;
  pl->squares = pl->inv_norm + up((size_t)kMaxMats * 4);
  pl->bytes = pl->squares + up((size_t)chunks * 4);
  pl->zero_from = pl->count;
  pl->zero_bytes = pl->inv_norm - pl->count;
  return true;
}

template <int PLANES>
cudaError_t launch_products(const MuonArgs& a, const CUtensorMap& map, cudaStream_t st) {
  auto* k = product_kernel<PLANES>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MuonCfg<PLANES>::kBytes);
  if (e != cudaSuccess) return e;
  const int most = std::max(a.total[0], std::max(a.total[1], a.total[2]));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * std::min(most, pair_count()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = MuonCfg<PLANES>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // the blocks wait on one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, map, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
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
      if (tensors[at + i].rows && tensors[at + i].cols) {
        Mat& m = a.mat[j++];
        m.g = grads[at + i];
        m.vec = aligned_to(m.m, 32) && aligned_to(m.g, 8 * ftype_bytes(m.grad_t));
      }
    unsigned char* ws = (unsigned char*)workspace_d;
    a.ws = ws;
    a.partial = (float*)(ws + pl.partial);
    a.count = (unsigned*)(ws + pl.count);
    a.done = (unsigned*)(ws + pl.done);
    a.ready = (unsigned*)(ws + pl.ready);
    a.failed = (unsigned*)(ws + pl.failed);
    a.inv_norm = (float*)(ws + pl.inv_norm);
    a.squares = (float*)(ws + pl.squares);
    a.flags = flags;
    a.grad_scale = o.grad_scale_d;
    a.beta = (float)o.momentum;
    a.omb = (float)(1.0 - o.momentum);
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
    // The tiles as rows of 128 bytes; they are swizzled already.  A load takes 64 rows.
    CUtensorMap map;
    if (!make_plain_map(&map, ws, pl.partial / 128, 64)) return fail(EMB_ERR_CUDA, "cuTensorMapEncodeTiled failed or is not available");
    const cudaError_t e = a.planes == 2 ? launch_products<2>(a, map, st) : launch_products<1>(a, map, st);
    if (e != cudaSuccess) return cuda_fail(e, "emb_muon_step launch");
  }
  return EMB_OK;
}
