// Rows of a plain embedding matrix by token, with a scale, and the matrix's gradient.
//   out[i] = scale W[t_i];    dW[v] (+)= scale * (sum over i with t_i = v of g[i])
// A token that is the padding gives zeros and no gradient; one outside [0, vocab) does
// too and raises a flag.
//
// The gradient.  The tokens are sorted by value, stably, so that a row's gradients are
// summed in the order in which they came: results repeat bitwise and do not depend on
// atomics.  Launches: a histogram of every digit; one pass a digit, which ranks 4096 tokens a
// block and learns from the blocks before it where its digits go; other blocks of these
// launches write zeros into dW meanwhile; the sums; the joining of runs.
//
// Sums.  Sorted positions are cut into chunks of equal length, so that a token which
// occurs a hundred thousand times costs no block more than another.  A thread walks one
// chunk for V neighbouring columns, eight rows of g (four of 32 bytes) on their way at a time.  A run of equal
// tokens inside a chunk is written at once; the piece of a run that began before the
// chunk, and the piece of one that goes on after it, are left as float32 and joined, in order.
//
// Bound by memory.  1,638,400 rows of 128 columns float32 to bf16: lookup 109 us; the gradient of as many bf16
// rows into a million: histogram 29, three passes of the sort 112 with the zeros, sums 81, joins 23.
#include <algorithm>

#include "emb_tc.cuh"

namespace emb {
namespace {

constexpr int kDigits = 256;
constexpr int kSortThreads = 256, kSortItems = 16, kSortTile = kSortThreads * kSortItems;
constexpr int kMaxPasses = 4;
constexpr long long kWalks = 32768;           // threads that walk, below which walks are shortened
constexpr int kMaxChunk = 64, kMinChunk = 8;  // sorted positions of one thread's walk
constexpr unsigned kAggregate = 1u << 30, kInclusive = 2u << 30, kCount = (1u << 30) - 1;

struct TokenArgs {
  const void* tokens;
  long long n, vocab, padding;
  int wide;              // tokens are int64
  unsigned* flags;
};

__device__ __forceinline__ long long token_at(const TokenArgs& a, long long i) {
  return a.wide ? __ldg((const long long*)a.tokens + i) : (long long)__ldg((const int*)a.tokens + i);
}
// Whether a token names a row; raises the flag for one that is neither a row nor the padding.
__device__ __forceinline__ bool names_row(const TokenArgs& a, long long t) {
  if (t == a.padding) return false;
  if ((unsigned long long)t < (unsigned long long)a.vocab) return true;
  atomicOr(a.flags, EMB_FLAG_BAD_TOKEN);
  return false;
}

// V neighbouring elements, as float32.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* o) {
  if constexpr (V == 8) {
    Raw8<T> r;
    r.load(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = r.get(j);
  } else if constexpr (V == 4 && sizeof(T) == 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    o[0] = f.x, o[1] = f.y, o[2] = f.z, o[3] = f.w;
  } else if constexpr (V == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = to_f32<T>(e[j]);
  } else {
    static_assert(V == 1, "vector widths");
    o[0] = to_f32<T>(*p);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* v) {
  if constexpr (V == 8) {
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.set2(j, v[2 * j], v[2 * j + 1]);
    r.store(p);
  } else if constexpr (V == 4 && sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (V == 4) {
    uint2 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = from_f32<T>(v[j]);
    *reinterpret_cast<uint2*>(p) = u;
  } else {
    *p = from_f32<T>(v[0]);
  }
}

// V neighbouring elements as they lie in memory.
template <typename T, int V>
struct RawV {
  T v[V];
  __device__ __forceinline__ void load(const T* p) { v[0] = *p; }
  __device__ __forceinline__ float get(int i) const { return to_f32<T>(v[i]); }
};
template <typename T>
struct RawV<T, 8> : Raw8<T> {};
template <typename T>
struct RawV<T, 4> {
  static constexpr int kWords = sizeof(T);
  unsigned w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ float get(int i) const { return to_f32<T>(reinterpret_cast<const T*>(w)[i]); }
};

// V = kStrided: rows off the vectors' alignment.  A thread has four columns, a quarter of a row apart,
// so that neighbouring threads still read side by side, and asks four times less often where its
// rows are (488,277 x 261 float32: 211 us, and 244 with one column a thread), though at three blocks an SM 376 bytes a
// thread are spilled.
constexpr int kStrided = -4;
template <typename T>
struct RawV<T, kStrided> {
  T v[4];
  __device__ __forceinline__ void load(const T* p, int step, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? p[j * step] : from_f32<T>(0.0f);
  }
  __device__ __forceinline__ float get(int i) const { return to_f32<T>(v[i]); }
};

// ------------------------------------------------------------------ lookup

struct LookupArgs {
  TokenArgs t;
  const void* w;
  void* out;
  long long ldw, ldo;
  int dim, pieces;       // of V elements, in a row
  float scale;
};

template <typename WT, typename OT, int V>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupArgs a) {
  const long long total = a.t.n * a.pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long row = total <= 0xffffffffLL ? (unsigned)i / (unsigned)a.pieces : i / a.pieces;
    const int piece = (int)(i - row * a.pieces);
    const long long t = token_at(a.t, row);
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.0f;
    if (names_row(a.t, t)) {
      load_v<WT, V>((const WT*)a.w + t * a.ldw + piece * V, v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= a.scale;
    }
    store_v<OT, V>((OT*)a.out + row * a.ldo + piece * V, v);
  }
}

// ------------------------------------------------------------------ sort

struct SortArgs {
  TokenArgs t;
  unsigned *hist;        // [kMaxPasses][kDigits]
  unsigned *next;        // [kMaxPasses]: the next tile of each pass
  unsigned *status;      // [passes][tiles][kDigits]: a tile's counts, alone or with all before it
  unsigned *valid;       // tokens that name rows; and whether a wait ran out
  unsigned *key[2], *val[2];
  int passes, bits, tiles;
  int lost_tile;         // the tile whose wait counts as run out; -1: none
};

// Zeros into dW, before the sums are written.  The sort is a chain of latencies that leaves the memory
// idle, so each of its launches has further blocks that write a share of them: one an SM, and
// the first ones, as the sort's fill what they leave (behind those, the two took turns).
struct ZeroArgs {
  void* dw;
  long long ldw, rows_a_launch, vocab;
  int pieces, w_t, blocks;   // pieces of V elements, in a row; blocks 0: nothing to do
  int rows_a_warp;           // at a time: up to 32, about 1024 pieces
};
template <int V>
__device__ __forceinline__ void zero_rows(const ZeroArgs& z, int launch, int block) {
  const int lane = threadIdx.x & 31, more = 32 / z.pieces, rest = 32 - more * z.pieces, warps = z.blocks * (kSortThreads / 32);
  const long long from = launch * z.rows_a_launch, to = min(z.vocab, from + z.rows_a_launch);
  float zero[V];
#pragma unroll
  for (int j = 0; j < V; ++j) zero[j] = 0.0f;
  for (long long w = from + (long long)(block * (kSortThreads / 32) + (threadIdx.x >> 5)) * z.rows_a_warp; w < to; w += (long long)warps * z.rows_a_warp) {
    const int rows = (int)min((long long)z.rows_a_warp, to - w);
    int r = lane / z.pieces, p = lane - r * z.pieces;
    while (r < rows) {
      const long long e = (w + r) * z.ldw + p * V;
      if (z.w_t == EMB_T_F32) store_v<float, V>((float*)z.dw + e, zero);
      else if (z.w_t == EMB_T_BF16) store_v<__nv_bfloat16, V>((__nv_bfloat16*)z.dw + e, zero);
      else store_v<__half, V>((__half*)z.dw + e, zero);
      r += more;
      p += rest;
      if (p >= z.pieces) p -= z.pieces, ++r;
    }
  }
}

// Eight tokens a thread at a time, all loads before any use.
template <int V>
__global__ void __launch_bounds__(256) histogram_kernel(const __grid_constant__ SortArgs a, const __grid_constant__ ZeroArgs z, int blocks) {
  constexpr int kBatch = 8;
  __shared__ unsigned h[kMaxPasses * kDigits];
  if ((int)blockIdx.x < z.blocks) {
    zero_rows<V>(z, a.passes, blockIdx.x);
    return;
  }
  for (int i = threadIdx.x; i < a.passes * kDigits; i += 256) h[i] = 0;
  __syncthreads();
  const unsigned mask = (1u << a.bits) - 1;
  for (long long i = (long long)(blockIdx.x - z.blocks) * 256 * kBatch + threadIdx.x; i < a.t.n; i += (long long)blocks * 256 * kBatch) {
    long long t[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) t[q] = i + q * 256 < a.t.n ? token_at(a.t, i + q * 256) : a.t.padding;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (!names_row(a.t, t[q])) continue;
      for (int p = 0; p < a.passes; ++p) atomicAdd(&h[p * kDigits + (((unsigned)t[q] >> (p * a.bits)) & mask)], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.passes * kDigits; i += 256)
    if (h[i]) atomicAdd(a.hist + i, h[i]);
}

// Exclusive sum over 256 threads' values; *total: their sum.
__device__ __forceinline__ unsigned scan256(unsigned v, unsigned* warp_sums, unsigned* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  unsigned before = 0, all = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    before += j < w ? warp_sums[j] : 0;
    all += warp_sums[j];
  }
  *total = all;
  return before + x - v;
}

// Ranks of a lane's items among the warp's equal digits, in order; `count`: how many of each the warp has.
__device__ __forceinline__ void rank_digits(const unsigned* k, unsigned in, int shift, unsigned mask, unsigned* count, unsigned* rank) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    const bool ok = (in >> q) & 1u;
    const unsigned digit = ok ? (k[q] >> shift) & mask : 0xffffu;
    const unsigned same = __match_any_sync(0xffffffffu, digit);
    const unsigned below = __popc(same & ((1u << lane) - 1));
    unsigned old = 0;
    if (ok) old = count[digit];
    __syncwarp();
    if (ok && below == 0) count[digit] = old + __popc(same);
    __syncwarp();
    if (q & 1) rank[q / 2] |= (old + below) << 16;
    else rank[q / 2] = old + below;
  }
}
__device__ __forceinline__ unsigned rank_of(const unsigned* rank, int q) { return q & 1 ? rank[q / 2] >> 16 : rank[q / 2] & 0xffffu; }

// All passes of one tile's tokens by one block, in shared memory: no histogram, no other
// launch (50 tokens of 64 columns into 1000 rows: 33 us with them).
template <int V>
__global__ void __launch_bounds__(kSortThreads) sort_one_kernel(const __grid_constant__ SortArgs a, const __grid_constant__ ZeroArgs z) {
  __shared__ unsigned count[8][kDigits], sums[8];
  __shared__ uint2 held[kSortTile];
  if ((int)blockIdx.x < z.blocks) {
    zero_rows<V>(z, 0, blockIdx.x);
    return;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, d = threadIdx.x, at = w * 32 * kSortItems + lane;
  const unsigned mask = (1u << a.bits) - 1;
  unsigned k[kSortItems], v[kSortItems], rank[kSortItems / 2], in = 0, all = 0;
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    const int i = at + q * 32;
    k[q] = v[q] = 0;
    if (i < a.t.n) {
      const long long t = token_at(a.t, i);
      k[q] = (unsigned)t;
      v[q] = (unsigned)i;
      in |= names_row(a.t, t) ? 1u << q : 0u;
    }
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
#pragma unroll
    for (int j = 0; j < 8; ++j) count[j][d] = 0;
    __syncthreads();
    rank_digits(k, in, shift, mask, count[w], rank);
    __syncthreads();
    unsigned mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned c = count[j][d];
      count[j][d] = mine;
      mine += c;
    }
    const unsigned first = scan256(mine, sums, &all);
#pragma unroll
    for (int j = 0; j < 8; ++j) count[j][d] += first;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortItems; ++q)
      if ((in >> q) & 1u) held[count[w][(k[q] >> shift) & mask] + rank_of(rank, q)] = make_uint2(k[q], v[q]);
    __syncthreads();
    in = 0;
#pragma unroll
    for (int q = 0; q < kSortItems; ++q) {
      const unsigned i = at + q * 32;
      if (i < all) {
        const uint2 item = held[i];
        k[q] = item.x;
        v[q] = item.y;
        in |= 1u << q;
      }
    }
  }
  const int end = (a.passes - 1) & 1;
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    if ((in >> q) & 1u) {
      a.key[end][at + q * 32] = k[q];
      a.val[end][at + q * 32] = v[q];
    }
  }
  if (threadIdx.x == 0) {
    a.valid[0] = all;
    a.valid[1] = 0;
  }
}

// One stable pass.  Tiles are numbered as they start, so those before one are at work or
// done, and what it waits for comes; the wait is bounded all the same.
template <bool FIRST, int V>
__global__ void __launch_bounds__(kSortThreads, 4) sort_kernel(const __grid_constant__ SortArgs a, const __grid_constant__ ZeroArgs z, int pass) {
  if ((int)blockIdx.x < z.blocks) {
    zero_rows<V>(z, pass, blockIdx.x);
    return;
  }
  __shared__ unsigned count[8][kDigits], base[kDigits], sums[8];
  __shared__ uint2 held[kSortTile];
  __shared__ int tile_slot;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, d = threadIdx.x;
  if (threadIdx.x == 0) tile_slot = (int)atomicAdd(a.next + pass, 1u);
#pragma unroll
  for (int j = 0; j < 8; ++j) count[j][d] = 0;
  unsigned valid;
  const unsigned first = scan256(a.hist[pass * kDigits + d], sums, &valid);  // of all tiles' digits below d; a barrier is inside
  const int tile = tile_slot;
  const long long n = FIRST ? a.t.n : valid, at = (long long)tile * kSortTile + w * 32 * kSortItems + lane;
  if ((long long)tile * kSortTile >= n) return;
  const unsigned *key = a.key[(pass & 1) ^ 1], *val = a.val[(pass & 1) ^ 1];
  const int shift = pass * a.bits;
  const unsigned mask = (1u << a.bits) - 1;
  unsigned k[kSortItems], v[kSortItems], rank[kSortItems / 2];   // ranks: two to a word
  unsigned in = 0;
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    const long long i = at + q * 32;
    k[q] = v[q] = 0;
    if (i < n) {
      if (FIRST) {
        const long long t = token_at(a.t, i);
        const bool row = t != a.t.padding && (unsigned long long)t < (unsigned long long)a.t.vocab;
        k[q] = (unsigned)t;
        v[q] = (unsigned)i;
        in |= row ? 1u << q : 0u;
      } else {
        k[q] = key[i];
        v[q] = val[i];
        in |= 1u << q;
      }
    }
  }
  rank_digits(k, in, shift, mask, count[w], rank);
  __syncthreads();
  unsigned mine = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned c = count[j][d];
    count[j][d] = mine;
    mine += c;
  }
  unsigned* st = a.status + ((long long)pass * a.tiles + tile) * kDigits + d;
  if (d <= mask) *(volatile unsigned*)st = mine | (tile == 0 ? kInclusive : kAggregate);
  // The tile in the order of its digits, in shared memory: a digit's items then leave as
  // neighbours (each from its own lane, a sector an item: twice the time).
  unsigned all;
  const unsigned local = scan256(mine, sums, &all);
#pragma unroll
  for (int j = 0; j < 8; ++j) count[j][d] += local;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    if ((in >> q) & 1u) {
      const unsigned to = count[w][(k[q] >> shift) & mask] + rank_of(rank, q);
      held[to] = make_uint2(k[q], v[q]);
    }
  }
  unsigned before = 0;
  if (d <= mask) {
    // 16 tiles' words at a time: one after the other, each a round trip to L2, they took
    // most of a pass.  A word that is not there yet is asked for again, from it on.
    constexpr int kLook = 16;
    int j = tile - 1;
    for (unsigned i = 0; j >= 0 && i < kWaitLimit && tile != a.lost_tile; ++i) {
      unsigned word[kLook];
#pragma unroll
      for (int q = 0; q < kLook; ++q)
        word[q] = q <= j ? *(volatile unsigned*)(st - (long long)(tile - j + q) * kDigits) : (unsigned)kInclusive;
      bool more = true;
#pragma unroll
      for (int q = 0; q < kLook; ++q) {
        if (more && word[q] >= kAggregate) {
          before += word[q] & kCount;
          --j;
          if (word[q] >= kInclusive) j = -1;
        }
        more = more && word[q] >= kAggregate && word[q] < kInclusive;
      }
    }
    if (j >= 0) {                                             // the wait ran out
      atomicOr(a.t.flags, EMB_FLAG_OP_TIMEOUT);
      *(volatile unsigned*)(a.valid + 1) = 1u;
    }
    if (tile) *(volatile unsigned*)st = (before + mine) | kInclusive;
  }
  base[d] = first + before - local;                           // less the item's place in the tile
  if (FIRST && tile == 0 && d == 0) *a.valid = valid;
  __syncthreads();
  unsigned *to_key = a.key[pass & 1], *to_val = a.val[pass & 1];
  for (unsigned i = threadIdx.x; i < all; i += kSortThreads) {
    const uint2 item = held[i];
    const unsigned to = base[(item.x >> shift) & mask] + i;
    if (to < valid) {  // always, unless a wait ran out
      to_key[to] = item.x;
      to_val[to] = item.y;
    }
  }
}

// ------------------------------------------------------------------ sums

struct SumArgs {
  const unsigned *key, *val, *valid;
  const void* g;
  void* dw;
  float *head, *tail;    // [chunks][dim]
  long long ldg, ldw, n;   // n: all tokens
  int dim, pieces, w_t, accumulate, chunk;
  float scale;
};

// Sorted positions to sum.  None after a wait that ran out: places that no token was written
// to hold anything, and would be taken for rows.
__device__ __forceinline__ unsigned sorted(const SumArgs& a) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.valid));
  return v.y ? 0u : v.x;
}

template <int V>
__device__ __forceinline__ void write_row(const SumArgs& a, unsigned row, int piece, float* acc) {
  const long long e = row * a.ldw + piece * V;
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] *= a.scale;
  auto put = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    if (a.accumulate) {
      float old[V];
#pragma unroll
      for (int j = 0; j < V; ++j) old[j] = to_f32<T>(p[j]);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += old[j];
    }
    store_v<T, V>(p, acc);
  };
  if (a.w_t == EMB_T_F32) put((float*)a.dw + e);
  else if (a.w_t == EMB_T_BF16) put((__nv_bfloat16*)a.dw + e);
  else put((__half*)a.dw + e);
}

template <typename GT, int V>
__global__ void __launch_bounds__(256, V == kStrided ? 3 : 2) sum_kernel(const __grid_constant__ SumArgs a) {
  const unsigned n = sorted(a);
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long chunk = i / a.pieces;
  const int piece = (int)(i - chunk * a.pieces);
  if (chunk * a.chunk >= n) return;
  const unsigned s = (unsigned)(chunk * a.chunk), e = min(n, s + a.chunk);
  unsigned cur = a.key[s];
  bool head = s > 0 && a.key[s - 1] == cur;
  constexpr int N = V == kStrided ? 4 : V;
  const int step = a.pieces, mine = V == kStrided ? (a.dim - piece + step - 1) / step : N;  // columns of this thread that there are
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  const long long first = chunk * a.dim + (V == kStrided ? piece : piece * V);
  auto flush = [&](float* to) {
    if constexpr (V == kStrided) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < mine) to[first + j * step] = acc[j];
    } else {
      store_v<float, V>(to + first, acc);
    }
  };
  auto whole = [&](unsigned row) {  // a run that is complete
    if constexpr (V == kStrided) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < mine) write_row<1>(a, row, piece + j * step, acc + j);
    } else {
      write_row<V>(a, row, piece, acc);
    }
  };
  constexpr int kRows = V * (int)sizeof(GT) > 16 || V == kStrided ? 4 : 8;   // on their way at a time
  unsigned k[kRows], v[kRows];
  auto ask = [&](unsigned b) {
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const unsigned at = min(b + q, e - 1);
      k[q] = __ldg(a.key + at);
      v[q] = __ldg(a.val + at);
    }
  };
  ask(s);
  for (unsigned b = s; b < e; b += kRows) {
    RawV<GT, V> x[kRows];
    unsigned now[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if constexpr (V == kStrided) x[q].load((const GT*)a.g + v[q] * a.ldg + piece, step, mine);
      else x[q].load((const GT*)a.g + v[q] * a.ldg + piece * V);
      now[q] = k[q];
    }
    if (b + kRows < e) ask(b + kRows);                  // the next ones' places, while these are on their way
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if (b + q < e) {
        if (now[q] != cur) {
          if (head) flush(a.head);
          else whole(cur);
          head = false;
          cur = now[q];
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += x[q].get(j);
      }
    }
  }
  if (head) flush(a.head);
  else if (e < n && a.key[e] == cur) flush(a.tail);
  else whole(cur);
}

// Joins the run that passes the end of `chunk` and begins in it: its tail here and the heads of the
// chunks up to `last`.  `threads` threads (this one is the `me`-th) take this block's 32 pieces of a
// row, and where threads are left, groups of them take consecutive shares of the heads, added in order.
template <int V, typename Sync>
__device__ __forceinline__ void join_run(const SumArgs& a, unsigned row, long long chunk, int last, int threads, int me, float* share, Sync sync) {
  const int heads = last - (int)chunk, p0 = blockIdx.y * 32;
  {
    const int width = min(32, a.pieces - p0), groups = min(threads / width, heads), g = me / width, piece = p0 + me % width;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    if (g < groups) {
      const int from = (int)chunk + 1 + (int)((long long)heads * g / groups), to = (int)chunk + 1 + (int)((long long)heads * (g + 1) / groups);
      if (g == 0) load_v<float, V>(a.tail + chunk * a.dim + piece * V, acc);
      constexpr int kBatch = V == 1 ? 16 : 4;
      int c = from;
      for (; c + kBatch <= to; c += kBatch) {
        float x[kBatch][V];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) load_v<float, V>(a.head + (long long)(c + q) * a.dim + piece * V, x[q]);
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += x[q][j];
      }
      for (; c < to; ++c) {
        float x[V];
        load_v<float, V>(a.head + (long long)c * a.dim + piece * V, x);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += x[j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) share[me * V + j] = acc[j];
    }
    sync();
    if (me < width) {
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.0f;
      for (int q = 0; q < groups; ++q)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += share[(q * width + me) * V + j];
      write_row<V>(a, row, piece, acc);
    }
    sync();
  }
}

// Runs that pass a chunk's end.  A warp takes the one that begins in its chunk, if there is
// one; a run of many chunks is left to the whole block.
template <int V>
__global__ void __launch_bounds__(256, 5) join_runs_kernel(const __grid_constant__ SumArgs a) {
  constexpr int kLong = 64;             // chunks
  __shared__ float share[256 * V];
  __shared__ int last_of[8];            // of a warp's run that is long, else -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long chunk = blockIdx.x * 8LL + warp, e = (chunk + 1) * a.chunk;
  // All that the usual run needs is asked for at once: keys past the valid ones are there, but mean nothing.
  const unsigned n = sorted(a);
  const long long ahead = e + lane * (long long)a.chunk;
  const unsigned start = ahead < a.n ? a.key[ahead] : 0;                // of the chunks that follow, one a lane
  unsigned here = 0, first = 0, before = 0;
  if (e < a.n) {
    here = a.key[e - 1];
    first = a.key[e - a.chunk];
    before = chunk > 0 ? a.key[e - a.chunk - 1] : ~0u;
  }
  const int chunks = (int)((n + a.chunk - 1LL) / a.chunk);
  if (blockIdx.x * 8LL >= chunks) return;
  const unsigned cur = __shfl_sync(0xffffffffu, start, 0);
  // a run passes the end, and it began here
  const bool have = e < n && here == cur && !(first == cur && before == cur);
  int lo = (int)chunk + 1;
  if (have) {  // the last chunk whose first token is `cur`
    int hi = chunks - 1;
    const unsigned same = __ballot_sync(0xffffffffu, ahead < n && start == cur);
    lo += __popc(same) - 1;
    if (same != ~0u) hi = lo;
    while (lo < hi) {  // 32 places at a time
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const unsigned more = __ballot_sync(0xffffffffu, at <= hi && a.key[(long long)at * a.chunk] == cur);
      lo += __popc(more) * step;
      hi = min(hi, lo + step - 1);
    }
  }
  const bool is_long = have && lo - (int)chunk > kLong;
  if (lane == 0) last_of[warp] = is_long ? lo : -1;
  if (have && !is_long) join_run<V>(a, cur, chunk, lo, 32, lane, share + warp * 32 * V, [] { __syncwarp(); });
  __syncthreads();
  for (int w = 0; w < 8; ++w) {
    if (last_of[w] < 0) continue;       // the same for the block
    const long long c = blockIdx.x * 8LL + w;
    join_run<V>(a, a.key[(c + 1) * a.chunk], c, last_of[w], 256, threadIdx.x, share, [] { __syncthreads(); });
  }
}

// ------------------------------------------------------------------ host side

struct TokenPlan {
  int passes = 0, bits = 0, tiles = 0, chunk = kMaxChunk;
  long long chunks = 0;
  size_t zero_bytes = 0;  // hist, next, status, from the start on
  size_t next = 0, status = 0, key[2] = {}, val[2] = {}, head = 0, tail = 0, bytes = 0;
};

TokenPlan plan_tokens(long long n, long long vocab, long long dim) {
  TokenPlan pl;
  if (n == 0 || vocab == 0 || dim == 0) return pl;
  int bits = 1;
  while (bits < 31 && (vocab - 1) >> bits) ++bits;
  pl.passes = (bits + 7) / 8;
  pl.bits = (bits + pl.passes - 1) / pl.passes;
  pl.tiles = (int)((n + kSortTile - 1) / kSortTile);
  // Shorter walks where there are few of them: half as many additions one after the other, twice as many
  // pieces to join.
  while (pl.chunk > kMinChunk && (n + pl.chunk - 1) / pl.chunk * ((dim + 7) / 8) < kWalks) pl.chunk /= 2;
  pl.chunks = (n + pl.chunk - 1) / pl.chunk;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl.next = kMaxPasses * kDigits * 4;
  pl.status = pl.next + 256;
  pl.zero_bytes = pl.status + (size_t)pl.passes * pl.tiles * kDigits * 4;
  size_t at = pl.zero_bytes;
  for (int j = 0; j < 2; ++j) {
    pl.key[j] = at;
    at += up((size_t)n * 4);
    pl.val[j] = at;
    at += up((size_t)n * 4);
  }
  pl.head = at;
  at += up((size_t)pl.chunks * dim * 4);
  pl.tail = at;
  pl.bytes = at + up((size_t)pl.chunks * dim * 4);
  return pl;
}

// Elements an access: 8, 4 or 1, as the rows' alignment allows.
int vector_of(int dim, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds, std::initializer_list<int> types) {
  for (int v : {8, 4}) {
    bool ok = dim % v == 0;
    auto ld = lds.begin();
    auto t = types.begin();
    for (const void* p : ptrs) {
      const size_t b = ftype_bytes(*t);
      ok = ok && aligned_to(p, v * b) && *ld % v == 0;
      ++ld;
      ++t;
    }
    if (ok) return v;
  }
  return 1;
}

emb_status check_tokens(const void* tokens, emb_itype t, int64_t n, int64_t vocab, int64_t dim) {
  if (t != EMB_I32 && t != EMB_I64) return fail(EMB_ERR_INVALID_ARG, "bad token type");
  if (n < 0 || vocab < 0 || dim < 0) return fail(EMB_ERR_INVALID_ARG, "negative n, vocab or dim");
  if (n > EMB_MAX_TOKENS) return fail(EMB_ERR_UNSUPPORTED, "more than EMB_MAX_TOKENS tokens");
  if (vocab > 0x7fffffffLL || dim > 65536) return fail(EMB_ERR_UNSUPPORTED, "vocab above 2^31 - 1 or dim above 65,536");
  if (n > 0 && dim > 0 && !tokens) return fail(EMB_ERR_INVALID_ARG, "tokens is NULL");
  if (!aligned_to(tokens, t == EMB_I64 ? 8 : 4)) return fail(EMB_ERR_INVALID_ARG, "tokens are not aligned to their elements");
  return EMB_OK;
}

template <typename WT, typename OT>
void launch_lookup(const LookupArgs& a, int v, cudaStream_t st) {
  const long long total = a.t.n * a.pieces;
  const int grid = (int)std::min<long long>((total + 255) / 256, 32LL * sm_count());
  if (v == 8) lookup_kernel<WT, OT, 8><<<grid, 256, 0, st>>>(a);
  else if (v == 4) lookup_kernel<WT, OT, 4><<<grid, 256, 0, st>>>(a);
  else lookup_kernel<WT, OT, 1><<<grid, 256, 0, st>>>(a);
}
template <typename WT>
void launch_lookup_to(const LookupArgs& a, emb_ftype out_t, int v, cudaStream_t st) {
  if (out_t == EMB_T_F32) launch_lookup<WT, float>(a, v, st);
  else if (out_t == EMB_T_BF16) launch_lookup<WT, __nv_bfloat16>(a, v, st);
  else launch_lookup<WT, __half>(a, v, st);
}

template <typename GT, int V>
cudaError_t launch_sums(const SumArgs& a, long long chunks, cudaStream_t st) {
  SumArgs w = a;
  if (V == 1) w.pieces = (a.dim + 3) / 4;
  const long long blocks = (chunks * w.pieces + 255) / 256;
  sum_kernel<GT, V == 1 ? kStrided : V><<<(unsigned)blocks, 256, 0, st>>>(w);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (chunks > 1) join_runs_kernel<V><<<dim3((unsigned)((chunks + 7) / 8), (a.pieces + 31) / 32), 256, 0, st>>>(a);
  return cudaGetLastError();
}
template <int V>
cudaError_t launch_sums_of(const SumArgs& a, emb_ftype g_t, long long chunks, cudaStream_t st) {
  if (g_t == EMB_T_F32) return launch_sums<float, V>(a, chunks, st);
  if (g_t == EMB_T_BF16) return launch_sums<__nv_bfloat16, V>(a, chunks, st);
  return launch_sums<__half, V>(a, chunks, st);
}
template <int V>
cudaError_t launch_grad(const SortArgs& s, const ZeroArgs& z, const SumArgs& a, emb_ftype g_t, long long chunks, size_t zero_bytes, cudaStream_t st) {
  cudaError_t e;
  if (s.tiles == 1) {
    sort_one_kernel<V><<<1 + z.blocks, kSortThreads, 0, st>>>(s, z);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_sums_of<V>(a, g_t, chunks, st) : e;
  }
  e = cudaMemsetAsync(s.hist, 0, zero_bytes, st);
  if (e != cudaSuccess) return e;
  const int blocks = (int)std::min<long long>((a.n + 2047) / 2048, 8LL * sm_count());
  histogram_kernel<V><<<blocks + z.blocks, 256, 0, st>>>(s, z, blocks);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  for (int p = 0; p < s.passes; ++p) {
    if (p == 0) sort_kernel<true, V><<<s.tiles + z.blocks, kSortThreads, 0, st>>>(s, z, p);
    else sort_kernel<false, V><<<s.tiles + z.blocks, kSortThreads, 0, st>>>(s, z, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_sums_of<V>(a, g_t, chunks, st);
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_token_fwd(const void* weight_d, emb_ftype weight_t, int64_t vocab, int64_t dim, int64_t ldw,
                                    const void* tokens_d, emb_itype token_t, int64_t n, int64_t padding, float scale, void* out_d,
                                    emb_ftype out_t, int64_t ldo, void* stream) {
  if (!good_ftype(weight_t) || !good_ftype(out_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  const emb_status rc = check_tokens(tokens_d, token_t, n, vocab, dim);
  if (rc != EMB_OK) return rc;
  if (ldw < dim || ldo < dim) return fail(EMB_ERR_INVALID_ARG, "ldw or ldo below dim");
  if (n == 0 || dim == 0) return EMB_OK;
  if (!out_d || (vocab > 0 && !weight_d)) return fail(EMB_ERR_INVALID_ARG, "weight or out is NULL");
  if (!aligned_to(weight_d, ftype_bytes(weight_t)) || !aligned_to(out_d, ftype_bytes(out_t)))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  unsigned* flags = nullptr;
  EMB_CUDA(op_flags(&flags));
  const int v = vector_of((int)dim, {weight_d, out_d}, {ldw, ldo}, {weight_t, out_t});
  const LookupArgs a{{tokens_d, n, vocab, padding, token_t == EMB_I64, flags}, weight_d, out_d, ldw, ldo, (int)dim, (int)dim / v, scale};
  cudaStream_t st = (cudaStream_t)stream;
  if (weight_t == EMB_T_F32) launch_lookup_to<float>(a, out_t, v, st);
  else if (weight_t == EMB_T_BF16) launch_lookup_to<__nv_bfloat16>(a, out_t, v, st);
  else launch_lookup_to<__half>(a, out_t, v, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "lookup_kernel launch");
  return EMB_OK;
}

extern "C" emb_status emb_token_bwd_workspace_size(int64_t n, int64_t vocab, int64_t dim, size_t* bytes) {
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  const emb_status rc = check_tokens((const void*)256, EMB_I64, n, vocab, dim);
  if (rc != EMB_OK) return rc;
  *bytes = plan_tokens(n, vocab, dim).bytes;
  return EMB_OK;
}

extern "C" emb_status emb_token_bwd(const void* grad_d, emb_ftype grad_t, int64_t ldg, const void* tokens_d, emb_itype token_t,
                                    int64_t n, int64_t padding, int64_t vocab, int64_t dim, float scale, int32_t accumulate,
                                    void* dweight_d, emb_ftype weight_t, int64_t ldw, void* workspace_d, size_t ws_bytes,
                                    void* stream) {
  if (!good_ftype(grad_t) || !good_ftype(weight_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  const emb_status rc = check_tokens(tokens_d, token_t, n, vocab, dim);
  if (rc != EMB_OK) return rc;
  if (ldw < dim || ldg < dim) return fail(EMB_ERR_INVALID_ARG, "ldw or ldg below dim");
  if (vocab == 0 || dim == 0) return EMB_OK;
  if (!dweight_d || (n > 0 && !grad_d)) return fail(EMB_ERR_INVALID_ARG, "grad or dweight is NULL");
  if (!aligned_to(grad_d, ftype_bytes(grad_t)) || !aligned_to(dweight_d, ftype_bytes(weight_t)))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  cudaStream_t st = (cudaStream_t)stream;
  if (n == 0) {
    if (!accumulate)
      EMB_CUDA(cudaMemset2DAsync(dweight_d, ldw * ftype_bytes(weight_t), 0, dim * ftype_bytes(weight_t), vocab, st));
    return EMB_OK;
  }
  const TokenPlan pl = plan_tokens(n, vocab, dim);
  if (!workspace_d || ws_bytes < pl.bytes)
    return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_token_bwd_workspace_size()");
  if (!aligned_to(workspace_d, 256)) return fail(EMB_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  unsigned* flags = nullptr;
  EMB_CUDA(op_flags(&flags));
  const int v = vector_of((int)dim, {grad_d, dweight_d}, {ldg, ldw}, {grad_t, weight_t});
  if ((pl.chunks * (dim / v) + 255) / 256 > 0x7fffffffLL) return fail(EMB_ERR_UNSUPPORTED, "n * dim too large");
  unsigned char* ws = (unsigned char*)workspace_d;
  SortArgs s{{tokens_d, n, vocab, padding, token_t == EMB_I64, flags},
             (unsigned*)ws, (unsigned*)(ws + pl.next), (unsigned*)(ws + pl.status), (unsigned*)(ws + pl.next) + kMaxPasses, {}, {}, pl.passes, pl.bits, pl.tiles, -1};
  int lost;
  unsigned lost_step;
  lost_wait(&lost, &lost_step);
  if (lost == 0) s.lost_tile = (int)std::min(lost_step, 0x7fffffffu);
  for (int j = 0; j < 2; ++j) {
    s.key[j] = (unsigned*)(ws + pl.key[j]);
    s.val[j] = (unsigned*)(ws + pl.val[j]);
  }
  const int end = (pl.passes - 1) & 1;
  const SumArgs a{s.key[end], s.val[end], s.valid, grad_d, dweight_d, (float*)(ws + pl.head), (float*)(ws + pl.tail),
                  ldg, ldw, n, (int)dim, (int)dim / v, weight_t, accumulate != 0, pl.chunk, scale};
  // blocks that write zeros: one an SM beside a sort's, four beside one block
  const long long share = pl.tiles == 1 ? vocab : (vocab + pl.passes) / (pl.passes + 1);   // of a launch's
  const int rows_a_warp = (int)std::max<long long>(1, std::min<long long>(32, 1024 / (dim / v)));
  const long long rows_a_block = rows_a_warp * (kSortThreads / 32);
  const ZeroArgs z{dweight_d, ldw, share, vocab, (int)dim / v, weight_t,
                   accumulate ? 0 : (int)std::min<long long>((share + rows_a_block - 1) / rows_a_block, (pl.tiles == 1 ? 4LL : 1LL) * sm_count()),
                   rows_a_warp};
  const cudaError_t e = v == 8 ? launch_grad<8>(s, z, a, grad_t, pl.chunks, pl.zero_bytes, st)
                        : v == 4 ? launch_grad<4>(s, z, a, grad_t, pl.chunks, pl.zero_bytes, st)
                                 : launch_grad<1>(s, z, a, grad_t, pl.chunks, pl.zero_bytes, st);
  if (e != cudaSuccess) return cuda_fail(e, "emb_token_bwd launch");
  return EMB_OK;
}
