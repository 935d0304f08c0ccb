// Rows of a plain embedding matrix by token, with a scale, and the matrix's gradient.
//   out[i] = scale W[t_i];    dW[v] (+)= scale * (sum over i with t_i = v of g[i])
// A token that is the padding gives zeros and no gradient; one outside [0, vocab) does
// too and raises a flag.
//
// The gradient.  The tokens are sorted by value, stably, so that a row's gradients are
// summed in the order in which they came: results repeat bitwise and do not depend on
// atomics.  Launches: a histogram of every digit (and a bit for each row that
// occurs); one pass a digit, which ranks 4096 tokens a block and learns from the blocks
// before it where its digits go; zeros into the rows that do not occur; the sums;
// the joining of runs.
//
// Sums.  Sorted positions are cut into chunks of equal length, so that a token which
// occurs a hundred thousand times costs no block more than another.  A thread walks one
// chunk for V neighbouring columns, eight rows of g on their way at a time.  A run of equal
// tokens inside a chunk is written at once; the piece of a run that began before the
// chunk, and the piece of one that goes on after it, are left as float32 and joined, in order.
#include <algorithm>

#include "emb_tc.cuh"

namespace emb {
namespace {

constexpr int kDigits = 256;
constexpr int kSortThreads = 256, kSortItems = 16, kSortTile = kSortThreads * kSortItems;
constexpr int kMaxPasses = 4;
constexpr int kChunk = 64;                    // sorted positions of one thread's walk
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
  unsigned *seen;        // a bit for each row
  unsigned *key[2], *val[2];
  int passes, bits, tiles;
};

__global__ void __launch_bounds__(256) histogram_kernel(const __grid_constant__ SortArgs a) {
  __shared__ unsigned h[kMaxPasses * kDigits];
  for (int i = threadIdx.x; i < a.passes * kDigits; i += 256) h[i] = 0;
  __syncthreads();
  const unsigned mask = (1u << a.bits) - 1;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < a.t.n; i += (long long)gridDim.x * 256) {
    const long long t = token_at(a.t, i);
    if (!names_row(a.t, t)) continue;
    const unsigned k = (unsigned)t;
    for (int p = 0; p < a.passes; ++p) atomicAdd(&h[p * kDigits + ((k >> (p * a.bits)) & mask)], 1u);
    if (!((*(volatile unsigned*)(a.seen + (k >> 5)) >> (k & 31)) & 1u)) atomicOr(a.seen + (k >> 5), 1u << (k & 31));
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

// One stable pass.  Tiles are numbered as they start, so those before one are at work or
// done, and what it waits for comes; the wait is bounded all the same.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs a, int pass) {
  __shared__ unsigned count[8][kDigits], base[kDigits], sums[8];
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
  unsigned k[kSortItems], v[kSortItems], rank[kSortItems];
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
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {  // rank among the warp's equal digits, in order
    const bool ok = (in >> q) & 1u;
    const unsigned digit = ok ? (k[q] >> shift) & mask : 0xffffu;
    const unsigned same = __match_any_sync(0xffffffffu, digit);
    const unsigned below = __popc(same & ((1u << lane) - 1));
    unsigned old = 0;
    if (ok) old = count[w][digit];
    __syncwarp();
    if (ok && below == 0) count[w][digit] = old + __popc(same);
    __syncwarp();
    rank[q] = old + below;
  }
  __syncthreads();
  unsigned mine = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned c = count[j][d];
    count[j][d] = mine;
    mine += c;
  }
  unsigned* st = a.status + ((long long)pass * a.tiles + tile) * kDigits + d;
  unsigned before = 0;
  if (d <= mask) {
    *(volatile unsigned*)st = mine | (tile == 0 ? kInclusive : kAggregate);
    for (int j = tile - 1; j >= 0; --j) {
      const volatile unsigned* s = st - (long long)(tile - j) * kDigits;
      unsigned word = *s;
      for (unsigned i = 0; word < kAggregate && i < kWaitLimit; ++i) word = *s;
      if (word < kAggregate) {  // the wait ran out
        atomicOr(a.t.flags, EMB_FLAG_OP_TIMEOUT);
        break;
      }
      before += word & kCount;
      if (word >= kInclusive) break;
    }
    if (tile) *(volatile unsigned*)st = (before + mine) | kInclusive;
  }
  base[d] = first + before;
  __syncthreads();
  unsigned *ok_ = a.key[pass & 1], *ov = a.val[pass & 1];
#pragma unroll
  for (int q = 0; q < kSortItems; ++q) {
    if ((in >> q) & 1u) {
      const unsigned digit = (k[q] >> shift) & mask, to = base[digit] + count[w][digit] + rank[q];
      if (to < valid) {  // always, unless a wait ran out
        ok_[to] = k[q];
        ov[to] = v[q];
      }
    }
  }
}

// ------------------------------------------------------------------ sums

struct SumArgs {
  const unsigned *key, *val, *hist, *seen;
  const void* g;
  void* dw;
  float *head, *tail;    // [chunks][dim]
  long long ldg, ldw, vocab;
  int dim, pieces, w_t, accumulate;
  float scale;
};

__device__ __forceinline__ unsigned valid_of(const unsigned* hist) {
  __shared__ unsigned all;
  if (threadIdx.x == 0) all = 0;
  __syncthreads();
  unsigned v = threadIdx.x < kDigits ? hist[threadIdx.x] : 0;
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) atomicAdd(&all, v);
  __syncthreads();
  return all;
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
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumArgs a) {
  const unsigned n = valid_of(a.hist);
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long chunk = i / a.pieces;
  const int piece = (int)(i - chunk * a.pieces);
  if (chunk * kChunk >= n) return;
  const unsigned s = (unsigned)(chunk * kChunk), e = min(n, s + kChunk);
  unsigned cur = a.key[s];
  bool head = s > 0 && a.key[s - 1] == cur;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  float* const hp = a.head + chunk * a.dim + piece * V;
  auto flush = [&](float* to) {
#pragma unroll
    for (int j = 0; j < V; ++j) to[j] = acc[j];
  };
  for (unsigned b = s; b < e; b += 8) {
    unsigned k[8], v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const unsigned at = min(b + q, e - 1);
      k[q] = __ldg(a.key + at);
      v[q] = __ldg(a.val + at);
    }
    float x[8][V];
#pragma unroll
    for (int q = 0; q < 8; ++q) load_v<GT, V>((const GT*)a.g + v[q] * a.ldg + piece * V, x[q]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (b + q < e) {
        if (k[q] != cur) {
          if (head) flush(hp);
          else write_row<V>(a, cur, piece, acc);
          head = false;
          cur = k[q];
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += x[q][j];
      }
    }
  }
  if (head) flush(hp);
  else if (e < n && a.key[e] == cur) flush(a.tail + chunk * a.dim + piece * V);
  else write_row<V>(a, cur, piece, acc);
}

// Runs that pass a chunk's end: a block takes the one that begins in its chunk, if there
// is one.  Groups of threads add consecutive shares of its pieces, and then the shares.
template <int V>
__global__ void __launch_bounds__(256) join_runs_kernel(const __grid_constant__ SumArgs a) {
  extern __shared__ float share[];   // [groups][columns of this block]
  const unsigned n = valid_of(a.hist);
  const long long chunk = blockIdx.x;
  const long long e = (chunk + 1) * kChunk;
  if (e >= n) return;
  const unsigned cur = a.key[e];
  if (a.key[e - 1] != cur) return;                                       // no run passes the end
  if (a.key[e - kChunk] == cur && chunk > 0 && a.key[e - kChunk - 1] == cur) return;  // it began before
  // the last chunk whose first token is `cur`
  const long long chunks = (n + kChunk - 1) / kChunk;
  long long lo = chunk + 1, hi = chunks - 1;
  while (lo < hi) {
    const long long mid = (lo + hi + 1) >> 1;
    if (a.key[mid * kChunk] == cur) lo = mid;
    else hi = mid - 1;
  }
  const int last = (int)lo, heads = last - (int)chunk;
  for (int p0 = 0; p0 < a.pieces; p0 += 256) {
    const int width = min(256, a.pieces - p0), groups = min(256 / width, heads), g = threadIdx.x / width, piece = p0 + threadIdx.x % width;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    if (g < groups) {
      const int from = (int)chunk + 1 + (int)((long long)heads * g / groups), to = (int)chunk + 1 + (int)((long long)heads * (g + 1) / groups);
      if (g == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = a.tail[chunk * a.dim + piece * V + j];
      }
#pragma unroll 8
      for (int c = from; c < to; ++c) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += a.head[(long long)c * a.dim + piece * V + j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) share[(g * width + threadIdx.x % width) * V + j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < width) {
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.0f;
      for (int q = 0; q < groups; ++q)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += share[(q * width + threadIdx.x) * V + j];
      write_row<V>(a, cur, piece, acc);
    }
    __syncthreads();
  }
}

// Zeros into the rows that no token names.
template <int V>
__global__ void __launch_bounds__(256) zero_rows_kernel(const __grid_constant__ SumArgs a) {
  const long long total = a.vocab * a.pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long row = total <= 0xffffffffLL ? (unsigned)i / (unsigned)a.pieces : i / a.pieces;
    const long long e = row * a.ldw + (i - row * a.pieces) * V;
    if ((__ldg(a.seen + (row >> 5)) >> (row & 31)) & 1u) continue;
    float z[V];
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = 0.0f;
    if (a.w_t == EMB_T_F32) store_v<float, V>((float*)a.dw + e, z);
    else if (a.w_t == EMB_T_BF16) store_v<__nv_bfloat16, V>((__nv_bfloat16*)a.dw + e, z);
    else store_v<__half, V>((__half*)a.dw + e, z);
  }
}

// ------------------------------------------------------------------ host side

struct TokenPlan {
  int passes = 0, bits = 0, tiles = 0;
  long long chunks = 0;
  size_t zero_bytes = 0;  // hist, next, status, seen, from the start on
  size_t next = 0, status = 0, seen = 0, key[2] = {}, val[2] = {}, head = 0, tail = 0, bytes = 0;
};

TokenPlan plan_tokens(long long n, long long vocab, long long dim) {
  TokenPlan pl;
  if (n == 0 || vocab == 0 || dim == 0) return pl;
  int bits = 1;
  while (bits < 31 && (vocab - 1) >> bits) ++bits;
  pl.passes = (bits + 7) / 8;
  pl.bits = (bits + pl.passes - 1) / pl.passes;
  pl.tiles = (int)((n + kSortTile - 1) / kSortTile);
  pl.chunks = (n + kChunk - 1) / kChunk;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  pl.next = kMaxPasses * kDigits * 4;
  pl.status = pl.next + 256;
  pl.seen = pl.status + (size_t)pl.passes * pl.tiles * kDigits * 4;
  pl.zero_bytes = pl.seen + up((size_t)(vocab + 31) / 32 * 4);
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
  const long long blocks = (chunks * a.pieces + 255) / 256;
  sum_kernel<GT, V><<<(unsigned)blocks, 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (chunks > 1) join_runs_kernel<V><<<(unsigned)(chunks - 1), 256, 256 * V * 4, st>>>(a);
  return cudaGetLastError();
}
template <int V>
cudaError_t launch_grad(const SumArgs& a, emb_ftype g_t, long long chunks, cudaStream_t st) {
  if (!a.accumulate) {
    const int grid = (int)std::min<long long>((a.vocab * a.pieces + 255) / 256, 32LL * sm_count());
    zero_rows_kernel<V><<<grid, 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (g_t == EMB_T_F32) return launch_sums<float, V>(a, chunks, st);
  if (g_t == EMB_T_BF16) return launch_sums<__nv_bfloat16, V>(a, chunks, st);
  return launch_sums<__half, V>(a, chunks, st);
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
             (unsigned*)ws, (unsigned*)(ws + pl.next), (unsigned*)(ws + pl.status), (unsigned*)(ws + pl.seen), {}, {}, pl.passes, pl.bits, pl.tiles};
  for (int j = 0; j < 2; ++j) {
    s.key[j] = (unsigned*)(ws + pl.key[j]);
    s.val[j] = (unsigned*)(ws + pl.val[j]);
  }
  EMB_CUDA(cudaMemsetAsync(ws, 0, pl.zero_bytes, st));
  histogram_kernel<<<(int)std::min<long long>((n + 2047) / 2048, 4LL * sm_count()), 256, 0, st>>>(s);
  EMB_CUDA(cudaGetLastError());
  for (int p = 0; p < pl.passes; ++p) {
    if (p == 0) sort_kernel<true><<<pl.tiles, kSortThreads, 0, st>>>(s, p);
    else sort_kernel<false><<<pl.tiles, kSortThreads, 0, st>>>(s, p);
    EMB_CUDA(cudaGetLastError());
  }
  const int end = (pl.passes - 1) & 1;
  const SumArgs a{s.key[end], s.val[end], s.hist, s.seen, grad_d, dweight_d, (float*)(ws + pl.head), (float*)(ws + pl.tail),
                  ldg, ldw, vocab, (int)dim, (int)dim / v, weight_t, accumulate != 0, scale};
  const cudaError_t e = v == 8 ? launch_grad<8>(a, grad_t, pl.chunks, st) : v == 4 ? launch_grad<4>(a, grad_t, pl.chunks, st)
                                                                                   : launch_grad<1>(a, grad_t, pl.chunks, st);
  if (e != cudaSuccess) return cuda_fail(e, "emb_token_bwd launch");
  return EMB_OK;
}
