// 4-bit quantiser and reading back (microscaled e2m1: 32 neighbouring elements
// share one power of two, stored as its exponent).
//
// With A the block's largest magnitude, E = floor(log2 A) - 2 puts A in [4, 8);
// 6 is the largest code.  x 2^-E is exact (or a denormal far below the smallest
// code's half), so the only rounding is the one to the nearest code.
//
// Bound by memory: x in once, half a byte an element out per orientation.  As in the
// 8-bit quantiser a block of 512 threads holds a tile of 128 x 128 in registers, warp
// w rows 8w..8w+7, a lane four neighbouring columns of each: the maxima of 32 columns
// are taken over eight lanes, those of 32 rows over four warps.  A row of codes of the
// tile is 64 bytes: eight rows' pieces are exchanged among eight lanes, so that each
// lane stores 16 bytes at once; the transposed codes go through shared memory.  The
// scales of a tile are 512 neighbouring bytes, in the order in which the tensor cores
// read them.  65,536 x 3200 float32 both ways: 197 us, 0.80 of the measured copy rate.
#include <algorithm>

#include "emb_dense.cuh"

namespace emb {
namespace {

constexpr int kTile = 128;
constexpr long long kMaxSide = 0x7fff0000LL;
constexpr int kWarps = 16, kRows = kTile / kWarps;  // rows of a warp

struct Quant4Args {
  const void* x;
  unsigned char *q, *s, *qt, *st;
  long long rows, cols, ldx, ldq, ldqt;
  long long row_tiles, col_tiles;
  int vec;
};

// Four neighbouring elements as they lie in memory.
template <typename T>
struct Piece4 {
  uint2 v;
  __device__ __forceinline__ void load(const T* p) { v = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float* o) const;
};
template <>
struct Piece4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = v.x;
    o[1] = v.y;
    o[2] = v.z;
    o[3] = v.w;
  }
};
template <>
__device__ __forceinline__ void Piece4<__half>::get(float* o) const {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  o[0] = a.x;
  o[1] = a.y;
  o[2] = b.x;
  o[3] = b.y;
}
template <>
__device__ __forceinline__ void Piece4<__nv_bfloat16>::get(float* o) const {
  o[0] = __uint_as_float(v.x << 16);
  o[1] = __uint_as_float(v.x & 0xffff0000u);
  o[2] = __uint_as_float(v.y << 16);
  o[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The scale byte of a block from the bits of its largest magnitude: the exponent less
// 2, not below 2^-127; 255 (NaN) where a value is not finite (its bits are then the largest).
__device__ __forceinline__ unsigned scale_byte(unsigned amax_bits) {
  return amax_bits >= 0x7f800000u ? 255u : (unsigned)max((int)(amax_bits >> 23) - 2, 0);
}
// 2^-E of a scale byte: 2^(127 - byte).  A byte of 255 gives 0: its codes mean nothing.
__device__ __forceinline__ float inverse_of(unsigned byte) { return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23); }
// 2^E of a scale byte; 2^-127 is a denormal number.
__device__ __forceinline__ float power_of(unsigned byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}
// Four values as e2m1 codes, to nearest (ties to even), 6 beyond it: the first in the low nibble.
__device__ __forceinline__ unsigned e2m1x4(const float* v, float inv) {
  unsigned r;
  asm("{\n.reg .b8 lo, hi;\n"
      "cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n"
      "mov.b32 %0, {lo, hi, 0, 0};\n}\n"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv));
  return r;
}

// Where a scale lies within its tile's 512 bytes: row r, block b (of four) of the tile.
__device__ __forceinline__ int scale_at(int r, int b) { return (r & 31) * 16 + (r >> 5) * 4 + b; }

template <typename T, bool SQUARE>
__global__ void __launch_bounds__(kWarps * 32, 2) quantize4_kernel(const __grid_constant__ Quant4Args a) {
  __shared__ __align__(16) unsigned tile_t[kTile * 16];    // transposed codes, swizzled: 16 words to a transposed row
  __shared__ __align__(16) unsigned part[kWarps][kTile];   // maxima of a warp's eight rows
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long tr = blockIdx.x / a.col_tiles, tc = blockIdx.x % a.col_tiles;
  const long long r0 = tr * kTile + w * kRows, c0 = tc * kTile + lane * 4;
  const T* x = (const T*)a.x;
  float v[kRows][4];
  if (a.vec && r0 + kRows <= a.rows && c0 + 4 <= a.cols) {
    Piece4<T> raw[kRows];  // all loads before any conversion
#pragma unroll
    for (int i = 0; i < kRows; ++i) raw[i].load(x + (r0 + i) * a.ldx + c0);
#pragma unroll
    for (int i = 0; i < kRows; ++i) raw[i].get(v[i]);
  } else {
    T raw[kRows][4];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        raw[i][k] = from_f32<T>(0.0f);
        if (r0 + i < a.rows && c0 + k < a.cols) raw[i][k] = x[(r0 + i) * a.ldx + c0 + k];
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = to_f32<T>(raw[i][k]);
  }
  // Magnitudes are compared by their bits: infinities and NaN are then the largest.
  auto bits = [](float f) { return __float_as_uint(f) & 0x7fffffffu; };
  unsigned square = 0;  // SQUARE: the scale byte of this lane's 32 x 32 block
  if (SQUARE) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) m = max(m, bits(v[i][k]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane % 8 == 0) part[w][lane / 8] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, part[(w & ~3) + j][lane / 8]);
    square = scale_byte(m);
  }
  if (a.q) {
    unsigned code[kRows], byte[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (SQUARE) {
        byte[i] = square;
      } else {
        unsigned m = max(max(bits(v[i][0]), bits(v[i][1])), max(bits(v[i][2]), bits(v[i][3])));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        byte[i] = scale_byte(m);
      }
      code[i] = e2m1x4(v[i], inverse_of(byte[i]));
    }
    // Lane 8b + j of block b's eight lanes keeps row j's scale and, of the codes, row j's 16 bytes.
    const int j = lane & 7;
    unsigned mine = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) mine = i == j ? byte[i] : mine;
    const int r = w * kRows + j;
    const bool inside = tr * kTile + r < a.rows && tc * kTile + (lane & ~7) * 4 < a.cols;
    a.s[blockIdx.x * 512LL + scale_at(r, lane >> 3)] = inside ? (unsigned char)mine : 0;
    // rows (2i, 2i + 1) between neighbours: a word each; then pairs of words, then four
    unsigned w1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned keep = j & 1 ? code[2 * i + 1] : code[2 * i], give = j & 1 ? code[2 * i] : code[2 * i + 1];
      const unsigned got = __shfl_xor_sync(0xffffffffu, give, 1);
      w1[i] = j & 1 ? got | (keep << 16) : keep | (got << 16);
    }
    uint2 w2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const unsigned keep = j & 2 ? w1[2 * i + 1] : w1[2 * i], give = j & 2 ? w1[2 * i] : w1[2 * i + 1];
      const unsigned got = __shfl_xor_sync(0xffffffffu, give, 2);
      w2[i] = j & 2 ? make_uint2(got, keep) : make_uint2(keep, got);
    }
    const uint2 keep = j & 4 ? w2[1] : w2[0], give = j & 4 ? w2[0] : w2[1];
    const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, give.x, 4), __shfl_xor_sync(0xffffffffu, give.y, 4));
    const uint4 o = j & 4 ? make_uint4(got.x, got.y, keep.x, keep.y) : make_uint4(keep.x, keep.y, got.x, got.y);
    // columns past the last one are zeros up to the row's next 16 bytes
    if (inside) *reinterpret_cast<uint4*>(a.q + (tr * kTile + r) * a.ldq + tc * (kTile / 2) + (lane >> 3) * 16) = o;
  }
  if (a.qt) {
    unsigned byte[4];
    unsigned char* st = a.st + (tc * a.row_tiles + tr) * 512;
    if (SQUARE) {
#pragma unroll
      for (int k = 0; k < 4; ++k) byte[k] = square;
    } else {
      uint4 top = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        top.x = max(top.x, bits(v[i][0]));
        top.y = max(top.y, bits(v[i][1]));
        top.z = max(top.z, bits(v[i][2]));
        top.w = max(top.w, bits(v[i][3]));
      }
      *reinterpret_cast<uint4*>(&part[w][lane * 4]) = top;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 o = *reinterpret_cast<const uint4*>(&part[(w & ~3) + j][lane * 4]);
        top = make_uint4(max(top.x, o.x), max(top.y, o.y), max(top.z, o.z), max(top.w, o.w));
      }
      byte[0] = scale_byte(top.x);
      byte[1] = scale_byte(top.y);
      byte[2] = scale_byte(top.z);
      byte[3] = scale_byte(top.w);
    }
    // A lane's column k holds eight codes, word w, of the transposed row 4 lane + k,
    // kept as row k * 32 + lane.  Word w lies at w ^ (lane / 2): a warp's stores meet
    // every bank once.
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float inv = inverse_of(byte[k]);
      const float lo[4] = {v[0][k], v[1][k], v[2][k], v[3][k]}, hi[4] = {v[4][k], v[5][k], v[6][k], v[7][k]};
      tile_t[(k * 32 + lane) * 16 + (w ^ (lane >> 1))] = e2m1x4(lo, inv) | (e2m1x4(hi, inv) << 16);
      if ((w & 3) == 0) {  // block w / 4 of the transposed row
        const bool inside = c0 + k < a.cols && tr * kTile + w * kRows < a.rows;
        st[scale_at(lane * 4 + k, w >> 2)] = inside ? (unsigned char)byte[k] : 0;
      }
    }
    __syncthreads();
    const int at = threadIdx.x >> 2, chunk = threadIdx.x & 3;  // 16 bytes of a transposed row
    // four threads to a row, rows in order: row c = 4 l + k is kept at k * 32 + l
    const int l = at >> 2, x4 = l >> 1;
    const long long col = tc * kTile + at, row = tr * kTile + chunk * 32;
    if (col < a.cols && row < a.rows) {
      const uint4 o = *reinterpret_cast<const uint4*>(&tile_t[((at & 3) * 32 + l) * 16 + ((chunk ^ (x4 >> 2)) << 2)]);
      uint4 u = x4 & 1 ? make_uint4(o.y, o.x, o.w, o.z) : o;
      if (x4 & 2) u = make_uint4(u.z, u.w, u.x, u.y);
      *reinterpret_cast<uint4*>(a.qt + col * a.ldqt + row / 2) = u;
    }
  }
}

// ------------------------------------------------------------------ reading back

struct Back4Args {
  const unsigned char *q, *s;
  void* out;
  long long rows, cols, ldq, ldo, col_tiles;
  unsigned pieces;  // of sixteen codes, in a row
  int vec;
};

// A thread turns sixteen neighbouring codes (eight bytes) into values: 32 or 64 bytes.
// Bound by the stores; 65,536 x 3200 to bf16: 90 us, and 120 with eight codes a thread.
template <typename T>
__global__ void __launch_bounds__(256) dequantize4_kernel(const __grid_constant__ Back4Args a) {
  const long long total = a.rows * a.pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long row = total <= 0xffffffffLL ? (unsigned)i / a.pieces : i / a.pieces;
    const long long col = (i - row * a.pieces) * 16;
    const int b = (int)(col >> 5);
    const uint2 code = __ldcs(reinterpret_cast<const uint2*>(a.q + row * a.ldq + col / 2));
    const float p = power_of(__ldg(a.s + ((row >> 7) * a.col_tiles + (b >> 2)) * 512 + scale_at((int)(row & 127), b & 3)));
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      unsigned h;
      asm("{\n.reg .b8 c;\nmov.b32 {c, _, _, _}, %1;\ncvt.rn.f16x2.e2m1x2 %0, c;\n}\n" : "=r"(h) : "r"((j < 4 ? code.x : code.y) >> (8 * (j & 3))));
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
      v[2 * j] = f.x * p;
      v[2 * j + 1] = f.y * p;
    }
    T* dst = (T*)a.out + row * a.ldo + col;
    if (a.vec && col + 16 <= a.cols) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Raw8<T> r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.set2(j, v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
        r.store(dst + 8 * k);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < a.cols) dst[j] = from_f32<T>(v[j]);
    }
  }
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_fp4_quantize(const void* x_d, emb_ftype x_t, int64_t rows, int64_t cols, int64_t ldx,
                                       int32_t block_rows, void* q_d, int64_t ldq, void* s_d, void* qt_d, int64_t ldqt,
                                       void* st_d, void* stream) {
  if (!good_ftype(x_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  if (rows < 0 || cols < 0) return fail(EMB_ERR_INVALID_ARG, "negative rows or cols");
  if (block_rows != 1 && block_rows != EMB_FP4_BLOCK) return fail(EMB_ERR_INVALID_ARG, "block_rows must be 1 or 32");
  if (rows == 0 || cols == 0) return EMB_OK;
  if (!q_d && !qt_d) return fail(EMB_ERR_INVALID_ARG, "q and qt are NULL");
  if ((q_d && !s_d) || (qt_d && !st_d)) return fail(EMB_ERR_INVALID_ARG, "codes need their scales");
  if (ldx < cols) return fail(EMB_ERR_INVALID_ARG, "ldx below cols");
  if ((q_d && (ldq < (cols - 1) / 2 + 1 || ldq % 16)) || (qt_d && (ldqt < (rows - 1) / 2 + 1 || ldqt % 16)))
    return fail(EMB_ERR_INVALID_ARG, "a row of codes must be a multiple of 16 bytes and hold the row");
  if (!aligned_to(q_d, 16) || !aligned_to(qt_d, 16)) return fail(EMB_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (!aligned_to(x_d, ftype_bytes(x_t))) return fail(EMB_ERR_INVALID_ARG, "x is not aligned to its elements");
  if (!x_d) return fail(EMB_ERR_INVALID_ARG, "x is NULL");
  const int64_t rt = (rows - 1) / kTile + 1, ct = (cols - 1) / kTile + 1;
  if (rows > kMaxSide || cols > kMaxSide) return fail(EMB_ERR_UNSUPPORTED, "rows or cols above 2^31 - 65536");
  if (rt > 0x7fffffffLL / ct) return fail(EMB_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  const int vec = ldx % 4 == 0 && aligned_to(x_d, 4 * ftype_bytes(x_t));
  const Quant4Args a{x_d, (unsigned char*)q_d, (unsigned char*)s_d, (unsigned char*)qt_d, (unsigned char*)st_d,
                     rows, cols, ldx, ldq, ldqt, rt, ct, vec};
  const int grid = (int)(rt * ct);
  cudaStream_t st = (cudaStream_t)stream;
#define EMB_QUANT(T)                                                                \
  do {                                                                              \
    if (block_rows != 1) quantize4_kernel<T, true><<<grid, kWarps * 32, 0, st>>>(a); \
    else quantize4_kernel<T, false><<<grid, kWarps * 32, 0, st>>>(a);                \
  } while (0)
  if (x_t == EMB_T_F32) EMB_QUANT(float);
  else if (x_t == EMB_T_BF16) EMB_QUANT(__nv_bfloat16);
  else EMB_QUANT(__half);
#undef EMB_QUANT
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "quantize4_kernel launch");
  return EMB_OK;
}

extern "C" emb_status emb_fp4_dequantize(const void* q_d, int64_t ldq, const void* s_d, int64_t rows, int64_t cols,
                                         void* out_d, emb_ftype out_t, int64_t ldo, void* stream) {
  if (!good_ftype(out_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  if (rows < 0 || cols < 0) return fail(EMB_ERR_INVALID_ARG, "negative rows or cols");
  if (rows == 0 || cols == 0) return EMB_OK;
  if (!q_d || !s_d || !out_d) return fail(EMB_ERR_INVALID_ARG, "q, s or out is NULL");
  if (ldq < (cols - 1) / 2 + 1 || ldq % 16) return fail(EMB_ERR_INVALID_ARG, "a row of codes must be a multiple of 16 bytes and hold the row");
  if (!aligned_to(q_d, 16)) return fail(EMB_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (ldo < cols) return fail(EMB_ERR_INVALID_ARG, "ldo below cols");
  if (!aligned_to(out_d, ftype_bytes(out_t))) return fail(EMB_ERR_INVALID_ARG, "out is not aligned to its elements");
  const int64_t rt = (rows - 1) / kTile + 1, ct = (cols - 1) / kTile + 1;
  if (rows > kMaxSide || cols > kMaxSide) return fail(EMB_ERR_UNSUPPORTED, "rows or cols above 2^31 - 65536");
  if (rt > 0x7fffffffLL / ct) return fail(EMB_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  const int64_t pieces = (cols + 15) / 16;
  const size_t wide = 8 * ftype_bytes(out_t);
  const Back4Args a{(const unsigned char*)q_d, (const unsigned char*)s_d, out_d, rows, cols, ldq, ldo, ct, (unsigned)pieces,
                    aligned_to(out_d, wide) && ldo * ftype_bytes(out_t) % wide == 0};
  const int grid = (int)std::min<int64_t>((rows * pieces + 255) / 256, 64LL * sm_count());
  cudaStream_t st = (cudaStream_t)stream;
  if (out_t == EMB_T_F32) dequantize4_kernel<float><<<grid, 256, 0, st>>>(a);
  else if (out_t == EMB_T_BF16) dequantize4_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else dequantize4_kernel<__half><<<grid, 256, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "dequantize4_kernel launch");
  return EMB_OK;
}
