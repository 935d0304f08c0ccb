// 8-bit quantiser: codes and block scales of a matrix and of its transpose.
//
// Bound by memory: x in once, one byte an element out per orientation.  A block
// of 512 threads takes one tile of 128 x 128: warp w holds rows 8w..8w+7, a
// lane four neighbouring columns of each, so a warp reads and writes whole
// 128-element row pieces.  The tile stays in registers while the largest
// magnitudes of its rows (warp reductions), its columns (in shared memory over
// the warps) or all of it are found; the transposed codes go through shared
// memory so that they leave as whole rows too.  In a loop, 65,536 x 3200 float32:
// 159 us one way (0.97 of the measured copy rate), 222 both ways (0.84; 254 with 256
// threads a tile); 131,072 x 1024 bf16 87 and 135.  Rows off the vectors' alignment
// go element by element: 65,536 x 1003 float32 68 and 94 (0.72 and 0.62).
#include <algorithm>

#include "emb_dense.cuh"

namespace emb {
namespace {

constexpr int kTile = EMB_FP8_BLOCK;
constexpr int kWarps = 16, kRows = kTile / kWarps;  // rows of a warp

struct QuantArgs {
  const void* x;
  unsigned char *q, *qt;
  float *s, *st;
  long long rows, cols, ldx, ldq, ldqt;
  long long col_tiles;
  long long srow, strow;  // scales in a row of s and of st
  int vec;
};

__device__ __forceinline__ unsigned amax_bits(float a) { return __reduce_max_sync(0xffffffffu, __float_as_uint(a)); }

// Four neighbouring elements as they lie in memory.
template <typename T>
struct Raw4 {
  uint2 v;
  __device__ __forceinline__ void load(const T* p) { v = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float* o) const;
};
template <>
struct Raw4<float> {
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
__device__ __forceinline__ void Raw4<__half>::get(float* o) const {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  o[0] = a.x;
  o[1] = a.y;
  o[2] = b.x;
  o[3] = b.y;
}
template <>
__device__ __forceinline__ void Raw4<__nv_bfloat16>::get(float* o) const {
  o[0] = __uint_as_float(v.x << 16);
  o[1] = __uint_as_float(v.x & 0xffff0000u);
  o[2] = __uint_as_float(v.y << 16);
  o[3] = __uint_as_float(v.y & 0xffff0000u);
}

template <typename T, bool SQUARE>
__global__ void __launch_bounds__(kWarps * 32, 2) quantize_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ __align__(16) unsigned char tile_t[kTile * kTile];  // transposed codes, swizzled
  __shared__ __align__(16) float part[kWarps][kTile];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long tr = blockIdx.x / a.col_tiles, tc = blockIdx.x % a.col_tiles;
  const long long r0 = tr * kTile + w * kRows, c0 = tc * kTile + lane * 4;
  const T* x = (const T*)a.x;
  float v[kRows][4];
  if (a.vec && r0 + kRows <= a.rows && c0 + 4 <= a.cols) {
    // all loads first: a conversion between them would wait for each in turn (bf16 131,072 x 1024: 222 us)
    Raw4<T> raw[kRows];
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
  // The largest magnitude of each row's four, from 0 on: fmaxf passes NaN over
  // beside a number, but of four NaN it makes NaN, whose bits would win the warp's
  // maximum.  A thread that meets an infinity makes its infinities NaN first (e4m3
  // has none) and takes the maxima again.
  float top[kRows];
  auto maxima = [&] {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      top[i] = fmaxf(fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3]))), 0.0f);
      m = fmaxf(m, top[i]);
    }
    return m;
  };
  float m = maxima();
  if (m > kFltMax) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!finite_f32(v[i][k])) v[i][k] = __uint_as_float(0x7fc00000u);
    m = maxima();
  }
  float tile_amax = 0.0f;
  if (SQUARE) {
    m = __uint_as_float(amax_bits(m));
    if (lane == 0) part[0][w] = m;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kWarps; ++j) tile_amax = fmaxf(tile_amax, part[0][j]);
    tile_amax = fmaxf(tile_amax, kAmaxFloor);
    if (threadIdx.x == 0) {
      if (a.s) a.s[tc * a.srow + tr] = scale_of(tile_amax);
      if (a.st) a.st[tr * a.strow + tc] = scale_of(tile_amax);
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = r0 + i;
      float amax = tile_amax;
      if (!SQUARE) {
        amax = fmaxf(__uint_as_float(amax_bits(top[i])), kAmaxFloor);
        if (lane == 0 && r < a.rows) a.s[tc * a.srow + r] = scale_of(amax);
      }
      const float inv = inv_of(amax);
      const unsigned c = e4m3x2(__fmul_rn(v[i][0], inv), __fmul_rn(v[i][1], inv)) |
                         (e4m3x2(__fmul_rn(v[i][2], inv), __fmul_rn(v[i][3], inv)) << 16);
      // columns past the last one are zeros up to the row's next 16 bytes
      if (r < a.rows && c0 < ((a.cols + 15) & ~15LL)) *reinterpret_cast<unsigned*>(a.q + r * a.ldq + c0) = c;
    }
  }
  if (a.qt) {
    float inv[4];
    if (SQUARE) {
#pragma unroll
      for (int k = 0; k < 4; ++k) inv[k] = inv_of(tile_amax);
    } else {
      float top_c[4] = {};
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) top_c[k] = fmaxf(top_c[k], fabsf(v[i][k]));
      *reinterpret_cast<float4*>(&part[w][lane * 4]) = make_float4(top_c[0], top_c[1], top_c[2], top_c[3]);
      __syncthreads();
      float4 m4 = make_float4(kAmaxFloor, kAmaxFloor, kAmaxFloor, kAmaxFloor);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float4 o = *reinterpret_cast<const float4*>(&part[j][lane * 4]);
        m4 = make_float4(fmaxf(m4.x, o.x), fmaxf(m4.y, o.y), fmaxf(m4.z, o.z), fmaxf(m4.w, o.w));
      }
      const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        inv[k] = inv_of(m[k]);
        if (w == 0 && c0 + k < a.cols) a.st[tr * a.strow + c0 + k] = scale_of(m[k]);
      }
    }
    // A lane's column k holds eight codes of the transposed row 4 lane + k, at
    // eight-byte piece w.  Piece p of row c lies at p ^ (c / 4 mod 16): a warp's
    // stores meet no bank twice, and two pieces that make up sixteen bytes stay
    // together, swapped where that number is odd.
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      unsigned c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        c[j] = e4m3x2(__fmul_rn(v[4 * j][k], inv[k]), __fmul_rn(v[4 * j + 1][k], inv[k])) |
               (e4m3x2(__fmul_rn(v[4 * j + 2][k], inv[k]), __fmul_rn(v[4 * j + 3][k], inv[k])) << 16);
      *reinterpret_cast<uint2*>(tile_t + (lane * 4 + k) * kTile + ((w ^ (lane & 15)) << 3)) = make_uint2(c[0], c[1]);
    }
    __syncthreads();
    const long long row_end = (a.rows + 15) & ~15LL;
#pragma unroll
    for (int j = 0; j < kTile * 8 / (kWarps * 32); ++j) {
      const int at = j * kWarps * 32 + threadIdx.x;  // 16-byte chunk of the tile: 8 to a transposed row
      const int c = at >> 3, chunk = at & 7, x = (c >> 2) & 15;
      const long long col = tc * kTile + c, row = tr * kTile + chunk * 16;
      if (col < a.cols && row < row_end) {
        const uint4 o = *reinterpret_cast<const uint4*>(tile_t + c * kTile + ((chunk ^ (x >> 1)) << 4));
        *reinterpret_cast<uint4*>(a.qt + col * a.ldqt + row) = x & 1 ? make_uint4(o.z, o.w, o.x, o.y) : o;
      }
    }
  }
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_fp8_quantize(const void* x_d, emb_ftype x_t, int64_t rows, int64_t cols, int64_t ldx,
                                       int32_t block_rows, void* q_d, int64_t ldq, float* s_d, void* qt_d, int64_t ldqt,
                                       float* st_d, void* stream) {
  if (!good_ftype(x_t)) return fail(EMB_ERR_INVALID_ARG, "bad element type");
  if (rows < 0 || cols < 0) return fail(EMB_ERR_INVALID_ARG, "negative rows or cols");
  if (block_rows != 1 && block_rows != EMB_FP8_BLOCK) return fail(EMB_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (rows == 0 || cols == 0) return EMB_OK;
  if (!q_d && !qt_d) return fail(EMB_ERR_INVALID_ARG, "q and qt are NULL");
  if ((q_d && !s_d) || (qt_d && !st_d)) return fail(EMB_ERR_INVALID_ARG, "codes need their scales");
  if (ldx < cols) return fail(EMB_ERR_INVALID_ARG, "ldx below cols");
  if ((q_d && (ldq < cols || ldq % 16)) || (qt_d && (ldqt < rows || ldqt % 16)))
    return fail(EMB_ERR_INVALID_ARG, "a row of codes must be a multiple of 16 bytes and hold the row");
  if (!aligned_to(q_d, 16) || !aligned_to(qt_d, 16)) return fail(EMB_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (!aligned_to(x_d, ftype_bytes(x_t)) || !aligned_to(s_d, 4) || !aligned_to(st_d, 4))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (!x_d) return fail(EMB_ERR_INVALID_ARG, "x is NULL");
  const int64_t rt = (rows - 1) / kTile + 1, ct = (cols - 1) / kTile + 1;
  if (rt > 0x7fffffffLL / ct) return fail(EMB_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles");
  const bool square = block_rows != 1;
  const int vec = ldx % 4 == 0 && aligned_to(x_d, 4 * ftype_bytes(x_t));
  const QuantArgs a{x_d, (unsigned char*)q_d, (unsigned char*)qt_d, q_d ? s_d : nullptr, qt_d ? st_d : nullptr, rows, cols,
                    ldx, ldq, ldqt, ct, square ? rt : rows, square ? ct : cols, vec};
  const int grid = (int)(rt * ct);
  cudaStream_t st = (cudaStream_t)stream;
#define EMB_QUANT(T)                                                        \
  do {                                                                      \
    if (square) quantize_kernel<T, true><<<grid, kWarps * 32, 0, st>>>(a);          \
    else quantize_kernel<T, false><<<grid, kWarps * 32, 0, st>>>(a);                \
  } while (0)
  if (x_t == EMB_T_F32) EMB_QUANT(float);
  else if (x_t == EMB_T_BF16) EMB_QUANT(__nv_bfloat16);
  else EMB_QUANT(__half);
#undef EMB_QUANT
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "quantize_kernel launch");
  return EMB_OK;
}
