// What the tiled products share (emb_fp8_matmul.cu, emb_fp4_matmul.cu): how tiles are
// cut into steps and dealt to the blocks, how a tile's sums leave the registers, the
// joining of tiles that several blocks computed, tensor maps.
//
// P, a kernel's arguments, has: out, ldo, bias, m, n; m_tiles, n_tiles, k_blocks (steps of
// a tile); steps (of all); per_cta (steps a block takes; 0: whole tiles, block-stride);
// partial (float32 tiles, one for each piece).  A tile is kBM x BN; of the eight warps
// that hold its sums, warp w has rows 32 (w % 4).. and columns BN/2 * (w / 4)..., a row a lane.
#pragma once

#include "emb_tc.cuh"

namespace emb {

constexpr int kBM = 128;     // rows of a tile
constexpr int kSumWarps = 8; // warps that hold a tile's sums

struct Unit {  // consecutive steps of one tile
  int tm, tn, kb0, kb1;
  long long tile;
};

// Tiles in groups of 16 rows of tiles, column by column within a group: the
// blocks at work at one time then share few slabs of a and b in L2.
template <class P>
__device__ __forceinline__ void tile_at(const P& p, long long t, int* tm, int* tn) {
  constexpr int kGroup = 16;
  const long long per_group = (long long)kGroup * p.n_tiles;
  const int g = (int)(t / per_group);
  const int in = (int)(t - g * per_group);
  const int rows = min(kGroup, p.m_tiles - g * kGroup);
  *tm = g * kGroup + in % rows;
  *tn = in / rows;
}

// A worker's (a block's, or a pair's) next unit from its position: a tile number, or a step.
template <class P>
__device__ __forceinline__ bool next_unit(const P& p, long long* pos, long long end, Unit* u, int workers) {
  if (*pos >= end) return false;
  if (p.per_cta == 0) {
    u->tile = *pos;
    u->kb0 = 0;
    u->kb1 = p.k_blocks;
    *pos += workers;
  } else {
    u->tile = *pos / p.k_blocks;
    u->kb0 = (int)(*pos - u->tile * p.k_blocks);
    u->kb1 = (int)min((long long)p.k_blocks, u->kb0 + (end - *pos));
    *pos += u->kb1 - u->kb0;
  }
  tile_at(p, u->tile, &u->tm, &u->tn);
  return true;
}
template <class P>
__device__ __forceinline__ void my_range(const P& p, long long* pos, long long* end, int worker) {
  if (p.per_cta == 0) {
    *pos = worker;
    *end = (long long)p.m_tiles * p.n_tiles;
  } else {
    *pos = worker * p.per_cta;
    *end = min(p.steps, *pos + p.per_cta);
  }
}

// A unit's sums, from the registers of this lane (`acc`: row `row`, columns col0..), to
// the output, or to the workspace where the tile has other pieces.  WIDE: rows of out
// are aligned to 32 bytes; else `stage` is this warp's 32 x 17 floats of shared memory.  BLOCKS:
// of a worker (a pair has two tiles of 128 rows, one below the other).
template <int BN, typename OT, bool WIDE, int BLOCKS = 1, class P>
__device__ __forceinline__ void store_unit(const P& p, const Unit& u, int warp, int lane, int row, int col0, float* acc, float* stage) {
  constexpr int kHalf = BN / 2;
  if (u.kb0 == 0 && u.kb1 == p.k_blocks) {
    if constexpr (WIDE) {
      if (row < p.m) {
        OT* dst = (OT*)p.out + row * p.ldo + col0;
        constexpr int kVec = 32 / sizeof(OT);
#pragma unroll
        for (int c = 0; c < kHalf; c += kVec) {
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
      // (the 8-bit product of 10,046 x 1293 x 475 to f16: 155 us with a row to a lane, 61 so; 39 by now)
#pragma unroll
      for (int c = 0; c < kHalf; c += 16) {
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
  } else if (row < p.m) {  // part of a tile: slot (worker + tile) is this piece's alone
    float* dst = p.partial + ((blockIdx.x / BLOCKS + u.tile) * BLOCKS + blockIdx.x % BLOCKS) * kBM * BN + (warp * kHalf * 4 + lane) * 8;
#pragma unroll
    for (int c = 0; c < kHalf; c += 8) store32<float>(dst + c * 32, acc + c);
  }
}

// Adds the pieces of each tile that several blocks computed, in k order.  A piece
// lies as the warps store it, whole kilobytes at a time: by warps, by 8 columns, by
// rows (the 8-bit product of 1664 x 452 x 30,584 to bf16: 52 us, and 56 with pieces laid
// out by rows).  One block takes 32 rows x 32 columns, four columns a thread.
template <int BN, typename OT, class P, int BLOCKS = 1>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ P p) {
  constexpr int kBlocks = kBM * BN / 1024, kHalf = BN / 2, kWarpBlocks = kHalf / 32;
  const long long sub = blockIdx.x / kBlocks, tile = sub / BLOCKS;
  const int q = (int)(blockIdx.x % kBlocks), warp = q / kWarpBlocks, x = threadIdx.x / 8, y = threadIdx.x % 8;
  const long long first = tile * p.k_blocks / p.per_cta, last = ((tile + 1) * p.k_blocks - 1) / p.per_cta;
  if (first == last) return;  // one block had it whole
  int tm, tn;
  tile_at(p, tile, &tm, &tn);
  const int row = (int)(tm * BLOCKS + sub % BLOCKS) * kBM + (warp & 3) * 32 + x, col = tn * BN + (warp >> 2) * kHalf + q % kWarpBlocks * 32 + y * 4;
  if (row >= p.m || col >= p.n) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* src = p.partial + ((first + tile) * BLOCKS + sub % BLOCKS) * kBM * BN + q * 1024 + y / 2 * 256 + x * 8 + y % 2 * 4;
#pragma unroll 8
  for (long long b = first; b <= last; ++b, src += (long long)BLOCKS * kBM * BN) {
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

// out = bias: a product over no k's.
template <typename OT, class P>
__global__ void __launch_bounds__(256) bias_kernel(const __grid_constant__ P p) {
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < (long long)p.m * p.n; e += (long long)gridDim.x * 256) {
    const long long i = e / p.n, j = e - i * p.n;
    ((OT*)p.out)[i * p.ldo + j] = from_f32<OT>(p.bias ? p.bias[j] : 0.0f);
  }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
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

// Slabs of 128 bytes by `box_rows` rows of a matrix of bytes; what lies outside is read as zeros.
inline bool make_map(CUtensorMap* map, const void* base, long long rows, long long bytes, long long ld, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles of scales, 512 bytes each, two at a time.
inline bool make_scale_map(CUtensorMap* map, const void* base, long long tiles) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)tiles}, strides[1] = {512};
  const cuuint32_t box[2] = {128, 2}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `box_rows` rows of 128 bytes from an array of such rows, as they lie in memory.
inline bool make_plain_map(CUtensorMap* map, const void* base, size_t rows, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace emb
