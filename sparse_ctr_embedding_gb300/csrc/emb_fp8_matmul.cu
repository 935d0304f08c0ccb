// Product of two 8-bit block-scaled matrices.
#include <algorithm>

#include "emb_dense.cuh"

namespace emb {
namespace {

__device__ unsigned g_op_flags;  // EMB_FLAG_OP_* bits since the last emb_check_op_flag

struct MatmulArgs {
  const unsigned char *a, *b;
  const float *sa, *sb, *bias;
  void* out;
  long long lda, ldb, ldo;
  long long sa_row, sb_row;  // scales in a row of sa and sb
  int m, n, k;
  int a_shift, b_shift;      // row i's scale is at i >> shift
};

__device__ __forceinline__ float code_to_f32(unsigned char c) { return e4m3x2_to_f32((unsigned short)c).x; }

template <typename OT>
__global__ void __launch_bounds__(256) matmul_kernel(const __grid_constant__ MatmulArgs p) {
  __shared__ float as[32][129], bs[32][129];
  const int i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[4] = {};
  for (int kb = 0; kb < (p.k + 127) / 128; ++kb) {
    for (int e = threadIdx.x; e < 32 * 128; e += 256) {
      const int r = e >> 7, c = e & 127, k = kb * 128 + c;
      as[r][c] = i0 + r < p.m && k < p.k ? code_to_f32(p.a[(i0 + r) * p.lda + k]) : 0.0f;
      bs[r][c] = j0 + r < p.n && k < p.k ? code_to_f32(p.b[(j0 + r) * p.ldb + k]) : 0.0f;
    }
    __syncthreads();
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + ty + 8 * q, j = j0 + tx;
      float s = 0.0f;
      for (int c = 0; c < 128; ++c) s += as[ty + 8 * q][c] * bs[tx][c];
      if (i < p.m && j < p.n)
        acc[q] += s * (p.sa[kb * p.sa_row + (i >> p.a_shift)] * p.sb[kb * p.sb_row + (j >> p.b_shift)]);
    }
    __syncthreads();
  }
  for (int q = 0; q < 4; ++q) {
    const int i = i0 + ty + 8 * q, j = j0 + tx;
    if (i < p.m && j < p.n) ((OT*)p.out)[i * p.ldo + j] = from_f32<OT>(acc[q] + (p.bias ? p.bias[j] : 0.0f));
  }
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  if (m < 0 || n < 0 || k < 0) return fail(EMB_ERR_INVALID_ARG, "negative m, n or k");
  if (m > 0x7fffffffLL || n > 0x7fffffffLL || k > 0x7fffffffLL) return fail(EMB_ERR_UNSUPPORTED, "m, n or k above 2^31 - 1");
  *bytes = 0;
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
  if (ldo < n) return fail(EMB_ERR_INVALID_ARG, "ldo below n");
  if (m == 0 || n == 0) return EMB_OK;
  if (!out_d || (k > 0 && (!a_d || !b_d || !sa_d || !sb_d))) return fail(EMB_ERR_INVALID_ARG, "a, b, a scale or out is NULL");
  if (!aligned_to(a_d, 16) || !aligned_to(b_d, 16)) return fail(EMB_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (!aligned_to(sa_d, 4) || !aligned_to(sb_d, 4) || !aligned_to(bias_d, 4) || !aligned_to(out_d, ftype_bytes(out_t)))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (need && (!workspace_d || ws_bytes < need))
    return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_fp8_matmul_workspace_size()");
  if (need && !aligned_to(workspace_d, 16)) return fail(EMB_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  const int as = a_block_rows == 1 ? 0 : 7, bs = b_block_rows == 1 ? 0 : 7;
  const MatmulArgs p{(const unsigned char*)a_d, (const unsigned char*)b_d, sa_d, sb_d, bias_d, out_d, lda, ldb, ldo,
                     as ? (m + 127) / 128 : m, bs ? (n + 127) / 128 : n, (int)m, (int)n, (int)k, as, bs};
  const dim3 grid((unsigned)((n + 31) / 32), (unsigned)((m + 31) / 32));
  if (grid.y > 65535u) return fail(EMB_ERR_UNSUPPORTED, "m too large");
  cudaStream_t st = (cudaStream_t)stream;
  if (out_t == EMB_T_F32) matmul_kernel<float><<<grid, 256, 0, st>>>(p);
  else if (out_t == EMB_T_BF16) matmul_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  else matmul_kernel<__half><<<grid, 256, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "matmul_kernel launch");
  return EMB_OK;
}

extern "C" emb_status emb_check_op_flag(void* stream, uint32_t* flags_out) {
  EMB_CUDA(cudaStreamSynchronize((cudaStream_t)stream));
  unsigned f = 0;
  const unsigned zero = 0;
  EMB_CUDA(cudaMemcpyFromSymbol(&f, g_op_flags, sizeof f));
  if (f) EMB_CUDA(cudaMemcpyToSymbol(g_op_flags, &zero, sizeof zero));
  if (flags_out) *flags_out = f;
  if (f) return fail(EMB_ERR_DEVICE_FLAG, "a dense operator's bounded wait ran out: its output is not valid");
  return EMB_OK;
}
