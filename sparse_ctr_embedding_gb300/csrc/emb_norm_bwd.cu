// Norm, gate, residual and norm in one pass (backward).
//
// With yhat = (y - mean) / sigma of the pre norm and fhat likewise of the post
// norm, a = act(gate), n = fhat * w_post + b_post, per row:
//   d  = dh * w_pre;   dt = dy + (d - yhat * mean(d * yhat) [- mean(d)]) / sigma_y
//   dx = res_scale * dt;   dgate = dt * n * act'(gate);   dn = dt * a
//   e  = dn * w_post;  df = (e - fhat * mean(e * fhat) [- mean(e)]) / sigma_f
// and over the rows  dw_pre = sum dh * yhat, db_pre = sum dh,
// dw_post = sum dn * fhat, db_post = sum dn ([..]: layer norm only).
//
// Bound by memory: five arrays in and three out, once each.  The sums over
// rows stay with the thread that owns the column (registers; shared memory for
// 1024-thread teams) over all rows of its team, are joined over a block's
// teams, and leave as one partial per block; a second launch adds the blocks'
// partials in order, so the result does not depend on which block ran first.
// 131,072 x 1024 bf16: 447 us in a loop, 0.71 of the measured copy rate.  Neither
// memory nor issue is full (DRAM 0.45, issue 0.54 of the time at 65,536 rows): the two
// dependent sums a row are latency, with 16 warps an SM to hide it.  The warps' sums and
// rows take 127 registers a thread; 85 spill and take 830 us, rows staged in shared
// memory instead of registers 540 (this form then 520).
// Teams of 1024 threads (dims above 4096, or above 2048 off the vectors' alignment)
// have 64 registers a thread and spill (0.2 to 1.5 KB of loads a thread): 16,384 x 8192 bf16 628 us
// (0.50), with layer norms 835 (0.38), float32 1575 (0.40).
#include <algorithm>

#include "emb_norm.cuh"

namespace emb {
namespace {

constexpr int kSums = 5;  // dw_post, db_post, dw_pre, db_pre, per-channel dgate
// Most blocks an SM is given: as many as the workspace has partials for.
constexpr int max_blocks_per_sm(int threads) { return 1024 / threads; }

struct BwdArgs {
  const void *dy, *dh, *y, *f, *gate;
  const float4* stats;
  const float *w_post, *b_post, *w_pre;
  void *dx, *df, *dgate;
  float* partial;  // [blocks][kSums][dim]
  long long rows;
  int dim, team, gate_kind, act;
  unsigned want;   // bit i: sum i is asked for
  float res_scale, inv_dim;
};

// Sums over a thread's rows for its columns: in registers, or for 1024-thread
// teams (64 registers a thread) in shared memory, in words of the thread's own.
template <bool kHold, int E>
struct ColSums {
  float v[kHold ? kSums : 1][E];
  float* sh;  // !kHold: [kSums][E][blockDim]
  __device__ __forceinline__ explicit ColSums(float* shared) : sh(shared) {
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if constexpr (kHold) v[s][k] = 0.0f;
        else sh[(s * E + k) * blockDim.x + threadIdx.x] = 0.0f;
      }
  }
  __device__ __forceinline__ void add(int s, int k, float x) {
    if constexpr (kHold) v[s][k] += x;
    else sh[(s * E + k) * blockDim.x + threadIdx.x] += x;
  }
  __device__ __forceinline__ float get(int s, int k) const {
    if constexpr (kHold) return v[s][k];
    else return sh[(s * E + k) * blockDim.x + threadIdx.x];
  }
};

// FULL: the usual case (every array there, a sigmoid gate per element), known when
// compiling: half the instructions of the other cases are their branches and
// what the branches' ends move between registers.
template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT, bool FULL>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) norm_gate_bwd_kernel(const __grid_constant__ BwdArgs a) {
  // A row is loaded while the one before it is reduced (131,072 x 1024 bf16: 447
  // us, 460 without), where registers allow: a layer norm's vector form would
  // spill (32,768 x 2048 bf16: 288 us without, 290 with).
  constexpr bool kPre = MAXT < 1024 && !(VEC && LAYER);
  constexpr bool kHold = MAXT < 1024;  // registers enough to keep the sums over the rows
  constexpr bool kFine = sizeof(BT) == 4;  // float32 gradients of the block and its gate: see activate()
  constexpr int E = norm_elems<VEC, MAXT>();
  extern __shared__ float dyn[];
  __shared__ float2 slots[4][64];
  const int team = a.team, dim = a.dim;
  const int my_team = threadIdx.x / team;
  TeamSum sums{team, (int)threadIdx.x % team, team >> 5, 1 + (my_team & 3), slots[my_team & 3]};
  const int t = sums.t;
  const int teams = blockDim.x / team;
  const long long stride = (long long)gridDim.x * teams;
  const bool has_f = FULL || a.f != nullptr, has_dh = FULL || a.dh != nullptr, has_dy = FULL || a.dy != nullptr;
  const int gate_kind = FULL ? (int)EMB_GATE_ELEM : a.gate_kind, act = FULL ? (int)EMB_ACT_SIGMOID : a.act;
  const bool gate_elem = gate_kind == EMB_GATE_ELEM;
  const float* const gate_col = gate_kind == EMB_GATE_COL ? (const float*)a.gate : nullptr;

  // the vectors are read for each row: registers go to the rows on their way and the sums
  VecPart<VEC, false, E, FULL> wp(a.w_post, 1.0f, t, team, dim), wq(a.w_pre, 1.0f, t, team, dim);
  VecPart<VEC, false, E, FULL && LAYER> bp(LAYER ? a.b_post : nullptr, 0.0f, t, team, dim);
  VecPart<VEC, false, E, false> gc(gate_col, 0.0f, t, team, dim);
  ColSums<kHold, E> cols(dyn);

  RowPart<ST, VEC, E> rdy, ry;
  RowPart<BT, VEC, E> rdh, rf, rg;
  float grow = 0.0f;
  float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto clear = [&] {  // no row: zeros, which add nothing to any sum
    rdy.clear();
    ry.clear();
    rdh.clear();
    rf.clear();
    rg.clear();
    st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  auto load = [&](long long r) {
    if (has_dy) rdy.load((const ST*)a.dy + r * dim, t, team, dim);
    if (has_dh) {
      rdh.load((const BT*)a.dh + r * dim, t, team, dim);
      ry.load((const ST*)a.y + r * dim, t, team, dim);
    }
    if (has_f) rf.load((const BT*)a.f + r * dim, t, team, dim);
    if (gate_elem) rg.load((const BT*)a.gate + r * dim, t, team, dim);
    if (gate_kind == EMB_GATE_ROW) grow = to_f32<BT>(((const BT*)a.gate)[r]);
    st = a.stats[r];
  };
  clear();

  const long long b_first = (long long)blockIdx.x * teams, r_first = b_first + my_team;
  const long long rounds = a.rows > b_first ? (a.rows - b_first + stride - 1) / stride : 0;
  if (kPre && r_first < a.rows) load(r_first);
  for (long long i = 0; i < rounds; ++i) {
    const long long r = r_first + i * stride;
    const bool live = r < a.rows;
    if (!kPre) {
      if (live) load(r);
      else clear();
    }
    float dt[E], dh[E], hat[E], f[E], g[E], w[E];
    const float4 s = st;
    const float gr = grow;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      // only a layer norm's mean makes something of the zeros past the row's end
      const bool in = !LAYER || part_col<VEC>(k, t, team) < dim;
      dt[k] = rdy.get(k);
      dh[k] = rdh.get(k);
      hat[k] = in ? (ry.get(k) - (LAYER ? s.z : 0.0f)) * s.w : 0.0f;
      f[k] = in ? (rf.get(k) - (LAYER ? s.x : 0.0f)) * s.y : 0.0f;
      g[k] = rg.get(k);
    }
    if (kPre) {
      if (r + stride < a.rows) load(r + stride);
      else clear();
    }
    if (has_dh) {
      float p = 0.0f, q = 0.0f;
      wq.get(w);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        cols.add(2, k, dh[k] * hat[k]);
        if (LAYER) cols.add(3, k, dh[k]);
        dh[k] *= w[k];
        p += dh[k] * hat[k];
        if (LAYER) q += dh[k];
      }
      const float2 m = sums.sum<LAYER>(p, q);
      const float c1 = m.x * a.inv_dim, c2 = LAYER ? m.y * a.inv_dim : 0.0f;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const bool in = !LAYER || part_col<VEC>(k, t, team) < dim;
        dt[k] = in ? dt[k] + s.w * (dh[k] - hat[k] * c1 - c2) : 0.0f;
      }
    }
    if (!has_f) {
      if (live && (FULL || a.dx)) RowPart<ST, VEC, E>::store((ST*)a.dx + r * dim, dt, t, team, dim);
      continue;
    }
    if (live && (FULL || a.dx)) {
      float dx[E];
#pragma unroll
      for (int k = 0; k < E; ++k) dx[k] = dt[k] * a.res_scale;
      RowPart<ST, VEC, E>::store((ST*)a.dx + r * dim, dx, t, team, dim);
    }
    if (gate_elem) {
#pragma unroll
      for (int k = 0; k < E; ++k) g[k] = activate<kFine>(g[k], act);
    } else if (gate_col) {
      gc.get(g);
#pragma unroll
      for (int k = 0; k < E; ++k) g[k] = activate<true>(g[k], act);
    } else {
      const float v = gate_kind == EMB_GATE_ROW ? activate<kFine>(gr, act) : 1.0f;
#pragma unroll
      for (int k = 0; k < E; ++k) g[k] = v;
    }
    float p = 0.0f, q = 0.0f;
    wp.get(w);
    if (gate_kind != EMB_GATE_NONE) {
      float n[E], dg_row = 0.0f;
#pragma unroll
      for (int k = 0; k < E; ++k) n[k] = 0.0f;
      if (LAYER) bp.get(n);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        n[k] = (f[k] * w[k] + n[k]) * dt[k];
        if (act == EMB_ACT_SIGMOID) n[k] *= g[k] * (1.0f - g[k]);
        dg_row += n[k];
        if (gate_col) cols.add(4, k, n[k]);
      }
      if (live && gate_elem && (FULL || a.dgate)) RowPart<BT, VEC, E>::store((BT*)a.dgate + r * dim, n, t, team, dim);
      if (gate_kind == EMB_GATE_ROW) {
        const float v = sums.sum<false>(dg_row, 0.0f).x;
        if (live && t == 0 && a.dgate) ((BT*)a.dgate)[r] = from_f32<BT>(v);
      }
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float dn = dt[k] * g[k];
      cols.add(0, k, dn * f[k]);
      if (LAYER) cols.add(1, k, dn);
      dt[k] = dn * w[k];
      p += dt[k] * f[k];
      if (LAYER) q += dt[k];
    }
    if (FULL || a.df) {
      const float2 m = sums.sum<LAYER>(p, q);
      const float c1 = m.x * a.inv_dim, c2 = LAYER ? m.y * a.inv_dim : 0.0f;
#pragma unroll
      for (int k = 0; k < E; ++k) dt[k] = s.y * (dt[k] - f[k] * c1 - c2);
      if (live) RowPart<BT, VEC, E>::store((BT*)a.df + r * dim, dt, t, team, dim);
    }
  }

  // join the block's teams in order, write the block's partial sums
#pragma unroll
  for (int c = 0; c < kSums; ++c) {
    if (!(a.want >> c & 1)) continue;
    float* out = a.partial + ((long long)blockIdx.x * kSums + c) * dim;
    if (teams == 1) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const int col = part_col<VEC>(k, t, team);
        if (col < dim) out[col] = cols.get(c, k);
      }
    } else if constexpr (kHold) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < E; ++k) dyn[my_team * team * E + part_col<VEC>(k, t, team)] = cols.get(c, k);
      __syncthreads();
      for (int col = threadIdx.x; col < dim; col += blockDim.x) {
        float v = 0.0f;
        for (int j = 0; j < teams; ++j) v += dyn[j * team * E + col];
        out[col] = v;
      }
    }
  }
}

struct JoinArgs {
  const float* partial;
  float* out[kSums];
  int dim, blocks;
};

// Sums the blocks' partials: 32 columns a block, 32 threads a column, each
// adding every 32nd partial, then the 32 in order.
constexpr int kJoin = 32;
__global__ void __launch_bounds__(32 * kJoin) norm_join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float part[kJoin][33];
  float* out = a.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < a.dim) {
    const float* p = a.partial + (long long)blockIdx.y * a.dim + col;
    const long long step = (long long)kSums * a.dim;
#pragma unroll 8
    for (int b = w; b < a.blocks; b += kJoin) v += p[b * step];
  }
  part[w][lane] = v;
  __syncthreads();
  if (w == 0 && col < a.dim) {
#pragma unroll
    for (int j = 1; j < kJoin; ++j) v += part[j][lane];
    out[col] = v;
  }
}

// Most blocks of a launch, whichever way its rows are read.
long long bwd_blocks(long long rows, int dim) {
  long long most = 0;
  for (const bool vec : {false, true}) {
    const int team = norm_team(dim, vec), threads = std::max(kNormBlock, team), teams = threads / team;
    most = std::max(most, std::min((rows + teams - 1) / teams, (long long)max_blocks_per_sm(threads) * sm_count()));
  }
  return most;
}

template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT, bool FULL>
cudaError_t launch_as(const BwdArgs& a, cudaStream_t st, int* blocks_out) {
  const int threads = std::max(kNormBlock, a.team);
  const int teams = threads / a.team;
  const size_t smem = sizeof(float) * threads * norm_elems<VEC, MAXT>() * (MAXT == 1024 ? kSums : teams > 1 ? 1 : 0);
  auto* k = norm_gate_bwd_kernel<ST, BT, VEC, LAYER, MAXT, FULL>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, smem);
  if (e != cudaSuccess) return e;
  per_sm = std::min(std::max(1, per_sm), max_blocks_per_sm(threads));
  const long long blocks = std::min((a.rows + teams - 1) / teams, (long long)per_sm * sm_count());
  k<<<(int)blocks, threads, smem, st>>>(a);
  *blocks_out = (int)blocks;
  return cudaGetLastError();
}
template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT>
cudaError_t launch_full(const BwdArgs& a, cudaStream_t st, int* blocks) {
  const bool full = a.gate_kind == EMB_GATE_ELEM && a.act == EMB_ACT_SIGMOID && a.f && a.dh && a.dy && a.dx && a.df &&
                    a.dgate && a.w_post && a.w_pre && aligned_to(a.w_post, 16) && aligned_to(a.w_pre, 16) &&
                    (!LAYER || (a.b_post && aligned_to(a.b_post, 16)));
  return full ? launch_as<ST, BT, VEC, LAYER, MAXT, true>(a, st, blocks) : launch_as<ST, BT, VEC, LAYER, MAXT, false>(a, st, blocks);
}
template <typename ST, typename BT, bool VEC>
cudaError_t launch(const BwdArgs& a, bool layer, cudaStream_t st, int* blocks) {
  if (a.team <= kNormBlock)
    return layer ? launch_full<ST, BT, VEC, true, kNormBlock>(a, st, blocks) : launch_full<ST, BT, VEC, false, kNormBlock>(a, st, blocks);
  if (a.team <= 512) return layer ? launch_full<ST, BT, VEC, true, 512>(a, st, blocks) : launch_full<ST, BT, VEC, false, 512>(a, st, blocks);
  return layer ? launch_full<ST, BT, VEC, true, 1024>(a, st, blocks) : launch_full<ST, BT, VEC, false, 1024>(a, st, blocks);
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_norm_gate_bwd_workspace_size(const emb_norm_gate_desc* desc, size_t* bytes) {
  const emb_status rc = check_norm(desc);
  if (rc != EMB_OK) return rc;
  if (!bytes) return fail(EMB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)bwd_blocks(desc->rows, desc->dim) * kSums * desc->dim * sizeof(float);
  return EMB_OK;
}

extern "C" emb_status emb_norm_gate_bwd(const emb_norm_gate_desc* desc, const void* dy_d, const void* dh_d,
                                        const void* y_d, const void* f_d, const void* gate_d, const float* stats_d,
                                        const float* w_post_d, const float* b_post_d, const float* w_pre_d, void* dx_d,
                                        void* df_d, void* dgate_d, float* dw_post_d, float* db_post_d, float* dw_pre_d,
                                        float* db_pre_d, void* workspace_d, size_t ws_bytes, void* stream) {
  emb_status rc = check_norm(desc);
  if (rc != EMB_OK) return rc;
  const emb_norm_gate_desc& d = *desc;
  if (!f_d && (gate_d || d.gate != EMB_GATE_NONE || w_post_d || b_post_d || df_d || dgate_d || dw_post_d || db_post_d) && d.rows > 0)
    return fail(EMB_ERR_INVALID_ARG, "without f there is no gate, post vector or gradient of them");
  if (!dh_d && (w_pre_d || dw_pre_d || db_pre_d) && d.rows > 0)
    return fail(EMB_ERR_INVALID_ARG, "without dh there is no pre vector or gradient of it");
  if (d.norm == EMB_NORM_RMS && (b_post_d || db_post_d || db_pre_d)) return fail(EMB_ERR_INVALID_ARG, "biases need EMB_NORM_LAYER");
  if (d.gate == EMB_GATE_NONE && (gate_d || dgate_d)) return fail(EMB_ERR_INVALID_ARG, "gate does not match desc->gate");
  if (d.rows > 0) {
    if (!dy_d && !dh_d) return fail(EMB_ERR_INVALID_ARG, "dy and dh are NULL");
    if (d.gate != EMB_GATE_NONE && !gate_d) return fail(EMB_ERR_INVALID_ARG, "gate does not match desc->gate");
    if ((dh_d && !y_d) || !stats_d) return fail(EMB_ERR_INVALID_ARG, "y or stats is NULL");
  }
  const size_t sb = ftype_bytes(d.stream_t), bb = ftype_bytes(d.block_t);
  const size_t gb = d.gate == EMB_GATE_COL ? 4 : bb;
  if (!aligned_to(dy_d, sb) || !aligned_to(y_d, sb) || !aligned_to(dx_d, sb) || !aligned_to(dh_d, bb) ||
      !aligned_to(f_d, bb) || !aligned_to(df_d, bb) || !aligned_to(gate_d, gb) || !aligned_to(dgate_d, gb))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  for (const void* p : {(const void*)w_post_d, (const void*)b_post_d, (const void*)w_pre_d, (const void*)dw_post_d,
                        (const void*)db_post_d, (const void*)dw_pre_d, (const void*)db_pre_d})
    if (!aligned_to(p, 4)) return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (!aligned_to(stats_d, 16)) return fail(EMB_ERR_INVALID_ARG, "stats must be 16-byte aligned");
  JoinArgs j{(const float*)workspace_d,
             {dw_post_d, db_post_d, dw_pre_d, db_pre_d, d.gate == EMB_GATE_COL ? (float*)dgate_d : nullptr},
             d.dim, 0};
  unsigned want = 0;
  for (int i = 0; i < kSums; ++i) want |= j.out[i] ? 1u << i : 0u;
  if (want && d.rows > 0) {
    size_t need = 0;
    rc = emb_norm_gate_bwd_workspace_size(desc, &need);
    if (rc != EMB_OK) return rc;
    if (!workspace_d || ws_bytes < need) return fail(EMB_ERR_WORKSPACE, "workspace missing or smaller than emb_norm_gate_bwd_workspace_size()");
    if (!aligned_to(workspace_d, 16)) return fail(EMB_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  }
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (d.rows > 0) {
    const bool ge = d.gate == EMB_GATE_ELEM;
    const bool vec = d.dim % 8 == 0 && aligned_to(dy_d, 8 * sb) && aligned_to(dh_d, 8 * bb) && aligned_to(y_d, 8 * sb) &&
                     aligned_to(f_d, 8 * bb) && aligned_to(dx_d, 8 * sb) && aligned_to(df_d, 8 * bb) &&
                     (!ge || (aligned_to(gate_d, 8 * bb) && aligned_to(dgate_d, 8 * bb)));
    const BwdArgs a{dy_d, dh_d, y_d, f_d, gate_d, (const float4*)stats_d, w_post_d, b_post_d, w_pre_d, dx_d, df_d,
                    dgate_d, (float*)workspace_d, d.rows, d.dim, norm_team(d.dim, vec), d.gate, d.act, want, d.res_scale,
                    1.0f / (float)d.dim};
    const bool layer = d.norm == EMB_NORM_LAYER;
#define EMB_NORM_BWD(S, B) e = vec ? launch<S, B, true>(a, layer, st, &j.blocks) : launch<S, B, false>(a, layer, st, &j.blocks)
    if (d.block_t == EMB_T_F32) EMB_NORM_BWD(float, float);
    else if (d.block_t == EMB_T_BF16 && d.stream_t == EMB_T_F32) EMB_NORM_BWD(float, __nv_bfloat16);
    else if (d.block_t == EMB_T_BF16) EMB_NORM_BWD(__nv_bfloat16, __nv_bfloat16);
    else if (d.stream_t == EMB_T_F32) EMB_NORM_BWD(float, __half);
    else EMB_NORM_BWD(__half, __half);
#undef EMB_NORM_BWD
    if (e != cudaSuccess) return cuda_fail(e, "norm_gate_bwd_kernel launch");
  }
  if (want) {
    norm_join_kernel<<<dim3((d.dim + 31) / 32, kSums), 32 * kJoin, 0, st>>>(j);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "norm_join_kernel launch");
  }
  return EMB_OK;
}
