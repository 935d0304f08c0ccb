// Norm, gate, residual and norm in one pass (forward).
//
//   y = res_scale * x + act(gate) * (norm(f) * w_post + b_post)
//   h = norm(y) * w_pre + b_pre
//
// Bound by memory: x, f and a per-element gate in, y and h out, once each; the
// vectors stay in registers over a team's rows.  Two row sums (four for a
// layer norm) separate the loads from the stores, so each team loads its next
// row before it reduces the current one.  In a loop, 131,072 x 1024 bf16: 219 us, 0.90
// of the measured copy rate; 16,384 x 1664 with a float32 stream 77 us, 0.73.  Rows
// that are not multiples of eight elements go one element at a time: 65,536 x 1003
// bf16 279 us, 0.35 (issue: about sixty instructions an element).  Teams of 1024
// threads have 64 registers a thread and spill in some forms (up to 160 bytes).
#include <algorithm>
#include <cmath>

#include "emb_norm.cuh"

namespace emb {
namespace {

struct FwdArgs {
  const void *x, *f, *gate;
  const float *w_post, *b_post, *w_pre, *b_pre;
  void *y, *h;
  float4* stats;
  long long rows;
  int dim, team, gate_kind, act;
  float eps, res_scale, inv_dim;
};

// MAXT: most threads of a block.  A thread of a 1024-thread team has 64
// registers, too few to hold its vectors' elements over the rows: it reads
// them again from L1 where it needs them.
// FULL: the usual case (every array there, a sigmoid gate per element), known when
// compiling: half the instructions of the other cases are their branches and
// what the branches' ends move between registers.
template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT, bool FULL>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) norm_gate_fwd_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ float2 slots[4][64];  // teams that need them: 64 threads or more, so at most 4 a block
  // A row is loaded while the one before it is reduced (16,384 x 1664, float32
  // stream: 77 us, 114 without; 131,072 x 1024 bf16 219, 288), where registers allow.
  constexpr bool kPre = MAXT < 1024;
  constexpr bool kHold = MAXT < 1024;  // registers enough to keep the vectors over the rows
  constexpr bool kFine = sizeof(ST) == 4;  // float32 rows: see activate()
  constexpr int E = norm_elems<VEC, MAXT>();
  const int team = a.team, dim = a.dim;
  const int my_team = threadIdx.x / team;
  TeamSum sums{team, (int)threadIdx.x % team, team >> 5, 1 + (my_team & 3), slots[my_team & 3]};
  const int t = sums.t;
  const int teams = blockDim.x / team;
  const long long stride = (long long)gridDim.x * teams;
  const bool has_f = FULL || a.f != nullptr, has_h = FULL || a.h != nullptr;
  const int gate_kind = FULL ? (int)EMB_GATE_ELEM : a.gate_kind, act = FULL ? (int)EMB_ACT_SIGMOID : a.act;
  const bool gate_elem = gate_kind == EMB_GATE_ELEM;
  const float* const gate_col = gate_kind == EMB_GATE_COL ? (const float*)a.gate : nullptr;
  VecPart<VEC, kHold, E, FULL> wp(a.w_post, 1.0f, t, team, dim), wq(a.w_pre, 1.0f, t, team, dim);
  VecPart<VEC, kHold, E, FULL && LAYER> bp(LAYER ? a.b_post : nullptr, 0.0f, t, team, dim), bq(LAYER ? a.b_pre : nullptr, 0.0f, t, team, dim);
  VecPart<VEC, kHold, E, false> gc(gate_col, 0.0f, t, team, dim);
  if (kHold && gate_col) {  // once, not for each row
#pragma unroll
    for (int k = 0; k < E; ++k) gc.v[kHold ? k : 0] = activate<true>(gc.v[kHold ? k : 0], act);
  }

  RowPart<ST, VEC, E> rx;
  RowPart<BT, VEC, E> rf, rg;
  float grow = 0.0f;
  rx.clear();
  rf.clear();
  rg.clear();
  auto load = [&](long long r) {
    rx.load((const ST*)a.x + r * dim, t, team, dim);
    if (has_f) rf.load((const BT*)a.f + r * dim, t, team, dim);
    if (gate_elem) rg.load((const BT*)a.gate + r * dim, t, team, dim);
    if (gate_kind == EMB_GATE_ROW) grow = to_f32<BT>(((const BT*)a.gate)[r]);
  };
  // norm of v in place; returns (mean, 1/sqrt)
  auto norm = [&](float* v) {
    float s = 0.0f, mean = 0.0f;
    if (LAYER) {
#pragma unroll
      for (int k = 0; k < E; ++k) s += v[k];
      mean = sums.sum<false>(s, 0.0f).x * a.inv_dim;
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = part_col<VEC>(k, t, team) < dim ? v[k] - mean : 0.0f;
    }
    s = 0.0f;  // of v^2 / dim: the sum itself could overflow where the mean does not
#pragma unroll
    for (int k = 0; k < E; ++k) s += (v[k] * a.inv_dim) * v[k];
    const float r = 1.0f / sqrtf(sums.sum<false>(s, 0.0f).x + a.eps);
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] *= r;
    return make_float2(mean, r);
  };

  // all teams of a block go through as many rounds, so that a warp's teams stay together
  const long long b_first = (long long)blockIdx.x * teams, r_first = b_first + my_team;
  const long long rounds = a.rows > b_first ? (a.rows - b_first + stride - 1) / stride : 0;
  if (kPre && r_first < a.rows) load(r_first);
  for (long long i = 0; i < rounds; ++i) {
    const long long r = r_first + i * stride;
    const bool live = r < a.rows;
    if (!kPre && live) load(r);
    float x[E], f[E], g[E], w[E], b[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      x[k] = rx.get(k);
      f[k] = rf.get(k);
      g[k] = rg.get(k);
    }
    const float gr = grow;
    if (kPre && r + stride < a.rows) load(r + stride);
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (has_f) {
      if (gate_elem) {
#pragma unroll
        for (int k = 0; k < E; ++k) g[k] = activate<kFine>(g[k], act);
      } else if (gate_col) {
        gc.get(g);
        if (!kHold) {
#pragma unroll
          for (int k = 0; k < E; ++k) g[k] = activate<true>(g[k], act);
        }
      } else {
        const float v = gate_kind == EMB_GATE_ROW ? activate<kFine>(gr, act) : 1.0f;
#pragma unroll
        for (int k = 0; k < E; ++k) g[k] = v;
      }
      const float2 s = norm(f);
      st.x = s.x;
      st.y = s.y;
      wp.get(w);
      if (LAYER) bp.get(b);
#pragma unroll
      for (int k = 0; k < E; ++k) x[k] = x[k] * a.res_scale + g[k] * (LAYER ? f[k] * w[k] + b[k] : f[k] * w[k]);
      if (live) RowPart<ST, VEC, E>::store((ST*)a.y + r * dim, x, t, team, dim);
    }
    if (has_h) {
#pragma unroll
      for (int k = 0; k < E; ++k) x[k] = to_f32<ST>(from_f32<ST>(x[k]));  // the stored residual
      const float2 s = norm(x);
      st.z = s.x;
      st.w = s.y;
      wq.get(w);
      if (LAYER) bq.get(b);
#pragma unroll
      for (int k = 0; k < E; ++k) x[k] = LAYER ? x[k] * w[k] + b[k] : x[k] * w[k];
      if (live) RowPart<BT, VEC, E>::store((BT*)a.h + r * dim, x, t, team, dim);
    }
    if ((FULL || a.stats) && t == 0 && live) a.stats[r] = st;
  }
}

template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT, bool FULL>
cudaError_t launch_as(const FwdArgs& a, cudaStream_t st) {
  const int threads = std::max(kNormBlock, a.team);
  const int teams = threads / a.team;
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_gate_fwd_kernel<ST, BT, VEC, LAYER, MAXT, FULL>, threads, 0);
  if (e != cudaSuccess) return e;
  const long long blocks = std::min((a.rows + teams - 1) / teams, (long long)std::max(1, per_sm) * sm_count());
  norm_gate_fwd_kernel<ST, BT, VEC, LAYER, MAXT, FULL><<<(int)blocks, threads, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename ST, typename BT, bool VEC, bool LAYER, int MAXT>
cudaError_t launch_full(const FwdArgs& a, cudaStream_t st) {
  const bool full = a.gate_kind == EMB_GATE_ELEM && a.act == EMB_ACT_SIGMOID && a.f && a.h && a.stats && a.w_post &&
                    a.w_pre && aligned_to(a.w_post, 16) && aligned_to(a.w_pre, 16) &&
                    (!LAYER || (a.b_post && a.b_pre && aligned_to(a.b_post, 16) && aligned_to(a.b_pre, 16)));
  return full ? launch_as<ST, BT, VEC, LAYER, MAXT, true>(a, st) : launch_as<ST, BT, VEC, LAYER, MAXT, false>(a, st);
}
template <typename ST, typename BT, bool VEC>
cudaError_t launch(const FwdArgs& a, bool layer, cudaStream_t st) {
  if (a.team <= kNormBlock)
    return layer ? launch_full<ST, BT, VEC, true, kNormBlock>(a, st) : launch_full<ST, BT, VEC, false, kNormBlock>(a, st);
  if (a.team <= 512) return layer ? launch_full<ST, BT, VEC, true, 512>(a, st) : launch_full<ST, BT, VEC, false, 512>(a, st);
  return layer ? launch_full<ST, BT, VEC, true, 1024>(a, st) : launch_full<ST, BT, VEC, false, 1024>(a, st);
}

}  // namespace

emb_status check_norm(const emb_norm_gate_desc* d) {
  if (!d) return fail(EMB_ERR_INVALID_ARG, "desc is NULL");
  if (d->rows < 0 || d->dim < 1) return fail(EMB_ERR_INVALID_ARG, "need rows >= 0 and dim >= 1");
  if (d->dim > EMB_NORM_MAX_DIM) return fail(EMB_ERR_UNSUPPORTED, "dim above EMB_NORM_MAX_DIM");
  if (d->rows > (1LL << 46)) return fail(EMB_ERR_UNSUPPORTED, "too many rows");
  if (!good_ftype(d->stream_t) || !good_ftype(d->block_t) ||
      (d->stream_t != d->block_t && d->stream_t != EMB_T_F32))
    return fail(EMB_ERR_INVALID_ARG, "stream_t must be block_t or EMB_T_F32");
  if (d->norm != EMB_NORM_RMS && d->norm != EMB_NORM_LAYER) return fail(EMB_ERR_INVALID_ARG, "bad norm");
  if (d->gate < EMB_GATE_NONE || d->gate > EMB_GATE_COL) return fail(EMB_ERR_INVALID_ARG, "bad gate");
  if (d->act != EMB_ACT_IDENTITY && d->act != EMB_ACT_SIGMOID) return fail(EMB_ERR_INVALID_ARG, "bad act");
  if (!(d->eps > 0) || !std::isfinite(d->eps) || !std::isfinite(d->res_scale))
    return fail(EMB_ERR_INVALID_ARG, "need eps > 0 and a finite res_scale");
  return EMB_OK;
}

}  // namespace emb

using namespace emb;

extern "C" emb_status emb_norm_gate_fwd(const emb_norm_gate_desc* desc, const void* x_d, const void* f_d,
                                        const void* gate_d, const float* w_post_d, const float* b_post_d,
                                        const float* w_pre_d, const float* b_pre_d, void* y_d, void* h_d,
                                        float* stats_d, void* stream) {
  const emb_status rc = check_norm(desc);
  if (rc != EMB_OK) return rc;
  const emb_norm_gate_desc& d = *desc;
  if (d.rows == 0) return EMB_OK;
  if (!f_d && (y_d || gate_d || w_post_d || b_post_d || d.gate != EMB_GATE_NONE))
    return fail(EMB_ERR_INVALID_ARG, "without f there is no y, gate or post vector");
  if (!h_d && (w_pre_d || b_pre_d)) return fail(EMB_ERR_INVALID_ARG, "without h there is no pre vector");
  if (d.norm == EMB_NORM_RMS && (b_post_d || b_pre_d)) return fail(EMB_ERR_INVALID_ARG, "biases need EMB_NORM_LAYER");
  if ((d.gate != EMB_GATE_NONE) != (gate_d != nullptr)) return fail(EMB_ERR_INVALID_ARG, "gate does not match desc->gate");
  if (!x_d || (f_d && !y_d) || (!f_d && !h_d)) return fail(EMB_ERR_INVALID_ARG, "x, y or h is NULL");
  const size_t sb = ftype_bytes(d.stream_t), bb = ftype_bytes(d.block_t);
  const size_t gb = d.gate == EMB_GATE_COL ? 4 : bb;
  if (!aligned_to(x_d, sb) || !aligned_to(y_d, sb) || !aligned_to(f_d, bb) || !aligned_to(h_d, bb) ||
      !aligned_to(gate_d, gb) || !aligned_to(w_post_d, 4) || !aligned_to(b_post_d, 4) || !aligned_to(w_pre_d, 4) ||
      !aligned_to(b_pre_d, 4))
    return fail(EMB_ERR_INVALID_ARG, "an array is not aligned to its elements");
  if (!aligned_to(stats_d, 16)) return fail(EMB_ERR_INVALID_ARG, "stats must be 16-byte aligned");
  const bool vec = d.dim % 8 == 0 && aligned_to(x_d, 8 * sb) && aligned_to(y_d, 8 * sb) && aligned_to(f_d, 8 * bb) &&
                   aligned_to(h_d, 8 * bb) && (d.gate != EMB_GATE_ELEM || aligned_to(gate_d, 8 * bb));
  const FwdArgs a{x_d, f_d, gate_d, w_post_d, b_post_d, w_pre_d, b_pre_d, y_d, h_d, (float4*)stats_d, d.rows, d.dim,
                  norm_team(d.dim, vec), d.gate, d.act, d.eps, d.res_scale, 1.0f / (float)d.dim};
  const bool layer = d.norm == EMB_NORM_LAYER;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
#define EMB_NORM_FWD(S, B) e = vec ? launch<S, B, true>(a, layer, st) : launch<S, B, false>(a, layer, st)
  if (d.block_t == EMB_T_F32) EMB_NORM_FWD(float, float);
  else if (d.block_t == EMB_T_BF16 && d.stream_t == EMB_T_F32) EMB_NORM_FWD(float, __nv_bfloat16);
  else if (d.block_t == EMB_T_BF16) EMB_NORM_FWD(__nv_bfloat16, __nv_bfloat16);
  else if (d.stream_t == EMB_T_F32) EMB_NORM_FWD(float, __half);
  else EMB_NORM_FWD(__half, __half);
#undef EMB_NORM_FWD
  if (e != cudaSuccess) return cuda_fail(e, "norm_gate_fwd_kernel launch");
  return EMB_OK;
}
