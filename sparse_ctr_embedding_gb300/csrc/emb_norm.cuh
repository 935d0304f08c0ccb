// Row access and row reductions shared by the norm kernels (emb_norm_fwd.cu,
// emb_norm_bwd.cu).
//
// A row is worked on by a team of T threads, T a power of two from 8 to 1024
// with 8 T >= dim, eight elements a thread: neighbouring ones read with one
// 16- or 32-byte access where dim and the pointers allow it (VEC), else T
// apart.  The whole row then sits in registers, every array is read once, and
// the norm's mean and variance are taken in two exact steps from there.
#pragma once

#include "emb_dense.cuh"

namespace emb {

// This thread's eight elements of a row.
template <typename T, bool VEC>
struct RowPart;
template <typename T>
struct RowPart<T, true> {
  Raw8<T> r;
  __device__ __forceinline__ void load(const T* row, int t, int, int dim) {
    if (t * 8 < dim) r.load(row + t * 8);
  }
  __device__ __forceinline__ float get(int k) const { return r.get(k); }
  __device__ __forceinline__ static void store(T* row, const float* v, int t, int, int dim) {
    if (t * 8 >= dim) return;
    Raw8<T> o;
#pragma unroll
    for (int k = 0; k < 4; ++k) o.set2(k, v[2 * k], v[2 * k + 1]);
    o.store(row + t * 8);
  }
};
template <typename T>
struct RowPart<T, false> {
  T v[8];
  __device__ __forceinline__ void load(const T* row, int t, int team, int dim) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (t + k * team < dim) v[k] = row[t + k * team];
  }
  __device__ __forceinline__ float get(int k) const { return to_f32<T>(v[k]); }
  __device__ __forceinline__ static void store(T* row, const float* v, int t, int team, int dim) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (t + k * team < dim) row[t + k * team] = from_f32<T>(v[k]);
  }
};

// Column of this thread's k-th element, and whether the row has it.
template <bool VEC>
__device__ __forceinline__ int part_col(int k, int t, int team) {
  return VEC ? t * 8 + k : t + k * team;
}

// This thread's eight elements of a float32 vector [dim] (NULL: all `absent`),
// held in registers over the rows, or read again at each use.
template <bool VEC, bool kHold>
struct VecPart {
  const float* p;
  float absent;
  int t, team, dim;
  float v[kHold ? 8 : 1];
  __device__ __forceinline__ float read(int k) const {
    const int c = part_col<VEC>(k, t, team);
    return p && c < dim ? __ldg(p + c) : absent;
  }
  __device__ __forceinline__ VecPart(const float* p_, float absent_, int t_, int team_, int dim_)
      : p(p_), absent(absent_), t(t_), team(team_), dim(dim_) {
    if constexpr (kHold) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = read(k);
    }
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (kHold) return v[k];
    else return read(k);
  }
};

// Sums over a team.  Teams of up to a warp use shuffles; larger ones one
// shared-memory exchange and one named barrier per sum.  Two sets of slots
// alternate: a thread writes a set again only after the barrier of the sum in
// between, which every reader of the set has passed.
struct TeamSum {
  int team;      // threads
  int t;         // this thread's number in the team
  int warps;     // team / 32, or 0
  int bar;       // named barrier of the team
  float2* slots; // 2 x 32 of the team
  int set = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    for (int o = min(team, 32) >> 1; o; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps > 1) {
      float2* s = slots + set * 32;
      set ^= 1;
      const int lane = threadIdx.x & 31;
      if (lane == 0) s[t >> 5] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(team) : "memory");
      const float2 v = s[lane & (warps - 1)];
      a = v.x;
      b = v.y;
      for (int o = warps >> 1; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
    }
    return make_float2(a, b);
  }
};

constexpr int kNormBlock = 256;  // threads of a block, unless one team is larger

inline int norm_team(int dim) {
  int t = 8;
  while (t * 8 < dim) t *= 2;
  return t;
}

__device__ __forceinline__ float activate(float g, int act) {
  return act == EMB_ACT_SIGMOID ? 1.0f / (1.0f + expf(-g)) : g;
}

emb_status check_norm(const emb_norm_gate_desc* d);

}  // namespace emb
