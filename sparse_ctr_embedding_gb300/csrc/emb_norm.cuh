// Row access and row reductions shared by the norm kernels (emb_norm_fwd.cu,
// emb_norm_bwd.cu).
//
// A row is worked on by a team of T threads, T a power of two from 8 to 1024,
// E elements a thread with E T >= dim.  Where dim and the pointers allow it
// (VEC) a thread has eight neighbours, read with one 16- or 32-byte access;
// else E (4, or 8 in teams of 1024) elements T apart.  The whole row then sits
// in registers, every array is read once, and a norm's mean and variance are
// taken in two exact steps from there.  Elements past the row's end are zeros
// in registers.
#pragma once

#include "emb_dense.cuh"

namespace emb {

constexpr int kNormBlock = 256;  // threads of a block, unless one team is larger

// Elements a thread has.
template <bool VEC, int MAXT>
__host__ __device__ constexpr int norm_elems() {
  return VEC || MAXT == 1024 ? 8 : 4;
}
inline int norm_team(int dim, bool vec) {
  int t = 8;
  while (t * (vec || t == 1024 ? 8 : 4) < dim) t *= 2;
  return t;
}

// This thread's elements of a row.
template <typename T, bool VEC, int E>
struct RowPart;
template <typename T, int E>
struct RowPart<T, true, E> {
  static_assert(E == 8, "one vector access");
  Raw8<T> r;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.set2(k, 0.0f, 0.0f);
  }
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
template <typename T, int E>
struct RowPart<T, false, E> {
  T v[E];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = from_f32<T>(0.0f);
  }
  __device__ __forceinline__ void load(const T* row, int t, int team, int dim) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (t + k * team < dim) v[k] = row[t + k * team];
  }
  __device__ __forceinline__ float get(int k) const { return to_f32<T>(v[k]); }
  __device__ __forceinline__ static void store(T* row, const float* v, int t, int team, int dim) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (t + k * team < dim) row[t + k * team] = from_f32<T>(v[k]);
  }
};

// Column of this thread's k-th element.
template <bool VEC>
__device__ __forceinline__ int part_col(int k, int t, int team) {
  return VEC ? t * 8 + k : t + k * team;
}

// This thread's elements of a float32 vector [dim] (NULL: all `absent`), held
// in registers over the rows, or read again (from L1) for each row.
// SURE: it is there, and aligned to 16 bytes.
template <bool VEC, bool kHold, int E, bool SURE>
struct VecPart {
  const float* p;
  float absent;
  int t, team, dim, vec;
  float v[kHold ? E : 1];
  __device__ __forceinline__ void read(float* o) const {
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = absent;
    if (!SURE && !p) return;
    if (VEC && (SURE || vec)) {
      if (t * 8 < dim) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + t * 8)), b = __ldg(reinterpret_cast<const float4*>(p + t * 8 + 4));
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
        if constexpr (E == 8) o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const int c = part_col<VEC>(k, t, team);
        if (c < dim) o[k] = __ldg(p + c);
      }
    }
  }
  __device__ __forceinline__ VecPart(const float* p_, float absent_, int t_, int team_, int dim_)
      : p(p_), absent(absent_), t(t_), team(team_), dim(dim_), vec((reinterpret_cast<uintptr_t>(p_) & 15) == 0) {
    if constexpr (kHold) read(v);
  }
  __device__ __forceinline__ void get(float* o) const {
    if constexpr (kHold) {
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] = v[k];
    } else {
      read(o);
    }
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
  template <bool TWO>
  __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      if (o < team) {  // the same in the whole block
        a += __shfl_xor_sync(0xffffffffu, a, o);
        if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
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
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (o < warps) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
    return make_float2(a, b);
  }
};

// 1 / (1 + e^-g), from the approximate power of two and reciprocal: the exact
// functions take over twenty instructions an element.  Results below 2^-126 are 0.
// FINE, where float32 values come of it: e^-g = 2^h (1 + l), h the rounded product
// -g log2(e), l the natural logarithm of what its rounding and the constant's left
// out.  Good to 9 rounding units (2^-24) for every gate, in ten instructions.
// Else, for gates of 8 or 11 bits in rows of such: h alone, in four.  Its error is up
// to 7 + 1.3 |g| units of the result for g < 0, at most 6 units of 1 (the result
// falls faster than |g| grows): far below the rows' own rounding, and in a sum over
// rows below the norm's.
template <bool FINE>
__device__ __forceinline__ float activate(float g, int act) {
  if (act != EMB_ACT_SIGMOID) return g;
  float e, a;
  if constexpr (FINE) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(88.0f));  // beyond, the result is 0 or 1 all the same
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(-88.0f));
    const float h = __fmul_rn(g, -1.44269502f);
    const float l = fmaf(fmaf(g, -1.44269502f, -h), 0.693147181f, g * -1.33497581e-8f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
    e = fmaf(e, l, e);
  } else {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.0f + e));
  return a;
}

emb_status check_norm(const emb_norm_gate_desc* d);

}  // namespace emb
