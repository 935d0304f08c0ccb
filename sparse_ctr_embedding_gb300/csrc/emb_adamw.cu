// AdamW over many tensors in one launch, states in float32 or in 8 bits.
//
// A pass over memory: w, m and v are read and written once, the gradient read
// once.  28 bytes a weight in float32: bound by memory (100M weights in 412 us in a
// loop, the measured copy rate).  14 bytes with bf16 gradients and 8-bit states: bound
// by issue (86 instructions: two 8-bit roundings and their hash, an exact division
// and square root: the result has to be the one that IEEE arithmetic gives), 200M
// weights in 603 us, 0.68 of the copy rate.  Each unit's loads are issued before
// the unit before it is computed (709 us without, at four blocks an SM instead of
// three), and plain products and sums are done in pairs (627 us without; both then
// against 612 to 651).  With bf16 copies or a gradient scale the kernel of mixed types
// runs: 100M weights, 8-bit states 351 us with copies (0.67), 336 with a scale (0.61);
// float32 states with both 431 (0.96).
//
// Work is cut into units of 256 consecutive elements of one tensor, one warp
// each, eight elements a lane: the unit is the block that shares a scale, so
// its largest magnitude is one warp reduction and no shared memory is needed.
// The tensors' descriptors travel in the kernel's parameters (no table in
// device memory to fill, so nothing to order or to free); a warp finds its
// unit's tensor by bisection over their first units.
#include <cmath>

#include "emb_dense.cuh"

namespace emb {
namespace {

struct TensorArg {
  void* p;
  void* copy;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long n;
  long long first;
  unsigned unit0;       // first unit of this tensor among the launch's
  unsigned char pt, gt, ct, vec;
};

// Launches of up to 40 tensors pass 4 KB of parameters, of up to 120 12 KB, larger ones 32 KB.
template <int N>
struct StepArgs {
  TensorArg t[N];
  int n_tensors;
  unsigned n_units;
  unsigned span;        // consecutive units a block takes
  float beta1, omb1, beta2, omb2, decay, lr_c1, rc2, eps, one;
  unsigned key;
  const float* grad_scale;
};

// Eight elements of a float type as they lie in memory (f32 in all of w, the
// others in its first half), loaded in one step and read in another.
struct Raw {
  unsigned w[8];
  __device__ __forceinline__ void load(const void* base, int type, long long i) {
    if (type == EMB_T_F32)
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"((const float*)base + i));
    else
      asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"((const unsigned short*)base + i));
  }
  __device__ __forceinline__ void get(int type, float* o) const {
    if (type == EMB_T_F32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __uint_as_float(w[k]);
    } else if (type == EMB_T_BF16) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = __uint_as_float(w[k] << 16);
        o[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        o[2 * k] = v.x;
        o[2 * k + 1] = v.y;
      }
    }
  }
};

__device__ __forceinline__ void store8(void* base, int type, long long i, const float* o) {
  if (type == EMB_T_F32) {
    Raw8<float> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.set2(k, o[2 * k], o[2 * k + 1]);
    r.store((float*)base + i);
  } else if (type == EMB_T_BF16) {
    Raw8<__nv_bfloat16> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.set2(k, o[2 * k], o[2 * k + 1]);
    r.store((__nv_bfloat16*)base + i);
  } else {
    Raw8<__half> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.set2(k, o[2 * k], o[2 * k + 1]);
    r.store((__half*)base + i);
  }
}
__device__ __forceinline__ float load1(const void* base, int type, long long i) {
  return type == EMB_T_F32 ? ((const float*)base)[i]
         : type == EMB_T_BF16 ? __bfloat162float(((const __nv_bfloat16*)base)[i])
                              : __half2float(((const __half*)base)[i]);
}
__device__ __forceinline__ void store1(void* base, int type, long long i, float x) {
  if (type == EMB_T_F32) ((float*)base)[i] = x;
  else if (type == EMB_T_BF16) ((__nv_bfloat16*)base)[i] = __float2bfloat16_rn(x);
  else ((__half*)base)[i] = __float2half_rn(x);
}

// MurmurHash3 32-bit finaliser (Appleby, public domain).
__device__ __forceinline__ unsigned fmix32(unsigned h) {
  h ^= h >> 16;
  h *= 0x85ebca6bu;
  h ^= h >> 13;
  h *= 0xc2b2ae35u;
  return h ^ (h >> 16);
}

// Two elements side by side: each is rounded by itself as in the scalar operation,
// in one issue slot for both.  A sum is written as a multiply-add by `one`, a
// kernel argument: of a product and a sum in pairs the assembler makes one
// multiply-add with one rounding, whatever their rounding modifiers say.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 x, y;\n"
      "mov.b64 x, {%2, %3};\n"
      "mov.b64 y, {%4, %5};\n"
      "mul.rn.f32x2 x, x, y;\n"
      "mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float one, float2 b) {  // one = -1: b - a
  float2 r;
  asm("{\n.reg .b64 x, y, z;\n"
      "mov.b64 x, {%2, %3};\n"
      "mov.b64 y, {%4, %4};\n"
      "mov.b64 z, {%5, %6};\n"
      "fma.rn.f32x2 x, x, y, z;\n"
      "mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(one), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(const float* a, int k) { return make_float2(a[2 * k], a[2 * k + 1]); }
__device__ __forceinline__ void put(float* a, int k, float2 x) {
  a[2 * k] = x.x;
  a[2 * k + 1] = x.y;
}

// A magnitude in code units to one of the two codes around it, upwards with the
// probability of its distance from the lower one.  Codes from 2^-6 on have 3
// mantissa bits: adding 20 random bits below them and cutting rounds to one of
// them.  Below 2^-6 codes are 2^-9 apart; adding 2^-6 first puts that spacing at
// the same bit.  The block's largest value is 448 up to three units in its last
// place, and r20 leaves seven, so it is never carried past 448.  mag is finite.
__device__ __forceinline__ float2 round_random(float2 mag, float one, unsigned r20x, unsigned r20y) {
  const float2 base = make_float2(mag.x < 0.015625f ? 0.015625f : 0.0f, mag.y < 0.015625f ? 0.015625f : 0.0f);
  const float2 sum = add2(mag, one, base);
  const unsigned x = (__float_as_uint(sum.x) + r20x) & ~0xFFFFFu, y = (__float_as_uint(sum.y) + r20y) & ~0xFFFFFu;
  return add2(base, -one, make_float2(__uint_as_float(x), __uint_as_float(y)));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned warp_max(float a) {  // a >= 0 or NaN: the bits order as the values, NaN last
  return __reduce_max_sync(0xffffffffu, __float_as_uint(a));
}
// PT, GT: the element types of all the launch's parameters and gradients (then
// without copies and gradient scale), or -1: each tensor's own, branched on for
// every eight elements.
template <bool kQ8, int N, int PT, int GT>
__global__ void __launch_bounds__(256, 3) adamw_kernel(const __grid_constant__ StepArgs<N> a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr bool kPlain = PT >= 0;
  const float gs = !kPlain && a.grad_scale ? *a.grad_scale : 1.0f;
  const unsigned end = min(a.n_units, (blockIdx.x + 1) * a.span);
  unsigned unit = blockIdx.x * a.span + warp;
  if (unit >= end) return;
  int lo = 0, hi = a.n_tensors - 1;  // last tensor whose unit0 <= unit
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].unit0 <= unit) lo = mid; else hi = mid - 1;
  }
  // What a unit reads; with 8-bit states the next unit's loads are under way
  // while one is computed (see kAhead).
  struct Loaded {
    Raw p, g, m, v;  // m, v: float32 states
    uint2 cm, cv;    // 8-bit ones
    float ms, vs;
  } in;
  auto fetch = [&](unsigned u, int at) {
    const TensorArg& t = a.t[at];
    const unsigned blk = u - t.unit0;
    const long long i0 = (long long)blk * EMB_ADAM_BLOCK + lane * 8;
    if (kQ8) {
      in.ms = t.ms[blk];
      in.vs = t.vs[blk];
    }
    if (!t.vec || t.n - i0 < 8) return;
    in.g.load(t.g, kPlain ? GT : t.gt, i0);
    in.p.load(t.p, kPlain ? PT : t.pt, i0);
    if (kQ8) {
      in.cm = *reinterpret_cast<const uint2*>((const unsigned char*)t.m + i0);
      in.cv = *reinterpret_cast<const uint2*>((const unsigned char*)t.v + i0);
    } else {
      in.m.load(t.m, EMB_T_F32, i0);
      in.v.load(t.v, EMB_T_F32, i0);
    }
  };
  auto tensor_of = [&](unsigned u, int at) {
    while (at + 1 < a.n_tensors && a.t[at + 1].unit0 <= u) ++at;
    return at;
  };
  constexpr bool kAhead = kQ8;
  if (kAhead) fetch(unit, lo);
  for (; unit < end; unit += 8) {
    if (!kAhead) {
      lo = tensor_of(unit, lo);
      fetch(unit, lo);
    }
    const TensorArg& t = a.t[lo];
    const unsigned blk = unit - t.unit0;
    const long long i0 = (long long)blk * EMB_ADAM_BLOCK + lane * 8;
    const int cnt = (int)max(0LL, min(8LL, t.n - i0));
    const bool vec = t.vec && cnt == 8;
    const int pt = kPlain ? PT : t.pt, gt = kPlain ? GT : t.gt;
    void* const copy = kPlain ? nullptr : t.copy;
    float p[8], g[8], m[8], u[8];
    if (vec) {
      in.g.get(gt, g);
      in.p.get(pt, p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] = k < cnt ? load1(t.g, gt, i0 + k) : 0.0f;
        p[k] = k < cnt ? load1(t.p, pt, i0 + k) : 0.0f;
      }
    }
    if constexpr (kQ8) {
      unsigned w[4] = {in.cm.x, in.cm.y, in.cv.x, in.cv.y};
      if (!vec) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cnt) {
            w[k >> 2] |= (unsigned)((const unsigned char*)t.m)[i0 + k] << (8 * (k & 3));
            w[2 + (k >> 2)] |= (unsigned)((const unsigned char*)t.v)[i0 + k] << (8 * (k & 3));
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        put(m, k, mul2(e4m3x2_to_f32((unsigned short)(w[k >> 1] >> (16 * (k & 1)))), both(in.ms)));
        const float2 y = mul2(e4m3x2_to_f32((unsigned short)(w[2 + (k >> 1)] >> (16 * (k & 1)))), both(in.vs));
        put(u, k, mul2(y, y));
      }
    } else {
      if (vec) {
        in.m.get(EMB_T_F32, m);
        in.v.get(EMB_T_F32, u);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = k < cnt ? ((const float*)t.m)[i0 + k] : 0.0f;
          u[k] = k < cnt ? ((const float*)t.v)[i0 + k] : 0.0f;
        }
      }
    }
    if (kAhead && unit + 8 < end) {
      lo = tensor_of(unit + 8, lo);
      fetch(unit + 8, lo);
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 gk = !kPlain && a.grad_scale ? mul2(pair(g, k), both(gs)) : pair(g, k);
      const float2 mk = add2(mul2(pair(m, k), both(a.beta1)), a.one, mul2(gk, both(a.omb1)));
      const float2 vk = add2(mul2(pair(u, k), both(a.beta2)), a.one, mul2(mul2(gk, gk), both(a.omb2)));
      const float2 uk = make_float2(__fsqrt_rn(vk.x), __fsqrt_rn(vk.y));
      const float2 den = add2(mul2(uk, both(a.rc2)), a.one, both(a.eps)), num = mul2(mk, both(a.lr_c1));
      const float2 quo = make_float2(__fdiv_rn(num.x, den.x), __fdiv_rn(num.y, den.y));
      put(p, k, add2(quo, -a.one, mul2(pair(p, k), both(a.decay))));
      put(m, k, mk);
      put(v, k, vk);
      put(u, k, uk);
    }
    if (vec) {
      store8(t.p, pt, i0, p);
      if (copy) store8(copy, t.ct, i0, p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < cnt) {
          store1(t.p, pt, i0 + k, p[k]);
          if (copy) store1(copy, t.ct, i0 + k, p[k]);
        }
    }
    if constexpr (kQ8) {
      float am = 0.0f, au = 0.0f;  // elements past the end are zeros, and so are their moments
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        am = max_nan(am, fabsf(m[k]));
        au = max_nan(au, u[k]);
      }
      unsigned bm = warp_max(am), bu = warp_max(au);
      const bool finite = max(bm, bu) < 0x7f800000u;  // the same in all lanes
      if (!finite) {
        am = au = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          am = fmaxf(am, finite_abs(m[k]));
          au = fmaxf(au, finite_abs(u[k]));
        }
        bm = warp_max(am);
        bu = warp_max(au);
      }
      am = fmaxf(__uint_as_float(bm), kAmaxFloor);
      au = fmaxf(__uint_as_float(bu), kAmaxFloor);
      const float im = inv_of(am), iu = inv_of(au);
      const unsigned long long e0 = (unsigned long long)(t.first + i0);  // a multiple of eight: the upper half is the same for all eight
      const unsigned mix = ((unsigned)(e0 >> 32) * 0x9e3779b9u) ^ a.key;
      float qm[8], qu[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned rx = fmix32(((unsigned)e0 + 2 * k) ^ mix), ry = fmix32(((unsigned)e0 + 2 * k + 1) ^ mix);
        const float2 xm = mul2(pair(m, k), both(im));
        const float2 rm = round_random(make_float2(fabsf(xm.x), fabsf(xm.y)), a.one, ((rx & 0xffffu) << 4) + 8u, ((ry & 0xffffu) << 4) + 8u);
        put(qm, k, make_float2(copysignf(rm.x, xm.x), copysignf(rm.y, xm.y)));
        const float2 ru = round_random(mul2(pair(u, k), both(iu)), a.one, ((rx >> 16) << 4) + 8u, ((ry >> 16) << 4) + 8u);
        put(qu, k, make_float2(fmaxf(ru.x, u[2 * k] > 0.0f ? 0.001953125f : 0.0f), fmaxf(ru.y, u[2 * k + 1] > 0.0f ? 0.001953125f : 0.0f)));
      }
      if (!finite) {  // such a value would have carried out of its bits: it becomes the code NaN
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!finite_f32(m[k])) qm[k] = __uint_as_float(0x7fc00000u);
          if (!finite_f32(u[k])) qu[k] = __uint_as_float(0x7fc00000u);
        }
      }
      unsigned wm[2], wu[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        wm[k] = e4m3x2(qm[4 * k], qm[4 * k + 1]) | (e4m3x2(qm[4 * k + 2], qm[4 * k + 3]) << 16);
        wu[k] = e4m3x2(qu[4 * k], qu[4 * k + 1]) | (e4m3x2(qu[4 * k + 2], qu[4 * k + 3]) << 16);
      }
      if (vec) {
        *reinterpret_cast<uint2*>((unsigned char*)t.m + i0) = make_uint2(wm[0], wm[1]);
        *reinterpret_cast<uint2*>((unsigned char*)t.v + i0) = make_uint2(wu[0], wu[1]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cnt) {
            ((unsigned char*)t.m)[i0 + k] = (unsigned char)(wm[k >> 2] >> (8 * (k & 3)));
            ((unsigned char*)t.v)[i0 + k] = (unsigned char)(wu[k >> 2] >> (8 * (k & 3)));
          }
      }
      if (lane == 0) {
        t.ms[blk] = scale_of(am);
        t.vs[blk] = scale_of(au);
      }
    } else {
      if (vec) {
        store8(t.m, EMB_T_F32, i0, m);
        store8(t.v, EMB_T_F32, i0, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cnt) {
            ((float*)t.m)[i0 + k] = m[k];
            ((float*)t.v)[i0 + k] = v[k];
          }
      }
    }
  }
}

const char* bad_tensor(const emb_adamw_tensor& t, const void* g, bool q8) {
  if (t.n < 0 || t.first < 0 || t.first % EMB_ADAM_BLOCK) return "n is negative, or first no multiple of 256";
  if (!good_ftype(t.param_t) || !good_ftype(t.grad_t)) return "bad element type";
  if (t.copy_d && (t.param_t != EMB_T_F32 || (t.copy_t != EMB_T_BF16 && t.copy_t != EMB_T_F16)))
    return "a copy is bf16 or f16 of float32 weights";
  if (t.n == 0) return nullptr;
  if (!t.param_d || !g || !t.m_d || !t.v_d) return "param, grad, m or v is NULL";
  if (q8 && (!t.m_scale_d || !t.v_scale_d)) return "8-bit states need their scales";
  const size_t st = q8 ? 1 : 4;
  if (!aligned_to(t.param_d, ftype_bytes(t.param_t)) || !aligned_to(g, ftype_bytes(t.grad_t)) ||
      !aligned_to(t.m_d, st) || !aligned_to(t.v_d, st) || !aligned_to(t.copy_d, 2) || !aligned_to(t.m_scale_d, 4) ||
      !aligned_to(t.v_scale_d, 4))
    return "an array is not aligned to its elements";
  return nullptr;
}

template <bool kQ8, int N>
cudaError_t launch(const emb_adamw_tensor* ts, const void* const* grads, int n, const emb_adamw_params* p,
                   unsigned n_units, cudaStream_t st) {
  StepArgs<N> a;
  unsigned unit = 0;
  a.n_tensors = 0;
  for (int i = 0; i < n; ++i) {
    const emb_adamw_tensor& t = ts[i];
    if (t.n == 0) continue;
    TensorArg& o = a.t[a.n_tensors++];
    o = {t.param_d, t.copy_d, grads[i], t.m_d, t.v_d, t.m_scale_d, t.v_scale_d, t.n, t.first, unit,
         (unsigned char)t.param_t, (unsigned char)t.grad_t, (unsigned char)t.copy_t, 0};
    const size_t sb = kQ8 ? 8 : 32;  // eight elements of a state
    o.vec = aligned_to(t.param_d, 8 * ftype_bytes(t.param_t)) && aligned_to(grads[i], 8 * ftype_bytes(t.grad_t)) &&
            aligned_to(t.m_d, sb) && aligned_to(t.v_d, sb) && aligned_to(t.copy_d, 16);
    unit += (unsigned)((t.n + EMB_ADAM_BLOCK - 1) / EMB_ADAM_BLOCK);
  }
  if (a.n_tensors == 0) return cudaSuccess;
  const double c1 = 1.0 - std::pow(p->beta1, (double)p->step), c2 = 1.0 - std::pow(p->beta2, (double)p->step);
  a.n_units = n_units;
  a.beta1 = (float)p->beta1;
  a.omb1 = (float)(1.0 - p->beta1);
  a.beta2 = (float)p->beta2;
  a.omb2 = (float)(1.0 - p->beta2);
  a.decay = (float)(1.0 - p->lr * p->weight_decay);
  a.lr_c1 = (float)(p->lr / c1);
  a.rc2 = (float)(1.0 / std::sqrt(c2));
  a.eps = (float)p->eps;
  a.one = 1.0f;
  a.key = p->seed * 0x9e3779b9u + (unsigned)p->step * 0x85ebca6bu;
  a.grad_scale = p->grad_scale_d;
  // a block takes up to 64 consecutive units (8 a warp), fewer when that would leave SMs without one
  const unsigned blocks_wanted = 6u * (unsigned)sm_count();
  a.span = 8;
  while (a.span < 64 && n_units / (2 * a.span) >= blocks_wanted) a.span *= 2;
  const int grid = (int)((n_units + a.span - 1) / a.span);
  bool same = a.grad_scale == nullptr;
  const int pt = a.t[0].pt, gt = a.t[0].gt;
  for (int i = 0; i < a.n_tensors && same; ++i) same = a.t[i].pt == pt && a.t[i].gt == gt && !a.t[i].copy;
  if (same && pt == EMB_T_F32 && gt == EMB_T_F32) adamw_kernel<kQ8, N, EMB_T_F32, EMB_T_F32><<<grid, 256, 0, st>>>(a);
  else if (same && pt == EMB_T_F32 && gt == EMB_T_BF16) adamw_kernel<kQ8, N, EMB_T_F32, EMB_T_BF16><<<grid, 256, 0, st>>>(a);
  else if (same && pt == EMB_T_BF16 && gt == EMB_T_BF16) adamw_kernel<kQ8, N, EMB_T_BF16, EMB_T_BF16><<<grid, 256, 0, st>>>(a);
  else if (same && pt == EMB_T_F16 && gt == EMB_T_F16) adamw_kernel<kQ8, N, EMB_T_F16, EMB_T_F16><<<grid, 256, 0, st>>>(a);
  else adamw_kernel<kQ8, N, -1, -1><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace emb

using namespace emb;

extern "C" emb_status emb_adamw_step(const emb_adamw_tensor* tensors, const void* const* grads, int32_t n_tensors,
                                     const emb_adamw_params* params, void* stream) {
  if (!params || n_tensors < 0 || (n_tensors > 0 && (!tensors || !grads)))
    return fail(EMB_ERR_INVALID_ARG, "params, tensors or grads is NULL, or n_tensors negative");
  const emb_adamw_params& p = *params;
  if (!(p.lr >= 0) || !(p.weight_decay >= 0) || !(p.beta1 >= 0 && p.beta1 < 1) || !(p.beta2 >= 0 && p.beta2 < 1) ||
      !(p.eps > 0) || !std::isfinite(p.lr) || !std::isfinite(p.weight_decay) || !std::isfinite(p.eps))
    return fail(EMB_ERR_INVALID_ARG, "need lr, weight_decay >= 0, 0 <= beta < 1, eps > 0");
  if (!((float)p.eps > 0)) return fail(EMB_ERR_INVALID_ARG, "eps is zero in float32");
  if (p.step < 1) return fail(EMB_ERR_INVALID_ARG, "step counts from 1");
  if (p.state != EMB_ADAM_F32 && p.state != EMB_ADAM_Q8) return fail(EMB_ERR_INVALID_ARG, "bad state kind");
  const bool q8 = p.state == EMB_ADAM_Q8;
  for (int i = 0; i < n_tensors; ++i) {
    if (const char* why = bad_tensor(tensors[i], grads[i], q8))
      return fail(EMB_ERR_INVALID_ARG, "tensor " + std::to_string(i) + ": " + why);
    if (tensors[i].n / EMB_ADAM_BLOCK >= 0x7fffff00LL) return fail(EMB_ERR_UNSUPPORTED, "a tensor has over 2^39 elements");
  }
  constexpr int kFew = 40, kSome = 120, kMany = 380;
  static_assert(sizeof(StepArgs<kFew>) <= 4096 && sizeof(StepArgs<kMany>) <= 32764, "kernel parameters");
  int done = 0;
  while (done < n_tensors) {
    // as many tensors as one launch takes: 380, or fewer so that units stay below 2^31
    int k = done;
    long long units = 0;
    while (k < n_tensors && k - done < kMany) {
      const long long u = (tensors[k].n + EMB_ADAM_BLOCK - 1) / EMB_ADAM_BLOCK;
      if (k > done && units + u > 0x7fffff00LL) break;
      units += u;
      ++k;
    }
    const emb_adamw_tensor* t = tensors + done;
    const void* const* g = grads + done;
    cudaError_t e;
    if (k - done <= kFew)
      e = q8 ? launch<true, kFew>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream)
             : launch<false, kFew>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream);
    else if (k - done <= kSome)
      e = q8 ? launch<true, kSome>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream)
             : launch<false, kSome>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream);
    else
      e = q8 ? launch<true, kMany>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream)
             : launch<false, kMany>(t, g, k - done, params, (unsigned)units, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "adamw_kernel launch");
    done = k;
  }
  return EMB_OK;
}
