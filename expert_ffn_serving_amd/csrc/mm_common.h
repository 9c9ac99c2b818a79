// What the kernels that multiply matrices share: types, activations, the groups' tiles, the epilogue, LDS barriers and
// launch limits.
#pragma once

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "eff_internal.h"

namespace eff {
namespace {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;
typedef bf16_t bf16x8_t __attribute__((ext_vector_type(8)));
typedef f16_t f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec8;
template <>
struct Vec8<bf16_t> { typedef bf16x8_t V; };
template <>
struct Vec8<f16_t> { typedef f16x8_t V; };

// ---- activations (fp32) ------------------------------------------------------------------------------

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// e^x to about 2 units in the last place, and 0 below 2^-126 (v_exp_f32 gives no subnormal numbers), for any x that is not
// NaN: 2^(x log2 e), the product's rounding error put back.  (expf and an IEEE division took two thirds of the time of the
// pass over dz.)
__device__ inline float exp_f32(float x) {
  x = fminf(fmaxf(x, -104.f), 89.f);  // past both ends the result is 0 or infinity anyway
  const float t = x * 1.44269504088896341f, lo = fmaf(x, 1.44269504088896341f, -t) + x * 1.92596299e-8f;
  return __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.693147180559945309f, 1.0f);
}
// The sigmoid of v from h = e^(-|v|/2): 1 / (1 + h^2), times h^2 where v < 0.  v_rcp_f32, good to one unit in the last place,
// gets numbers in [1, 2]; 1 / (1 + e^-v) is below 2^-126 for v < -87.3, where it would give 0.
struct Sigmoid {
  float h, r;
  bool pos;
  __device__ explicit Sigmoid(float v) : h(exp_f32(-0.5f * fabsf(v))), r(__builtin_amdgcn_rcpf(fmaf(h, h, 1.0f))), pos(v >= 0.f) {}
  __device__ float value() const { return pos ? r : h * h * r; }
  // z times it, of which z * h * h may still be a normal number where h * h is none
  __device__ float times(float z) const { return pos ? z * r : z * h * (h * r); }
};
// NaN gives 0 (or 1), and stays NaN through the factor z that every use has
__device__ inline float sigmoid(float z) { return Sigmoid(z).value(); }
__device__ inline float act_silu(float z) { return Sigmoid(z).times(z); }
__device__ inline float act_one(int act, float z) {
  switch (act) {
    case EFF_ACT_SILU: return act_silu(z);
    case EFF_ACT_GELU: return 0.5f * z * erfcf(-z * kInvSqrt2);
    case EFF_ACT_GELU_TANH: return Sigmoid(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)).times(z);  // (1 + tanh u) / 2 = sigmoid(2u)
    default: return z;
  }
}
// d silu / dz = s + z s (1 - s), s the sigmoid.  Where s (1 - s) is 0 its product with a large z is 0 too.
__device__ inline float dact_silu(float z, float s) {
  const float t = s * (1.0f - s);
  return t > 0.f ? fmaf(z, t, s) : z == z ? s : z;
}
__device__ inline float dact_one(int act, float z) {
  switch (act) {
    case EFF_ACT_SILU: return dact_silu(z, sigmoid(z));
    case EFF_ACT_GELU: {
      const float g = expf(-0.5f * z * z) * kInvSqrt2Pi, p = 0.5f * erfcf(-z * kInvSqrt2);
      return g > 0.f ? fmaf(z, g, p) : p;
    }
    case EFF_ACT_GELU_TANH: {
      const float s = sigmoid(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)), t = s * (1.0f - s);
      return t > 0.f ? fmaf(z * t, 2.0f * kSqrt2OverPi * fmaf(3.0f * kGeluCubic * z, z, 1.0f), s) : z == z ? s : z;
    }
    default: return 1.0f;
  }
}

// ---- groups ------------------------------------------------------------------------------------------

__device__ inline int64_t clamp_offset(int64_t v, int64_t m) { return v < 0 ? 0 : v > m ? m : v; }
// rows of group e: [lo, hi) inside [0, m) whatever the offsets hold
__device__ inline void group_rows(const int32_t* offsets, int e, int64_t m, int64_t* lo, int64_t* hi) {
  *lo = clamp_offset(offsets[e], m);
  *hi = max(*lo, clamp_offset(offsets[e + 1], m));
}

// The row tile `tile` of the groups' tiles in group order (BM rows each, every group's last one ragged): its group and
// rows, or false past the last.  All threads of the workgroup take part; s: 20 ints of LDS, free again on return.
// Tiles are numbered without gaps, so the launch's spare workgroups come last, where they cost nothing (numbered by
// rows, with the spare ones in between and no scan, 16 tokens over 512 experts took 107 us and not 91).
template <int BM>
__device__ inline bool find_tile(const int32_t* offsets, int E, int64_t m, int tile, int* s, int* group, int64_t* row0,
                                 int64_t* row1) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nt = blockDim.x;
  const int per = (E + nt - 1) / nt, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    int64_t lo, hi;
    group_rows(offsets, e, m, &lo, &hi);
    mine += (int)((hi - lo + BM - 1) / BM);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) s[wave] = incl;
  if (tid == 0) s[16] = -1;
  __syncthreads();
  int at = incl - mine;
  for (int i = 0; i < wave; ++i) at += s[i];
  if (tile >= at && tile < at + mine) {
    for (int e = e0; e < e1; ++e) {
      int64_t lo, hi;
      group_rows(offsets, e, m, &lo, &hi);
      const int n = (int)((hi - lo + BM - 1) / BM);
      if (tile < at + n) {
        s[16] = e;
        s[17] = (int)(lo + (int64_t)(tile - at) * BM);
        s[18] = (int)min(hi, lo + (int64_t)(tile - at + 1) * BM);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  *group = s[16];
  *row0 = s[17];
  *row1 = s[18];
  __syncthreads();
  return *group >= 0;
}

// ---- epilogue of CL consecutive columns n.. of row m -----------------------------------------------------
// z: the sums (SwiGLU: gate, u: up); nb: the group's place in bias; yo: its place in y.  With a.vec every row of
// bias, residual, pre and y is a whole number of CL-wide vectors.

template <typename T, int CL>
__device__ inline void get_cl(const void* p, int64_t i, int left, bool vec, float* o) {
  typedef T V __attribute__((ext_vector_type(CL)));
  const T* s = reinterpret_cast<const T*>(p) + i;
  if (vec) {
    const V v = *reinterpret_cast<const V*>(s);
#pragma unroll
    for (int e = 0; e < CL; ++e) o[e] = (float)v[e];
  } else if (left == CL) {  // no branch between the loads
#pragma unroll
    for (int e = 0; e < CL; ++e) o[e] = (float)s[e];
  } else {
#pragma unroll
    for (int e = 0; e < CL; ++e) o[e] = e < left ? (float)s[e] : 0.f;
  }
}
template <typename T, int CL>
__device__ inline void put_cl(void* p, int64_t i, int left, bool vec, const float* v, bool stream = false) {
  typedef T V __attribute__((ext_vector_type(CL)));
  T* d = reinterpret_cast<T*>(p) + i;
  if (vec) {
    V o;
#pragma unroll
    for (int e = 0; e < CL; ++e) o[e] = (T)v[e];
    if (stream) __builtin_nontemporal_store(o, reinterpret_cast<V*>(d));
    else *reinterpret_cast<V*>(d) = o;
  } else {
#pragma unroll
    for (int e = 0; e < CL; ++e)
      if (e < left) d[e] = (T)v[e];
  }
}

// what the epilogue reads for CL columns (n < N): bias (SwiGLU: of both halves) and residual; zeros where there is none
template <int CL>
struct Extra {
  float bias[CL], up[CL], residual[CL];
};
template <typename T, int CL, bool GLU>
__device__ inline void mm_fetch(const MmArgs& a, int64_t m, int64_t n, int64_t nb, Extra<CL>* x) {
  const int left = (int)min((int64_t)CL, a.N - n);
  if (a.bias) {
    get_cl<T, CL>(a.bias, nb + n, left, a.vec, x->bias);
    if (GLU) get_cl<T, CL>(a.bias, nb + a.N + n, left, a.vec, x->up);
  }
  if (a.residual) get_cl<T, CL>(a.residual, m * a.ldr + n, left, a.vec, x->residual);
}
template <typename T, int CL, bool GLU>
__device__ inline void mm_apply(const MmArgs& a, int64_t m, int64_t n, int64_t yo, float* z, float* u, const Extra<CL>& x) {
  const int left = (int)min((int64_t)CL, a.N - n);
  const bool vec = a.vec;
  if (a.bias) {
#pragma unroll
    for (int e = 0; e < CL; ++e) {
      z[e] += x.bias[e];
      if (GLU) u[e] += x.up[e];
    }
  }
  if (a.pre) {
    put_cl<T, CL>(a.pre, m * a.ldp + n, left, vec, z);
    if (GLU) put_cl<T, CL>(a.pre, m * a.ldp + a.N + n, left, vec, u);
  }
#pragma unroll
  for (int e = 0; e < CL; ++e) z[e] = GLU ? act_silu(z[e]) * u[e] : act_one(a.act, z[e]);
  if (a.residual) {
#pragma unroll
    for (int e = 0; e < CL; ++e) z[e] += x.residual[e];
  }
  const int64_t o = yo + m * a.ldy + n;
  if (a.y_f32) put_cl<float, CL>(a.y, o, left, vec, z, a.stream);
  else put_cl<T, CL>(a.y, o, left, vec, z, a.stream);
}
template <typename T, int CL, bool GLU>
__device__ inline void mm_finish(const MmArgs& a, int64_t m, int64_t n, int64_t nb, int64_t yo, float* z, float* u) {
  if (n >= a.N) return;
  Extra<CL> x;
  mm_fetch<T, CL, GLU>(a, m, n, nb, &x);
  mm_apply<T, CL, GLU>(a, m, n, yo, z, u, x);
}

// ---- LDS ----------------------------------------------------------------------------------------------

__device__ const uint4 g_zero16[1] = {{0u, 0u, 0u, 0u}};  // what a copy past the last k reads

// this wave's LDS reads are done, then every wave's; nothing moves across
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ---- launches ----------------------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// tiles of BM rows over the groups at most
int64_t group_tiles(int64_t M, int64_t groups, int64_t BM) { return M / BM + std::min(groups, M); }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// whether one launch holds so many workgroups: its threads stay below 2^32
bool fits(int64_t workgroups, int threads) { return workgroups * threads < (int64_t)1 << 32; }

bool aligned16(std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> sizes, int bytes) {
  for (const void* p : ptrs)
    if ((uintptr_t)p % 16) return false;
  for (int64_t v : sizes)
    if (v * bytes % 16) return false;
  return true;
}

// lets a kernel use `bytes` of dynamic LDS, once per device (a bit each; calls may race, the attribute is the same)
hipError_t allow_lds(const void* fn, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (done->load(std::memory_order_acquire) & bit) return hipSuccess;
  err = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == hipSuccess) done->fetch_or(bit, std::memory_order_release);
  return err;
}

}  // namespace
}  // namespace eff
