// What the kernels that multiply matrices share: types, activations, the groups' tiles, the epilogue, LDS barriers and
// launch limits.
#pragma once

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

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
  *group = __builtin_amdgcn_readfirstlane(s[16]);
  *row0 = __builtin_amdgcn_readfirstlane(s[17]);
  *row1 = __builtin_amdgcn_readfirstlane(s[18]);
  __syncthreads();
  return *group >= 0;
}

// ---- fp16 operands scaled by powers of two ---------------------------------------------------------------
//
// dz of a backward pass may be far larger or smaller than fp16 holds although the gradients are not (an fp32 dy, dy * up,
// a mean over many tokens).  In fp16 it enters dx scaled per row and dw per column of its group, by the power of two that
// brings the largest finite magnitude there into [2^14, 2^15), and the sums are scaled back: both are exact, what is
// left is the rounding to 11 bits, and 2^-39 of the largest where an element is that small.  bf16 has fp32's range.
__device__ inline int top_exponent(uint32_t largest) { return max((int)(largest >> 23), 15); }  // both powers stay normal
__device__ inline float scale_to_fp16(uint32_t largest) { return __uint_as_float((uint32_t)(268 - top_exponent(largest)) << 23); }
__device__ inline float scale_back(uint32_t largest) { return __uint_as_float((uint32_t)(top_exponent(largest) - 14) << 23); }
// what the sums of output row m (of group g) are multiplied with
template <typename T>
__device__ inline float unscale(const MmArgs& a, int g, int64_t m) {
  if constexpr (std::is_same<T, f16_t>::value)
    if (a.row_max) return scale_back(a.row_max[(a.mode == MM_K_GROUPS ? g * a.M : 0) + m]);
  return 1.0f;
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

// ---- tiles through LDS ----------------------------------------------------------------------------------

// 16-byte chunk `phys` of LDS row `row` holds the row's chunk phys ^ swizzle
// (k-contiguous operand of BK k a row, whose rows are read 16 at a time, as 4 rows of each of 4 runs of GRP rows with
// GRP > 1: 8 lanes hit 8 different 16-byte places of the 128 bytes of all banks)
template <int BK, int GRP>
__device__ inline int swz_rows(int row) {
  if (BK == 32) return GRP == 1 ? (row >> 1) & 3 : ((row >> 1) & 1) | (((row / GRP) & 1) << 1);
  return GRP == 1 ? row & 7 : (row & 3) | (((row / GRP) & 1) << 2);
}
// BM x BN tile, WM x WN waves, BK k per step, S steps in LDS; AHEAD: operands are read half a step ahead (below)
template <int BM_, int BN_, int WM_, int WN_, int BK_, int S_, bool AHEAD_>
struct TileCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_, TH = 64 * WM_ * WN_;
  static constexpr bool AHEAD = AHEAD_;
};

// subtiles of 16 rows per wave that the epilogue's LDS holds at once
template <class C>
constexpr int rows_fit(int mt) {
  int ip = mt;
  while (ip > 1 && C::WM * 16 * ip * (C::BN + 4) * 4 > C::S * (C::BM + C::BN) * C::BK * 2) ip /= 2;
  return ip;
}

// A tile's sums to y: bias, activation, residual, pre.  Called by the whole workgroup; s_tile: its S steps of LDS.
template <typename T, class C, bool WK, bool GLU, int MT, int NT>
__device__ __forceinline__ void store_tile(const MmArgs& a, f32x4_t (&acc)[MT][NT], uint8_t* s_tile, int g, int64_t m0, int64_t m1, int64_t n0) {
  typedef typename Vec8<T>::V V8;
  constexpr int BN = C::BN, TH = C::TH, TM = C::BM / C::WM, TN = BN / C::WN;
  constexpr int HALVES = GLU ? 2 : 1, NTH = NT / HALVES, TNH = TN / HALVES, BNH = BN / HALVES, RUN = NTH * 4;
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  // Epilogue through LDS, RP rows at a time: the sums change from the matrix core's layout to whole rows, so that
  // bias, residual, pre and y move as 16-byte vectors, a row's side by side.
  constexpr int LDC = BN + 4;
  constexpr int IP = rows_fit<C>(MT) ;
  constexpr int RP = C::WM * 16 * IP, VR = BNH / 8, ROUND = TH / VR;
  static_assert(TH % VR == 0 && RP % ROUND == 0, "rows of a round");
  const int64_t yo = a.mode == MM_K_GROUPS ? g * a.syg : 0;
  float* s_c = reinterpret_cast<float*>(s_tile);
  const int64_t nb = (int64_t)g * (GLU ? 2 * a.N : a.N);
  const int64_t n = n0 + (tid % VR) * 8;
  constexpr int NR = RP / ROUND;
  auto row_of = [&](int p, int rr) { return m0 + (rr / (16 * IP)) * TM + p * (16 * IP) + rr % (16 * IP); };
#pragma unroll
  for (int p = 0; p < MT / IP; ++p) {
    V8 res[NR];
    if (a.simple && a.residual) {  // on its way while the sums go through LDS
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        const int64_t m = row_of(p, tid / VR + h * ROUND);
        if (m < m1 && n < a.N) res[h] = *reinterpret_cast<const V8*>(reinterpret_cast<const T*>(a.residual) + m * a.ldr + n);
      }
    }
    meet();
#pragma unroll
    for (int i = 0; i < IP; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int col = (j / NTH) * BNH + wn * TNH + (WK ? q * RUN + (j % NTH) * 4 : (j % NTH) * 16 + q * 4);
        *reinterpret_cast<f32x4_t*>(s_c + ((wm * IP + i) * 16 + r) * LDC + col) = acc[p * IP + i][j];
      }
    meet();
    // Whole vectors, no bias, nothing saved, no other activation: every round's accesses at once.  8192 x 4096 x 2048 by epilogue:
    // none 125 us, residual 134; the general rounds below: fp32 output 133, silu 142, gelu 168, bias, gelu and pre 175.
    if (a.simple) {
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        const int64_t m = row_of(p, tid / VR + h * ROUND);
        const float* c = s_c + (tid / VR + h * ROUND) * LDC + (tid % VR) * 8;
        const float back = unscale<T>(a, g, min(m, m1 - 1));
        V8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float z = c[e] * back;
          if (GLU) z = act_silu(z) * c[BNH + e];
          if (a.residual) z += (float)res[h][e];
          o[e] = (T)z;
        }
        if (m < m1 && n < a.N) {
          V8* d = reinterpret_cast<V8*>(reinterpret_cast<T*>(a.y) + yo + m * a.ldy + n);
          if (a.stream) __builtin_nontemporal_store(o, d);
          else *d = o;
        }
      }
      continue;
    }
#pragma unroll 1
    for (int rr = tid / VR; rr < RP; rr += ROUND) {
      const int64_t m = row_of(p, rr);
      if (m >= m1) continue;
      const float* c = s_c + rr * LDC + (tid % VR) * 8;
      float z[8], u[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(c + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[4 * h + e] = v[e];
        if (GLU) {
          const f32x4_t v2 = *reinterpret_cast<const f32x4_t*>(c + BNH + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) u[4 * h + e] = v2[e];
        }
      }
      if (a.part) {
        float* o = a.part + ((int64_t)blockIdx.y * a.M + m) * a.ldpart + n;
        if (n < a.N) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<f32x4_t*>(o + 4 * h) = f32x4_t{z[4 * h], z[4 * h + 1], z[4 * h + 2], z[4 * h + 3]};
            if (GLU) *reinterpret_cast<f32x4_t*>(o + a.ldpart / 2 + 4 * h) = f32x4_t{u[4 * h], u[4 * h + 1], u[4 * h + 2], u[4 * h + 3]};
          }
        }
      } else {
        const float back = unscale<T>(a, g, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= back;
        mm_finish<T, 8, GLU>(a, m, n, nb, yo, z, u);
      }
    }
  }
}

// The same straight from the registers of a tile with k-contiguous weights, where a lane's columns of a row are consecutive:
// no LDS, no barrier, accesses of up to 16 bytes of 4 lanes side by side.  SIMPLE: a.simple, and nothing else in the code.
template <typename T, class C, bool GLU, bool SIMPLE, int MT, int NT>
__device__ __forceinline__ void store_regs(const MmArgs& a, f32x4_t (&acc)[MT][NT], int g, int64_t m0, int64_t m1, int64_t n0) {
  constexpr int TM = C::BM / C::WM, TN = C::BN / C::WN, HALVES = GLU ? 2 : 1, NTH = NT / HALVES, TNH = TN / HALVES, RUN = NTH * 4;
  constexpr int CL = RUN < 8 ? RUN : 8;
  typedef T V __attribute__((ext_vector_type(CL)));
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int64_t nb = (int64_t)g * (GLU ? 2 * a.N : a.N);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = m0 + wm * TM + i * 16 + r;
    if (m >= m1) continue;
#pragma unroll
    for (int h = 0; h < RUN / CL; ++h) {
      const int64_t n = n0 + wn * TNH + q * RUN + h * CL;
      float z[CL], u[CL];
#pragma unroll
      for (int e = 0; e < CL; ++e) {
        z[e] = acc[i][(h * CL + e) / 4][e % 4];
        if (GLU) u[e] = acc[i][NTH + (h * CL + e) / 4][e % 4];
      }
      if constexpr (SIMPLE) {
        if (n >= a.N) continue;
        V o;
#pragma unroll
        for (int e = 0; e < CL; ++e) z[e] = GLU ? act_silu(z[e]) * u[e] : z[e];
        if (a.residual) {
          const V res = *reinterpret_cast<const V*>(reinterpret_cast<const T*>(a.residual) + m * a.ldr + n);
#pragma unroll
          for (int e = 0; e < CL; ++e) z[e] += (float)res[e];
        }
#pragma unroll
        for (int e = 0; e < CL; ++e) o[e] = (T)z[e];
        V* d = reinterpret_cast<V*>(reinterpret_cast<T*>(a.y) + m * a.ldy + n);
        if (a.stream) __builtin_nontemporal_store(o, d);
        else *d = o;
      } else {
        mm_finish<T, CL, GLU>(a, m, n, nb, 0, z, u);
      }
    }
  }
}

// ---- launches ----------------------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// tiles of BM rows over the groups at most
int64_t group_tiles(int64_t M, int64_t groups, int64_t BM) { return M / BM + std::min(groups, M); }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

bool fits(int64_t workgroups, int threads) { return workgroups <= most_workgroups(threads); }

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
