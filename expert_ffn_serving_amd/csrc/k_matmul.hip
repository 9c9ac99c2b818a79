// Dense and grouped products with bias, activation and residual in the epilogue, and their gradients.
//
// Everything is one form, y[m,n] = sum_k x(m,k) w(n,k): the forward product (x, W), dx (dz, W^T) and dw
// (dz^T, x^T) differ in the strides of the two operands.  Products of 16-bit values are exact in fp32 and
// the matrix cores add them in fp32; each output is rounded once.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "eff_internal.h"
#include "lds_dma.h"

namespace eff {
namespace {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;
typedef bf16_t bf16x8_t __attribute__((ext_vector_type(8)));
typedef f16_t f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ inline f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x4_t mfma(f16x8_t a, f16x8_t b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
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

// ---- any strides, any alignment ------------------------------------------------------------------------
// Workgroup = 64 rows x 64 columns (SwiGLU: 32 gate and 32 up columns), 4 waves of 32 x 32, 32 k at a time
// staged through registers with every bound checked.
constexpr int kAnyBM = 64, kAnyBN = 64, kAnyBK = 32, kAnyLD = kAnyBK + 8;

template <typename T, bool GLU>
__global__ void __launch_bounds__(256)
k_mm_any(MmArgs a) {
  typedef typename Vec8<T>::V V8;
  __shared__ T s_x[kAnyBM][kAnyLD], s_w[kAnyBN][kAnyLD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane >> 4, r = lane & 15;
  constexpr int NC = GLU ? kAnyBN / 2 : kAnyBN;  // output columns of the tile
  const int nt = (int)((a.N + NC - 1) / NC), tile = blockIdx.x / nt;
  const int64_t n0 = (int64_t)(blockIdx.x % nt) * NC;
  int g = 0;
  int64_t m0, m1, k0 = 0, k1 = a.K;
  if (a.mode == MM_ROW_GROUPS) {
    if (!find_tile<kAnyBM>(a.offsets, a.groups, a.M, tile, reinterpret_cast<int*>(s_x), &g, &m0, &m1)) return;
  } else {
    m0 = (int64_t)tile * kAnyBM;
    m1 = min(a.M, m0 + kAnyBM);
    if (a.mode == MM_K_GROUPS) {
      g = blockIdx.y;
      group_rows(a.offsets, g, a.K, &k0, &k1);
    }
  }
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* w = reinterpret_cast<const T*>(a.w) + (a.mode == MM_ROW_GROUPS ? g * a.swg : 0);
  f32x4_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  T vx[8], vw[8];
  // this thread's values of the step at kb; consecutive lanes along whichever index is contiguous in memory
  auto place = [&](int z, int along_k, int rows, int* rr, int* kk) {
    const int i = z * 256 + tid;
    *rr = along_k ? i / kAnyBK : i % rows;
    *kk = along_k ? i % kAnyBK : i / rows;
  };
  auto load = [&](int64_t kb) {
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      int rr, kk;
      place(z, a.xk, kAnyBM, &rr, &kk);
      vx[z] = (T)0.f;
      if (m0 + rr < m1 && kb + kk < k1) vx[z] = x[(m0 + rr) * a.sxm + (kb + kk) * a.sxk];
      place(z, a.wk, kAnyBN, &rr, &kk);
      // tile columns: per wave 32, with SwiGLU 16 gate then 16 up
      const int64_t c = GLU ? n0 + (rr >> 5) * 16 + (rr & 15) : n0 + rr;
      const int64_t wr = c + (GLU && (rr & 16) ? a.N : 0);
      vw[z] = (T)0.f;
      if (c < a.N && kb + kk < k1) vw[z] = w[wr * a.swn + (kb + kk) * a.swk];
    }
  };
  if (k0 < k1) load(k0);
  for (int64_t kb = k0; kb < k1; kb += kAnyBK) {
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      int rr, kk;
      place(z, a.xk, kAnyBM, &rr, &kk);
      s_x[rr][kk] = vx[z];
      place(z, a.wk, kAnyBN, &rr, &kk);
      s_w[rr][kk] = vw[z];
    }
    if (kb + kAnyBK < k1) load(kb + kAnyBK);  // in flight while this step's products run
    __syncthreads();
    V8 fx[2], fw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fx[i] = *reinterpret_cast<const V8*>(&s_x[wm + i * 16 + r][q * 8]);
      fw[i] = *reinterpret_cast<const V8*>(&s_w[wn + i * 16 + r][q * 8]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma(fw[j], fx[i], acc[i][j]);
    __syncthreads();
  }
  // lane: row m = wm + 16 i + r, columns 16 j + 4 q + c of its wave
  const int64_t nb = (int64_t)g * (GLU ? 2 * a.N : a.N);
  const int64_t yo = a.mode == MM_K_GROUPS ? g * a.syg : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm + i * 16 + r;
    if (m >= m1) continue;
    const float back = unscale<T>(a, g, m);
#pragma unroll
    for (int j = 0; j < (GLU ? 1 : 2); ++j) {
      const int64_t n = GLU ? n0 + (wn >> 1) + 4 * q : n0 + wn + j * 16 + 4 * q;
      float z[4], u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[c] = acc[i][j][c] * back;
        if (GLU) u[c] = acc[i][1][c];
      }
      mm_finish<T, 4, GLU>(a, m, n, nb, yo, z, u);
    }
  }
}

// ---- aligned operands: tiles through LDS ---------------------------------------------------------------
//
// Workgroup = BM rows x BN columns, WM x WN waves of (BM/WM) x (BN/WN), BK k per step.  Both operands go to LDS by
// direct 16-byte copies (no registers), S steps deep; one barrier per step.  An operand is either k-contiguous
// (LDS: rows of BK k) or contiguous along its own index (LDS: BK rows of BM or BN values, read back transposed by
// ds_read_b64_tr_b16: lane l of a group of 16 gets value l%4 of the 8 bytes that lanes l/4, 4 + l/4, .. address).
// A copy writes LDS in lane order, so bank conflicts are avoided by permuting which 16 bytes a lane fetches: chunk c
// of a row sits at chunk c ^ f(row), f chosen so that the lanes that read together hit different banks (conflicts: 1 % of LDS cycles).
// k past the end is fetched from 16 zero bytes on both sides; rows and columns past the end repeat the last ones, and
// their sums are dropped.
//
// The weights are the matrix core's first operand, so a lane holds 4 consecutive columns of one row per product;
// with k-contiguous weights the LDS rows are dealt to the products so that a lane's columns of all of them are
// consecutive.
//
// Measured: 8192^3 814 us, 1350 TFLOP/s (the library's product 1575 in the same run), 4096^3 114 us (103); the three layouts
// within 7 %.  The
// matrix cores are busy 68 % of the time at 1.8 GHz (the library's 92 % at 1.5 GHz: both run into the power limit); the
// rest is the step's barrier and the workgroups' starts and epilogues, 14 us of a 256 x 256 tile's 64 at 2048 k.  Steps
// of 32 k of 256-row tiles fetch half lines, twice the L2 requests (8192^3 954 us and not 922 when it was tried).  256 experts x 48 rows (4096 ->
// 2 x 2048, SwiGLU) are bound by the 8.6 GB of weights: 1.67 ms, 5.2 TB/s of the 6.4 that a plain read reaches; 32-row,
// 128-row and 256-column tiles, other depths and steps of 32 or 128 k took 1.69 to 2.6 ms.
__device__ const uint4 g_zero16[1] = {{0u, 0u, 0u, 0u}};  // what a copy past the last k reads

// this wave's LDS reads are done, then every wave's; nothing moves across
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

__device__ inline s16x4_t read_tr(const void* lds) {
  typedef __attribute__((address_space(3))) s16x4_t* P;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)lds);
}

// 16-byte chunk `phys` of LDS row `row` holds the row's chunk phys ^ swizzle
// (k-contiguous operand of BK k a row, whose rows are read 16 at a time, as 4 rows of each of 4 runs of GRP rows with
// GRP > 1: 8 lanes hit 8 different 16-byte places of the 128 bytes of all banks)
template <int BK, int GRP>
__device__ inline int swz_rows(int row) {
  if (BK == 32) return GRP == 1 ? (row >> 1) & 3 : ((row >> 1) & 1) | (((row / GRP) & 1) << 1);
  return GRP == 1 ? row & 7 : (row & 3) | (((row / GRP) & 1) << 2);
}
// operand contiguous along its index, LDS row = k: pairs of chunks (32 bytes) move
__device__ inline int swz_k(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

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

template <typename T, class C, bool XK, bool WK, bool GLU>
__global__ void __launch_bounds__(C::TH)
k_mm_tile(MmArgs a) {
  typedef typename Vec8<T>::V V8;
  constexpr int BM = C::BM, BN = C::BN, S = C::S, TH = C::TH, BK = C::BK, KS = BK / 32, CK = BK / 8;
  constexpr int TM = BM / C::WM, TN = BN / C::WN, MT = TM / 16, NT = TN / 16;
  constexpr int HALVES = GLU ? 2 : 1, NTH = NT / HALVES, TNH = TN / HALVES, BNH = BN / HALVES;
  constexpr int RUN = NTH * 4;                       // a lane's consecutive columns (k-contiguous weights)
  constexpr int XB = BM * BK * 2, WB = BN * BK * 2, STEP = XB + WB;
  constexpr int SX = BM * CK / TH, SW = BN * CK / TH, CP = SX + SW;  // copies of one thread per step
  static_assert(BM * CK % TH == 0 && BN * CK % TH == 0 && NT % HALVES == 0, "tile");
  extern __shared__ __attribute__((aligned(128))) uint8_t s_tile[];
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;

  // which tile
  const int nt = (int)((a.N + BNH - 1) / BNH);
  int g = 0, mt_i, nt_i;
  int64_t m0, m1, k0 = 0, k1 = a.K;
  if (a.mode == MM_ROW_GROUPS) {
    mt_i = blockIdx.x / nt;
    nt_i = blockIdx.x % nt;
    if (!find_tile<BM>(a.offsets, a.groups, a.M, mt_i, reinterpret_cast<int*>(s_tile), &g, &m0, &m1)) return;
  } else {
    // Workgroups go to the 8 XCDs in turn, each with its own L2: an XCD takes a contiguous part of the tiles, in bands of
    // 8 row tiles walked column by column, so that the tiles it has in flight share rows of x and of W.
    const int all = gridDim.x, xcd = blockIdx.x & 7, id = xcd * (all >> 3) + min(xcd, all & 7) + (blockIdx.x >> 3);
    const int mts = all / nt, band = id / (8 * nt), in_band = id - band * 8 * nt, height = min(8, mts - band * 8);
    mt_i = band * 8 + in_band % height;
    nt_i = in_band / height;
    m0 = (int64_t)mt_i * BM;
    m1 = min(a.M, m0 + BM);
    if (a.mode == MM_K_GROUPS) {
      g = blockIdx.y;
      group_rows(a.offsets, g, a.K, &k0, &k1);
    } else if (a.part) {  // this split's share of the k
      k0 = (int64_t)blockIdx.y * a.split_steps * 64;
      k1 = min(a.K, k0 + (int64_t)a.split_steps * 64);
    }
  }
  const int64_t n0 = (int64_t)nt_i * BNH;

  // this thread's copies: byte offsets from a uniform address that advances with the steps (plan_matmul keeps them < 2^32)
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* w = reinterpret_cast<const T*>(a.w) + (a.mode == MM_ROW_GROUPS ? g * a.swg : 0);
  const int64_t xcols = a.x_padded ? (a.M + 7) & ~(int64_t)7 : a.M;  // x contiguous along m
  const int64_t wcols = a.w_padded ? (a.N + 7) & ~(int64_t)7 : a.N;  // w contiguous along n
  const char* bx = reinterpret_cast<const char*>(XK ? x + m0 * a.sxm + k0 : x + k0 * a.sxk + m0);
  const char* bw = reinterpret_cast<const char*>(WK ? w + n0 * a.swn + k0 : w + k0 * a.swk + n0);
  uint32_t ox[SX], ow[SW];
  int kx[SX], kw[SW];  // the copy's first k inside a step
#pragma unroll
  for (int i = 0; i < SX; ++i) {
    const int idx = i * TH + tid;
    if (XK) {
      const int row = idx / CK, c = (idx % CK) ^ swz_rows<BK, 1>(row);
      kx[i] = c * 8;
      ox[i] = (uint32_t)((min((int64_t)row, m1 - 1 - m0) * a.sxm + c * 8) * 2);
    } else {
      constexpr int CH = BM / 8;
      const int k = idx / CH, p = idx % CH, c = ((((p >> 1) ^ swz_k(k)) << 1) | (p & 1)) % CH;
      kx[i] = k;
      ox[i] = (uint32_t)((k * a.sxk + min((int64_t)c * 8, xcols - 8 - m0)) * 2);
    }
  }
#pragma unroll
  for (int i = 0; i < SW; ++i) {
    const int idx = i * TH + tid;
    if (WK) {
      const int row = idx / CK, c = (idx % CK) ^ swz_rows<BK, RUN>(row);
      const int col = (row / TN) * TNH + (row % TNH);
      kw[i] = c * 8;
      ow[i] = (uint32_t)((min((int64_t)col, a.N - 1 - n0) * a.swn + c * 8) * 2);
    } else {
      constexpr int CH = BN / 8;
      const int k = idx / CH, p = idx % CH, c = ((((p >> 1) ^ swz_k(k)) << 1) | (p & 1)) % CH;
      kw[i] = k;
      ow[i] = (uint32_t)((k * a.swk + min((int64_t)c * 8, wcols - 8 - n0)) * 2);
    }
  }
  const int64_t stepx = XK ? BK * 2 : a.sxk * (BK * 2), stepw = WK ? BK * 2 : a.swk * (BK * 2);
  const int64_t up_rows = GLU ? a.N * a.swn * 2 : 0;  // bytes from gate to up rows
  const uint32_t lds0 = lds_address(s_tile);
  const int64_t klen = k1 - k0;
  const int steps = (int)((klen + BK - 1) / BK);

  auto issue = [&](int t) {
    const uint32_t base = lds0 + (t % S) * STEP + wave * 1024;
    const int left = (int)min((int64_t)BK, klen - (int64_t)t * BK);
    const char *sx = bx + t * stepx, *sw = bw + t * stepw;
    // a wave copies whole rows, on one side of a tile's gate and up rows
    auto side = [&](int i) { return GLU && ((i * TH + wave * 64) / CK) % TN >= TNH ? sw + up_rows : sw; };
    if (left == BK) {
#pragma unroll
      for (int i = 0; i < SX; ++i) lds_copy16(sx, ox[i], base + i * (TH * 16));
#pragma unroll
      for (int i = 0; i < SW; ++i) lds_copy16(side(i), ow[i], base + XB + i * (TH * 16));
    } else {
      const char* zero = reinterpret_cast<const char*>(g_zero16);
#pragma unroll
      for (int i = 0; i < SX; ++i) lds_copy16(kx[i] < left ? sx + ox[i] : zero, base + i * (TH * 16));
#pragma unroll
      for (int i = 0; i < SW; ++i) lds_copy16(kw[i] < left ? side(i) + ow[i] : zero, base + XB + i * (TH * 16));
    }
  };

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto frag_x = [&](const uint8_t* b, int i, int ks) -> V8 {
    if (XK) {
      const int row = wm * TM + i * 16 + r;
      return *reinterpret_cast<const V8*>(b + row * (BK * 2) + (((ks * 4 + q) ^ swz_rows<BK, 1>(row)) << 4));
    } else {
      // lane: k row ks*32 + q*8 + r/4 (and + 4), columns 4 (r%4) of its 16
      constexpr int CH = BM / 8;
      const int k = ks * 32 + q * 8 + (r >> 2), col = wm * TM + i * 16 + (r & 3) * 4;
      const int pair = ((col >> 4) ^ swz_k(k)) % (CH / 2);
      const uint8_t* p = b + k * (BM * 2) + pair * 32 + (col & 15) * 2;
      const s16x4_t lo = read_tr(p), hi = read_tr(p + 4 * (BM * 2));
      return __builtin_bit_cast(V8, (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto frag_w = [&](const uint8_t* b, int j, int ks) -> V8 {
    if (WK) {
      const int row = wn * TN + (j / NTH) * TNH + (r >> 2) * RUN + (j % NTH) * 4 + (r & 3);
      return *reinterpret_cast<const V8*>(b + XB + row * (BK * 2) + (((ks * 4 + q) ^ swz_rows<BK, RUN>(row)) << 4));
    } else {
      constexpr int CH = BN / 8;
      const int k = ks * 32 + q * 8 + (r >> 2), col = wn * TN + j * 16 + (r & 3) * 4;
      const int pair = ((col >> 4) ^ swz_k(k)) % (CH / 2);
      const uint8_t* p = b + XB + k * (BN * 2) + pair * 32 + (col & 15) * 2;
      const s16x4_t lo = read_tr(p), hi = read_tr(p + 4 * (BN * 2));
      return __builtin_bit_cast(V8, (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };

  // this wave's copies of every step up to the last CP * N issued ones are in LDS
  auto arrived = [&](bool all) {
    if (all) vm_wait<0>();
    else vm_wait<(S - 2) * CP>();
  };
  auto buffer = [&](int t) { return s_tile + (t % S) * STEP; };

#pragma unroll
  for (int t = 0; t < S - 1; ++t)
    if (t < steps) issue(t);
  if constexpr (C::AHEAD) {
    // One wave's products hide its LDS reads: an x operand is read again for the next half step as soon as its products
    // are issued, the w operands are read one half step ahead into a second set (both in a second set spill).  The barrier
    // of a step stands inside the last half's products, when the reads before it have long returned.  8192^3: 1350 to
    // 1374 TFLOP/s (with 1 to 6 operands before the barrier, or raised priority: the same); each half's reads before its products 1137, two groups of waves taking turns at LDS and the matrix cores 1312.
    static_assert(KS == 2 && S == 2, "two halves, two buffers");
    constexpr int LATE = 2;  // x operands whose products stand before the barrier
    V8 fw[2][NT], fx[MT];
    auto products = [&](int from, int i) {
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma(fw[from][j], fx[i], acc[i][j]);
    };
    auto read_w = [&](int into, const uint8_t* b, int ks) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fw[into][j] = frag_w(b, j, ks);
    };
    if (steps > 0) {
      arrived(true);
      meet();
      if (steps > 1) issue(1);
      read_w(0, buffer(0), 0);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[i] = frag_x(buffer(0), i, 0);
      for (int t = 0; t < steps - 1; ++t) {
        const uint8_t *b = buffer(t), *next = buffer(t + 1);
        read_w(1, b, 1);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          products(0, i);
          fx[i] = frag_x(b, i, 1);
        }
#pragma unroll
        for (int i = 0; i < LATE; ++i) products(1, i);
        arrived(true);
        meet();                      // step t + 1 is in LDS and step t in registers
        if (t + 2 < steps) issue(t + 2);
        read_w(0, next, 0);
#pragma unroll
        for (int i = 0; i < LATE; ++i) fx[i] = frag_x(next, i, 0);
#pragma unroll
        for (int i = LATE; i < MT; ++i) {
          products(1, i);
          fx[i] = frag_x(next, i, 0);
        }
      }
      const uint8_t* b = buffer(steps - 1);
      read_w(1, b, 1);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        products(0, i);
        fx[i] = frag_x(b, i, 1);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) products(1, i);
    }
  } else {
    for (int t = 0; t < steps; ++t) {
      arrived(t + S - 1 > steps);
      meet();
      if (t + S - 1 < steps) issue(t + S - 1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        V8 fw[NT], fx[MT];
#pragma unroll
        for (int j = 0; j < NT; ++j) fw[j] = frag_w(buffer(t), j, ks);
#pragma unroll
        for (int i = 0; i < MT; ++i) fx[i] = frag_x(buffer(t), i, ks);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mfma(fw[j], fx[i], acc[i][j]);
      }
    }
  }

  // Epilogue through LDS, RP rows at a time: the sums change from the matrix core's layout to whole rows, so that
  // bias, residual, pre and y move as 16-byte vectors, a row's side by side.
  constexpr int LDC = BN + 4;
  constexpr int IP = rows_fit<C>(MT) ;
  constexpr int RP = C::WM * 16 * IP, VR = BNH / 8, ROUND = TH / VR;
  static_assert(TH % VR == 0 && RP % ROUND == 0, "rows of a round");
  const int64_t yo = a.mode == MM_K_GROUPS ? g * a.syg : 0;
  if (!WK && a.plain) {
    // nothing to add: straight from the registers, 4 columns of 16 rows at a time (1000^3 13.6 -> 11.8 us)
    typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int64_t m = m0 + wm * TM + i * 16 + r, n = n0 + wn * TN + q * 4;
      T* row = reinterpret_cast<T*>(a.y) + yo + m * a.ldy + n;
      if (m < m1) {
        const float back = unscale<T>(a, g, m);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          V4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (T)(acc[i][j][e] * back);
          if (n + j * 16 < a.N) *reinterpret_cast<V4*>(row + j * 16) = v;
        }
      }
    }
    return;
  }
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

// A split k's sums added in order of k, and the epilogue (333 x 515, 7 splits: 6 us, a launch and two trips to memory).  grid: ceil(M * vectors / 256); a thread takes 8 columns.
template <typename T, bool GLU>
__global__ void __launch_bounds__(256)
k_mm_join(MmArgs a, int splits) {
  const int64_t vr = (a.N + 7) / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * vr) return;
  const int64_t m = i / vr, n = i % vr * 8;
  float z[8], u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = u[e] = 0.f;
  const float* p = a.part + m * a.ldpart + n;
#pragma unroll 8
  for (int s = 0; s < splits; ++s, p += a.M * a.ldpart)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[4 * h + e] += v[e];
      if (GLU) {
        const f32x4_t v2 = *reinterpret_cast<const f32x4_t*>(p + a.ldpart / 2 + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[4 * h + e] += v2[e];
      }
    }
  const float back = unscale<T>(a, 0, m);
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] *= back;
  mm_finish<T, 8, GLU>(a, m, n, 0, 0, z, u);
}

// ---- operands that cannot be copied 16 bytes at a time ---------------------------------------------------
// rows x cols values with any stride into rows of ceil(cols / 8) * 8 values, zeros behind cols (rows = groups *
// group_rows), for both operands in one launch.  A thread writes 16 bytes.  Reading and writing the matrix once more
// is what this costs; the general kernel took 361 us where this and the tiles take 24 (333 x 515 x 2563).
struct PackJob {
  const void* src;
  void* dst;
  int64_t rows, cols, ld, group_rows, sg, blocks;
};

template <typename T>
__global__ void __launch_bounds__(256)
k_mm_pack(PackJob a, PackJob b) {
  const bool first = blockIdx.x < a.blocks;
  const PackJob& p = first ? a : b;
  const int64_t vr = (p.cols + 7) / 8, i = (int64_t)(blockIdx.x - (first ? 0 : a.blocks)) * 256 + threadIdx.x;
  if (i >= p.rows * vr) return;
  const int64_t row = i / vr, c = i % vr * 8;
  const T* s = reinterpret_cast<const T*>(p.src) + (row / p.group_rows) * p.sg + (row % p.group_rows) * p.ld + c;
  typename Vec8<T>::V v;
  if (c + 8 <= p.cols) {  // no branch between the loads
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < p.cols ? s[e] : (T)0.f;
  }
  *reinterpret_cast<typename Vec8<T>::V*>(reinterpret_cast<T*>(p.dst) + (row * vr * 8 + c)) = v;
}

// ---- few rows --------------------------------------------------------------------------------------------
//
// Up to 16 MT rows of x against 16 rows of W per workgroup (SwiGLU: 8 gate and 8 up rows), the k split over its waves:
// bound by the stream of W, so every wave keeps U chunks of 64 k (2 KiB of W each) in flight in registers and nothing
// waits for a barrier before the end, where the waves' sums meet in LDS in wave order.  The lane of W row r and k group
// q takes 32 consecutive bytes of a chunk: k = 16 q .. 16 q + 15 (the order of k inside a product is free as long as
// both operands share it), so a chunk is one 128-byte line of every row.  16 rows, 4096 -> 2 x 2048 SwiGLU: 10.2 us, 3.3
// TB/s of W (33 MB: a launch, one trip to memory and the join; two chunks in flight 12.3 us, 64 x 128 tiles 32 us).
template <int MT>
constexpr int few_unroll() { return MT == 1 ? 4 : 2; }

template <typename T, int MT, bool GLU>
__global__ void __launch_bounds__(1024)
k_mm_few(MmArgs a, int slices) {
  typedef typename Vec8<T>::V V8;
  constexpr int U = few_unroll<MT>(), BM = 16 * MT;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_few[];
  f32x4_t* s_acc = reinterpret_cast<f32x4_t*>(s_few);                       // [waves][MT][64]
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int tile = blockIdx.x / slices, n0 = (int)(blockIdx.x % slices) * (GLU ? 8 : 16);
  int g = 0;
  int64_t m0 = (int64_t)tile * BM, m1 = min(a.M, m0 + BM);
  if (a.mode == MM_ROW_GROUPS && !find_tile<BM>(a.offsets, a.groups, a.M, tile, reinterpret_cast<int*>(s_few), &g, &m0, &m1)) return;
  const T* x = reinterpret_cast<const T*>(a.x);
  const int K = (int)a.K, chunks = (int)((a.K + 63) / 64);  // k is below 2^31, the next multiple of 64 need not be
  const int64_t col = min((int64_t)n0 + (GLU ? r & 7 : r), a.N - 1);
  const T* w = reinterpret_cast<const T*>(a.w) + g * a.swg + (col + (GLU && r >= 8 ? a.N : 0)) * a.swn + q * 16;
  const T* xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = x + min(m0 + i * 16 + r, m1 - 1) * a.sxm + q * 16;
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  V8 fw[U][2], fx[U][MT][2];
  // chunk c of this wave's into slot s; past the end the first chunk again (not used)
  auto load = [&](int c, int s) {
    const int k = c < chunks ? c * 64 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = k + q * 16 + h * 8 < K ? k + h * 8 : -(q * 16);      // past the last k: the row's first values
      fw[s][h] = *reinterpret_cast<const V8*>(w + kk);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[s][i][h] = *reinterpret_cast<const V8*>(xr[i] + kk);
    }
  };
  auto use = [&](int c, int s) {
    if (c >= chunks) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (c * 64 > K - 64 && c * 64 + q * 16 + h * 8 >= K) {              // nothing there: zeros on both sides
        fw[s][h] = V8{};
#pragma unroll
        for (int i = 0; i < MT; ++i) fx[s][i][h] = V8{};
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = mfma(fw[s][h], fx[s][i][h], acc[i]);
    }
  };
#pragma unroll
  for (int s = 0; s < U; ++s) load(wave + s * waves, s);
  // what the finishing wave's epilogue reads is on its way with the operands
  const int64_t nb = (int64_t)g * (GLU ? 2 * a.N : a.N);
  Extra<4> extra;
  if (wave < MT && m0 + wave * 16 + r < m1 && n0 + 4 * q < a.N && (!GLU || q < 2))
    mm_fetch<T, 4, GLU>(a, m0 + wave * 16 + r, n0 + 4 * q, nb, &extra);
  int c = wave;
  for (; c + U * waves < chunks; c += U * waves) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      use(c + s * waves, s);
      load(c + (s + U) * waves, s);
    }
  }
#pragma unroll
  for (int s = 0; s < U; ++s) use(c + s * waves, s);
#pragma unroll
  for (int i = 0; i < MT; ++i) s_acc[(wave * MT + i) * 64 + lane] = acc[i];
  __syncthreads();
  // one wave per 16 rows of x: lane's row m = r, W rows 4 q .. 4 q + 3 of the slice
  for (int i = wave; i < MT; i += waves) {
    const int64_t m = m0 + i * 16 + r, n = n0 + 4 * q;
    f32x4_t sum = s_acc[i * 64 + lane];
    for (int v = 1; v < waves; ++v) sum += s_acc[(v * MT + i) * 64 + lane];
    float z[4], u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[e] = sum[e];
      if (GLU) u[e] = __shfl_down(z[e], 32);
    }
    if (m < m1 && n < a.N && (!GLU || q < 2)) {
      if (i != wave) mm_fetch<T, 4, GLU>(a, m, n, nb, &extra);
      mm_apply<T, 4, GLU>(a, m, n, 0, z, u, extra);
    }
  }
}

// ---- dz and dbias --------------------------------------------------------------------------------------
//
// One pass over dy and pre: a workgroup takes ROWS rows of one group and 64 VEC columns, each of its 4 waves every
// fourth row.  It writes dz rounded to T (the operand that dx and dw multiply: the matrix cores take 16 bits, and a second
// term for the bits below would double both products, 116 and 123 us of 247 here; the gradients' error in norm is 2.3e-3 in
// bf16 where their own rounding alone makes 1.7e-3; columns up to lddz are zeroed, so that dz's rows are whole 16-byte
// vectors) and the columns' fp32 sums over its rows, which a second kernel adds up in row
// order.  Bound by HBM, every value read and written once: 4096 x 2 x 2048 SwiGLU 21 us, 4.0 TB/s.
// Rows of one workgroup: 32, or 8 where 32 leave most of the chip idle (100 rows x 640, gelu: 21 -> 8 us; with 8 rows
// everywhere the sums' second pass reads four times as much).

template <typename T, int VEC>
struct Piece {
  typedef T V __attribute__((ext_vector_type(VEC)));
};
template <typename T>
struct Piece<T, 1> {
  typedef T V;
};
template <typename T, int VEC>
__device__ inline void widen(const typename Piece<T, VEC>::V& v, float* o) {
  if constexpr (VEC == 1) {
    o[0] = (float)v;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = (float)v[e];
  }
}
template <typename T, int VEC>
__device__ inline typename Piece<T, VEC>::V piece(const void* p, int64_t i) {
  return *reinterpret_cast<const typename Piece<T, VEC>::V*>(reinterpret_cast<const T*>(p) + i);
}
template <typename T, int VEC>
__device__ inline void store_row(void* p, int64_t i, const float* v) {
  if constexpr (VEC == 1) {
    reinterpret_cast<T*>(p)[i] = (T)v[0];
  } else {
    typedef T V __attribute__((ext_vector_type(VEC)));
    V o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = (T)v[e];
    *reinterpret_cast<V*>(reinterpret_cast<T*>(p) + i) = o;
  }
}

// dz of VEC columns of a row from dy (d), the saved sums z and, with SwiGLU, u: in d, SwiGLU's second half in u
template <int VEC>
__device__ inline void dz_values(int act, float* d, const float* z, float* u) {
  if (act == EFF_ACT_SWIGLU) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float sg = sigmoid(z[e]), up = d[e] * z[e] * sg;
      d[e] = d[e] * u[e] * dact_silu(z[e], sg);
      u[e] = up;
    }
  } else if (act != EFF_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) d[e] *= dact_one(act, z[e]);
  }
}

__global__ void __launch_bounds__(256)
k_mm_zero(uint32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// The largest finite |dz| of every row (row_max) and of every column of a group (col_max), as the bits of the floats, whose
// order is theirs: integer maxima, so the order of the atomics is free.  One more pass over dy and pre, and two launches:
// fp16 gradients of 4096 rows, 4096 <-> 2 x 2048 SwiGLU take 276 us where bf16's take 247, of 1024^3 44 where 31 (a lane's
// columns taken by the lane itself, 32 bytes apart in every atomic: 316 and 62).
template <typename D, int VEC, int ROWS>
__global__ void __launch_bounds__(256)
k_mm_dz_max(MmGrad a, int cols) {
  __shared__ uint32_t s_max[2][4][64][VEC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = blockIdx.x / cols;
  const int64_t n = ((int64_t)(blockIdx.x % cols) * 64 + lane) * VEC;
  int g = 0;
  int64_t m0 = (int64_t)tile * ROWS, m1 = min(a.M, m0 + ROWS);
  if (a.offsets && !find_tile<ROWS>(a.offsets, a.groups, a.M, tile, reinterpret_cast<int*>(s_max), &g, &m0, &m1)) return;
  const bool glu = a.act == EFF_ACT_SWIGLU, live = n < a.N;
  auto magnitude = [](float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
  };
  uint32_t col[VEC], up[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) col[e] = up[e] = 0;
  for (int64_t m = m0 + wave; m < m1; m += 4) {  // the same rows for every lane of a wave
    uint32_t row = 0;
    if (live) {
      float d[VEC], z[VEC], u[VEC];
      widen<D, VEC>(piece<D, VEC>(a.dy, m * a.ldy + n), d);
      if (a.act != EFF_ACT_NONE) widen<f16_t, VEC>(piece<f16_t, VEC>(a.pre, m * a.ldp + n), z);
      if (glu) widen<f16_t, VEC>(piece<f16_t, VEC>(a.pre, m * a.ldp + a.N + n), u);
      dz_values<VEC>(a.act, d, z, u);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const uint32_t v = magnitude(d[e]), w = glu ? magnitude(u[e]) : 0u;
        col[e] = max(col[e], v), up[e] = max(up[e], w), row = max(row, max(v, w));
      }
    }
    if (a.row_max) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) row = max(row, (uint32_t)__shfl_xor((int)row, o));
      if (lane == 0) atomicMax(a.row_max + m, row);
    }
  }
  if (!a.col_max) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    s_max[0][wave][lane][e] = col[e];
    s_max[1][wave][lane][e] = up[e];
  }
  __syncthreads();
  // consecutive lanes take consecutive columns
  const int64_t n0 = (int64_t)(blockIdx.x % cols) * 64 * VEC;
  uint32_t* out = a.col_max + (int64_t)g * (glu ? 2 * a.N : a.N) + n0;
  for (int i = threadIdx.x; i < (glu ? 2 : 1) * 64 * VEC; i += 256) {
    const int h = i / (64 * VEC), c = i % (64 * VEC);
    if (n0 + c >= a.N) continue;
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) v = max(v, (&s_max[h][w][0][0])[c]);
    if (v > 0) atomicMax(out + h * a.N + c, v);
  }
}

// SCALED: with row_max, dz is scaled by rows, and with col_max dz_cols, scaled by columns, is written too
template <typename T, typename D, int VEC, int ROWS, bool SCALED>
__global__ void __launch_bounds__(256)
k_mm_dz(MmGrad a, int cols) {
  __shared__ float s_sum[2][4][64][VEC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = blockIdx.x / cols;
  const int64_t n = ((int64_t)(blockIdx.x % cols) * 64 + lane) * VEC;
  int g = 0;
  int64_t m0 = (int64_t)tile * ROWS, m1 = min(a.M, m0 + ROWS);
  if (a.offsets && !find_tile<ROWS>(a.offsets, a.groups, a.M, tile, reinterpret_cast<int*>(s_sum), &g, &m0, &m1)) return;
  const bool glu = a.act == EFF_ACT_SWIGLU;
  const int64_t nw = glu ? 2 * a.N : a.N;
  float sum[VEC], sup[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum[e] = sup[e] = 0.f;
  if (n < a.N && m0 + wave < m1) {
    // a row is in flight while the one before it is used; past the end the last row again (not used)
    typename Piece<D, VEC>::V dn;
    typename Piece<T, VEC>::V zn, un;
    auto fetch = [&](int64_t m) {
      m = min(m, m1 - 1);
      dn = piece<D, VEC>(a.dy, m * a.ldy + n);
      if (a.act != EFF_ACT_NONE) zn = piece<T, VEC>(a.pre, m * a.ldp + n);
      if (glu) un = piece<T, VEC>(a.pre, m * a.ldp + a.N + n);
    };
    float cs[VEC], us[VEC];  // SCALED: of this lane's columns
    if constexpr (SCALED) {
      if (a.col_max) {
        const uint32_t* c = a.col_max + g * nw + n;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          cs[e] = scale_to_fp16(c[e]);
          us[e] = glu ? scale_to_fp16(c[a.N + e]) : 0.f;
        }
      }
    }
    auto scaled = [](const float* v, const float* by, float one, float* o) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = v[e] * (by ? by[e] : one);
    };
    fetch(m0 + wave);
    for (int64_t m = m0 + wave; m < m1; m += 4) {
      float d[VEC], z[VEC], u[VEC];
      widen<D, VEC>(dn, d);
      if (a.act != EFF_ACT_NONE) widen<T, VEC>(zn, z);
      if (glu) widen<T, VEC>(un, u);
      fetch(m + 4);
      dz_values<VEC>(a.act, d, z, u);
      if (glu) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) sup[e] += u[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += d[e];
      if constexpr (SCALED) {
        float o[VEC];
        if (a.col_max) {
          scaled(d, cs, 0.f, o);
          store_row<T, VEC>(a.dz_cols, m * a.lddz + n, o);
          if (glu) {
            scaled(u, us, 0.f, o);
            store_row<T, VEC>(a.dz_cols, m * a.lddz + a.N + n, o);
          }
        }
        if (a.row_max) {
          const float rs = scale_to_fp16(a.row_max[m]);
          scaled(d, nullptr, rs, o);
          store_row<T, VEC>(a.dz, m * a.lddz + n, o);
          if (glu) {
            scaled(u, nullptr, rs, o);
            store_row<T, VEC>(a.dz, m * a.lddz + a.N + n, o);
          }
        }
      } else if (a.dz) {
        if (glu) store_row<T, VEC>(a.dz, m * a.lddz + a.N + n, u);
        store_row<T, VEC>(a.dz, m * a.lddz + n, d);
      }
    }
  }
  // the zeros behind a row
  if (blockIdx.x % cols == 0 && nw + lane < a.lddz)
    for (int64_t m = m0 + wave; m < m1; m += 4) {
      if (a.dz) reinterpret_cast<T*>(a.dz)[m * a.lddz + nw + lane] = (T)0.f;
      if (SCALED && a.dz_cols) reinterpret_cast<T*>(a.dz_cols)[m * a.lddz + nw + lane] = (T)0.f;
    }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    s_sum[0][wave][lane][e] = sum[e];
    s_sum[1][wave][lane][e] = sup[e];
  }
  __syncthreads();
  const int h = wave;   // wave 0: the sums, wave 1: SwiGLU's second half
  if (h > (glu ? 1 : 0) || n >= a.N) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float v = s_sum[h][0][lane][e];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += s_sum[h][w][lane][e];
    a.part[(int64_t)tile * nw + h * a.N + n + e] = v;
  }
}

// grid: (ceil(nw / 64), groups).  A group's tiles' sums added in row order by 4 waves (tile t by wave t % 4), then in
// wave order.
template <typename T>
__global__ void __launch_bounds__(256)
k_mm_dbias(MmGrad a) {
  __shared__ float s_sum[4][64];
  __shared__ int64_t s_before[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.y;
  const int64_t nw = a.act == EFF_ACT_SWIGLU ? 2 * a.N : a.N, n = (int64_t)blockIdx.x * 64 + lane;
  int64_t lo = 0, hi = a.M, first = 0;
  if (a.offsets) {  // tiles of the groups before this one
    int64_t before = 0;
    for (int i = threadIdx.x; i < e; i += 256) {
      group_rows(a.offsets, i, a.M, &lo, &hi);
      before += (hi - lo + a.rows - 1) / a.rows;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor((long long)before, o);
    if (lane == 0) s_before[wave] = before;
    __syncthreads();
    first = s_before[0] + s_before[1] + s_before[2] + s_before[3];
    group_rows(a.offsets, e, a.M, &lo, &hi);
  }
  const int64_t count = (hi - lo + a.rows - 1) / a.rows, last = min(first + count, a.tiles);
  float sum = 0.f;
  if (n < nw)
#pragma unroll 8
    for (int64_t t = first + wave; t < last; t += 4) sum += a.part[t * nw + n];
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave || n >= nw) return;
  reinterpret_cast<T*>(a.dbias)[(int64_t)e * nw + n] = (T)((s_sum[0][lane] + s_sum[1][lane]) + (s_sum[2][lane] + s_sum[3][lane]));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// row tiles of BM rows: dense, or at most this many over the groups
int64_t group_tiles(int64_t M, int64_t groups, int64_t BM) { return M / BM + std::min(groups, M); }
int64_t row_tiles(const MmArgs& a, int64_t BM) {
  return a.mode == MM_ROW_GROUPS ? group_tiles(a.M, a.groups, BM) : ceil_div(a.M, BM);
}

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

// ---- which kernel ----------------------------------------------------------------------------------------

typedef TileCfg<256, 256, 2, 4, 64, 2, true> Big;
typedef TileCfg<128, 256, 2, 4, 32, 3, false> Wide;
typedef TileCfg<128, 128, 2, 2, 64, 2, false> Mid;
typedef TileCfg<64, 128, 1, 4, 64, 3, false> Low;

struct Plan {
  int kind, splits;
  int64_t pack_x, pack_w, part;  // workspace bytes of each (multiples of 256)
};

constexpr int64_t kMaxStride = (int64_t)1 << 22;  // rows further apart are packed (a tile's 256 of them: 2^31 bytes)
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t w_rows(const MmArgs& a) { return a.act == EFF_ACT_SWIGLU ? 2 * a.N : a.N; }
// rows and contiguous values of an operand in memory
int64_t x_rows(const MmArgs& a) { return a.xk ? a.M : a.K; }
int64_t x_cols(const MmArgs& a) { return a.xk ? a.K : a.M; }
int64_t w_mem_rows(const MmArgs& a) { return (a.mode == MM_ROW_GROUPS ? a.groups : 1) * (a.wk ? w_rows(a) : a.K); }
int64_t w_cols(const MmArgs& a) { return a.wk ? a.K : a.N; }

// From sizes and strides alone (pointers that are not 16-byte aligned are the launch's business).
Plan plan_matmul(const MmArgs& a) {
  Plan p = {KIND_ANY, 1, 0, 0, 0};
  if (a.M == 0 || a.K == 0) return p;   // zeros: any kernel writes them
  const bool glu = a.act == EFF_ACT_SWIGLU;
  const int64_t groups = std::max(1, a.groups);
  // Rows of whole 16-byte vectors, or padded with zeros up to one: an x row may then be read past K against rows of w
  // that are padded too, or (w contiguous along n) masked.
  const int64_t ldx = a.xk ? a.sxm : a.sxk, ldw = a.wk ? a.swn : a.swk;
  const bool x_ok = ldx % 8 == 0 && ldx < kMaxStride && (x_cols(a) % 8 == 0 || a.x_padded);
  const bool w_ok = ldw % 8 == 0 && ldw < kMaxStride && a.swg % 8 == 0 && (w_cols(a) % 8 == 0 || a.w_padded);
  if (!x_ok) p.pack_x = up(x_rows(a) * up(x_cols(a), 8) * 2, 256);
  if (!w_ok) p.pack_w = up(w_mem_rows(a) * up(w_cols(a), 8) * 2, 256);
  // Packing copies the weights of all groups, with rows or without; the general kernel reads what it needs, value by value.
  // y and dx in us, packed and general: 8 groups of 1024 x 1025, 64 rows 18 and 23, 31 and 33; 512 rows 23 and 25, 38 and 39;
  // 64 groups, 512 rows 75 and 85, 64 and 69; 4096 rows 92 and 96, 76 and 84; 256 groups of 1024 x 2049, 160 rows 492 and 488,
  // 216 and 230; 4096 rows 611 and 604, 441 and 454; 512 groups of 640 x 2561, 160 rows 624 and 615, 146 and 119.
  if (p.pack_w && a.mode == MM_ROW_GROUPS && a.M < 16 * groups) return Plan{KIND_ANY, 1, 0, 0, 0};
  const int64_t n = w_rows(a);
  const int64_t rows = a.mode == MM_ROW_GROUPS ? a.M / std::max<int64_t>(1, std::min(groups, a.M)) : a.M;
  if (a.xk && a.wk) {
    // The tiles' waves share x, the split of k over waves fills the chip when there are few tiles.  In us, streamed and tiles:
    // 2560 -> 512, 1 row 7.1 and 9.3, 32 rows 10.7 and 10.3; 4096 -> 4096, 1 row 7.9 and 12.4, 16 rows 10.4 and 15.7, 32 rows
    // 13.9 and 13.9, 33 rows 19.9 and 13.6; 4096 -> 16384, 1 row 22.7 and 25.1, 16 rows 31 and 25, 32 rows 45 and 26; 17 rows of
    // 4096 -> 4096 16 at a time 15.6, 32 at a time 11.4.  Groups: 8 of 8 rows, 2048 -> 1024 (64 tiles) 11.6 and 18.6; with 512
    // tiles and more, 64 of 8 rows, 2048 -> 1024 54 and 44, 512 of 16 rows, 1024 -> 512 166 and 103.
    const bool fill = row_tiles(a, Low::BM) * ceil_div(n, Low::BN) >= 512;
    if (rows <= 16 && !fill) return p.kind = KIND_FEW1, p;
    if (rows <= 32 && !fill) return p.kind = KIND_FEW2, p;
  }
  // 256 x 256 tiles have the most products per byte; 128 x 256 tiles, two workgroups on a CU so that one's epilogue runs under
  // the other's products, win where sums are short; 128 x 128 and 64 x 128 fill the chip when there are few tiles and waste
  // less on experts with few rows.  Each forced everywhere, us (in this order): 4096^3 114, 145, 132, 182; 8192 x 4096 x 2048
  // 122, 142, 136, 176; 8192 x 4096 x 512 47, 47, 49, 62; 2048^3 44, 40, 29, 26; 1000^3 27, 23, 15, 12; 333 x 512 x 2560 23, 19,
  // 16, 15; 256 experts of 128 rows, 2048 <-> 1024, dw 453, 435, 515, 607 and dx 332, 275, 289, 327; of 48 rows, 4096 -> 4096
  // 2089, 1770, 1807, 1737.
  // Tiles and splits of k by an estimate of the time: rounds of workgroups over 256 CUs (`occ` on each; with one on each
  // a step is faster), 64-k steps, a workgroup's start and epilogue, and a split's sums written, read and joined.  The
  // constants (us) fit 4096^3, 8192 x 4096 x {512, 2048}, 2048^3 and 333 x 512 x 2560 to 15 %.
  struct Tile { int kind; int64_t bm, bn, bk; int occ; double alone, step, fixed; };
  const Tile tiles[] = {{KIND_BIG, Big::BM, Big::BN, Big::BK, 1, 1.55, 1.55, 14},
                        {KIND_WIDE, Wide::BM, Wide::BN, Wide::BK, 2, 1.05, 2.05, 8},
                        {KIND_MID, Mid::BM, Mid::BN, Mid::BK, 2, 0.75, 1.0, 7},
                        {KIND_LOW, Low::BM, Low::BN, Low::BK, 2, 0.42, 0.64, 6}};
  // A tile's lanes hold unsigned 32-bit byte offsets from its first element.  Packing does not shorten a row that is long
  // itself (2^23 values and 256 of them, say): such rows go to a tile of fewer, or to the general kernel.
  const int64_t ld_x = p.pack_x ? up(x_cols(a), 8) : ldx, ld_w = p.pack_w ? up(w_cols(a), 8) : ldw;
  auto reaches = [&](const Tile& t) {
    const int64_t wide = std::min(glu ? t.bn / 2 : t.bn, a.N);
    const int64_t x = a.xk ? (std::min(t.bm, a.M) - 1) * ld_x + t.bk : (t.bk - 1) * ld_x + t.bm;
    const int64_t w = a.wk ? (wide - 1) * ld_w + t.bk : (t.bk - 1) * ld_w + t.bn;
    return std::max(x, w) * 2 < (int64_t)1 << 32;
  };
  const int64_t k = a.mode == MM_K_GROUPS ? std::max<int64_t>(1, a.K / groups) : a.K, steps = ceil_div(k, 64);
  double best = 0;
  for (const Tile& t : tiles) {
    if (!reaches(t)) continue;
    double count = (double)ceil_div(n, t.bn);
    if (a.mode == MM_ROW_GROUPS) count *= std::max<double>((double)ceil_div(rows, t.bm) * std::min(groups, a.M), a.M / (double)t.bm);
    else count *= (double)ceil_div(a.M, t.bm) * (a.mode == MM_K_GROUPS ? groups : 1);
    for (int64_t s = 1; s <= 16 && (s == 1 || (a.mode == MM_DENSE && s * 4 <= steps)); ++s) {
      const double each = (double)ceil_div(steps, s), full = std::floor(count * s / (256.0 * t.occ)), rest = count * s - full * 256 * t.occ;
      double us = full * (t.step * each + t.fixed);
      if (rest > 0) us += (rest <= 256 ? t.alone : t.step) * each + t.fixed;
      if (s > 1) us += 5 + s * (double)a.M * n * 8 / 8e6;
      if (best == 0 || us < best) best = us, p.kind = t.kind, p.splits = (int)s;
    }
  }
  if (best == 0) return Plan{KIND_ANY, 1, 0, 0, 0};
  if (p.splits > 1) {
    p.splits = (int)ceil_div(steps, ceil_div(steps, p.splits));  // none empty
    p.part = up((int64_t)p.splits * a.M * (glu ? 2 : 1) * up(a.N, 8) * 4, 256);
  }
  return p;
}

template <typename T, class C, bool XK, bool WK, bool GLU>
hipError_t launch_tile_c(const MmArgs& a, int splits, hipStream_t s) {
  const int64_t tiles = ceil_div(a.N, GLU ? C::BN / 2 : C::BN) * row_tiles(a, C::BM);
  constexpr int lds = C::S * (C::BM + C::BN) * C::BK * 2;
  auto* fn = &k_mm_tile<T, C, XK, WK, GLU>;
  static std::atomic<uint64_t> done{0};
  const hipError_t set = allow_lds(reinterpret_cast<const void*>(fn), lds, &done);
  if (set != hipSuccess) return set;
  hipLaunchKernelGGL(fn, dim3((unsigned)tiles, a.mode == MM_K_GROUPS ? (unsigned)a.groups : (unsigned)splits), dim3(C::TH), lds, s, a);
  if (splits > 1)
    hipLaunchKernelGGL((k_mm_join<T, GLU>), dim3((unsigned)ceil_div(a.M * ceil_div(a.N, 8), 256)), dim3(256), 0, s, a, splits);
  return hipGetLastError();
}

template <typename T, int MT, bool GLU>
hipError_t launch_few(const MmArgs& a, hipStream_t s) {
  const int64_t slices = ceil_div(a.N, GLU ? 8 : 16), jobs = slices * row_tiles(a, 16 * MT);
  // waves per workgroup: up to 32 per CU over the launch, each with at least two chunks of k
  int waves = 16;
  while (waves > 1 && (jobs * waves > 8192 || waves * 128 > a.K + 127)) waves /= 2;
  hipLaunchKernelGGL((k_mm_few<T, MT, GLU>), dim3((unsigned)jobs), dim3(64 * waves), waves * MT * 1024, s, a, (int)slices);
  return hipGetLastError();
}

template <typename T, bool XK, bool WK, bool GLU>
hipError_t launch_kind(const MmArgs& a, const Plan& p, hipStream_t s) {
  if constexpr (XK && WK) {
    if (p.kind == KIND_FEW1) return launch_few<T, 1, GLU>(a, s);
    if (p.kind == KIND_FEW2) return launch_few<T, 2, GLU>(a, s);
  }
  if (p.kind == KIND_BIG) return launch_tile_c<T, Big, XK, WK, GLU>(a, p.splits, s);
  if (p.kind == KIND_WIDE) return launch_tile_c<T, Wide, XK, WK, GLU>(a, p.splits, s);
  if (p.kind == KIND_MID) return launch_tile_c<T, Mid, XK, WK, GLU>(a, p.splits, s);
  return launch_tile_c<T, Low, XK, WK, GLU>(a, p.splits, s);
}

template <typename T>
hipError_t launch_typed(MmArgs a, Plan p, char* ws, hipStream_t s) {
  const bool glu = a.act == EFF_ACT_SWIGLU;
  // The workspace is sized without the pointers, so an operand that only begins at an odd place is not packed.  8192 x 4096 x
  // 2048: 730 us where the tiles take 126 (packed for an odd stride: 132), its gradients 948 where 256.
  if ((!p.pack_x && (uintptr_t)a.x % 16) || (!p.pack_w && (uintptr_t)a.w % 16)) p.kind = KIND_ANY;
  if (p.kind == KIND_ANY) {
    const int64_t tiles = ceil_div(a.N, glu ? kAnyBN / 2 : kAnyBN) * row_tiles(a, kAnyBM);
    const dim3 g((unsigned)tiles, a.mode == MM_K_GROUPS ? (unsigned)a.groups : 1u);
    if (glu) hipLaunchKernelGGL((k_mm_any<T, true>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_mm_any<T, false>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (p.pack_x || p.pack_w) {
    PackJob jobs[2] = {};
    if (p.pack_x) {
      int64_t* ld = a.xk ? &a.sxm : &a.sxk;
      jobs[0] = {a.x, ws, x_rows(a), x_cols(a), *ld, x_rows(a), 0, ceil_div(x_rows(a) * ceil_div(x_cols(a), 8), 256)};
      a.x = ws, a.x_padded = 1, *ld = up(x_cols(a), 8);
    }
    if (p.pack_w) {
      int64_t* ld = a.wk ? &a.swn : &a.swk;
      const int64_t rows = a.wk ? w_rows(a) : a.K;
      jobs[1] = {a.w, ws + p.pack_x, w_mem_rows(a), w_cols(a), *ld, rows, a.swg, ceil_div(w_mem_rows(a) * ceil_div(w_cols(a), 8), 256)};
      a.w = ws + p.pack_x, a.w_padded = 1, *ld = up(w_cols(a), 8);
      a.swg = rows * *ld;
    }
    const int64_t blocks = jobs[0].blocks + jobs[1].blocks;
    hipLaunchKernelGGL((k_mm_pack<T>), dim3((unsigned)blocks), dim3(256), 0, s, jobs[0], jobs[1]);
  }
  if (p.splits > 1) {
    a.part = reinterpret_cast<float*>(ws + p.pack_x + p.pack_w);
    a.ldpart = (glu ? 2 : 1) * up(a.N, 8), a.plain = a.simple = 0;
    a.split_steps = (int)ceil_div(ceil_div(a.K, 64), p.splits);
  }
  if (a.xk && a.wk) return glu ? launch_kind<T, true, true, true>(a, p, s) : launch_kind<T, true, true, false>(a, p, s);
  return a.xk ? launch_kind<T, true, false, false>(a, p, s) : launch_kind<T, false, false, false>(a, p, s);
}

}  // namespace

MmChoice matmul_choice(const MmArgs& a) {
  const Plan p = plan_matmul(a);
  return {p.kind, p.splits, p.pack_x ? up(x_cols(a), 8) : a.xk ? a.sxm : a.sxk, p.pack_w ? up(w_cols(a), 8) : a.wk ? a.swn : a.swk};
}

bool matmul_fits(const MmArgs& a) {
  if (a.M == 0) return true;
  const Plan p = plan_matmul(a);
  const int64_t n = w_rows(a);
  // the general kernel too, which takes over where pointers are not aligned
  bool ok = fits(ceil_div(n, kAnyBN) * row_tiles(a, kAnyBM), 256);
  ok = ok && fits(ceil_div(p.pack_x, 4096) + ceil_div(p.pack_w, 4096) + 2, 256);
  if (p.kind == KIND_FEW1 || p.kind == KIND_FEW2) ok = ok && fits(ceil_div(n, 16) * row_tiles(a, 16), 1024);
  return ok;
}

bool matmul_dz_fits(int64_t M, int64_t N, int groups) {
  return fits(ceil_div(N, 64) * matmul_dz_tiles(M, N, groups), 256) && fits(ceil_div(2 * N, 64), 256);
}

int64_t matmul_workspace(const MmArgs& a) {
  const Plan p = plan_matmul(a);
  return p.pack_x + p.pack_w + p.part;
}

hipError_t launch_matmul(const MmArgs& in, void* workspace, hipStream_t s) {
  MmArgs a = in;
  a.vec = aligned16({a.y, a.bias, a.residual, a.pre}, {a.N, a.ldy, a.syg, a.residual ? a.ldr : 0, a.pre ? a.ldp : 0}, 2);
  // Outputs that no cache holds (256 MiB) are stored past it: the next kernels find their inputs there (gradients of 256
  // experts, 1 GiB of dw: 794 -> 760 us when it was tried).
  a.stream = a.M * a.N * (a.mode == MM_K_GROUPS ? a.groups : 1) * (a.y_f32 ? 4 : 2) > (int64_t)256 << 20;
  a.plain = a.vec && !a.stream && !a.bias && !a.residual && !a.pre && !a.y_f32 && a.act == EFF_ACT_NONE;
  a.simple = a.vec && !a.bias && !a.pre && !a.y_f32 && (a.act == EFF_ACT_NONE || a.act == EFF_ACT_SWIGLU);
  const Plan p = plan_matmul(a);
  char* ws = static_cast<char*>(workspace);
  return a.dtype == EFF_DT_BF16 ? launch_typed<bf16_t>(a, p, ws, s) : launch_typed<f16_t>(a, p, ws, s);
}

// rows of a workgroup in the pass over dz, and its row tiles (those of the partial sums)
static int64_t dz_tiles(int64_t M, int groups, int64_t rows) { return groups ? group_tiles(M, groups, rows) : ceil_div(M, rows); }
static int dz_rows(int64_t M, int64_t N, int groups) { return ceil_div(N, 512) * dz_tiles(M, groups, 32) < 256 ? 8 : 32; }
int64_t matmul_dz_tiles(int64_t M, int64_t N, int groups) { return dz_tiles(M, groups, dz_rows(M, N, groups)); }

hipError_t launch_matmul_dz(const MmGrad& in, hipStream_t s) {
  MmGrad a = in;
  const int groups = a.offsets ? a.groups : 0;
  a.rows = dz_rows(a.M, a.N, groups);
  a.tiles = matmul_dz_tiles(a.M, a.N, groups);
  const int64_t nw = a.act == EFF_ACT_SWIGLU ? 2 * a.N : a.N;
  const bool vec = aligned16({a.dy, a.act ? a.pre : nullptr, a.dz, a.dz_cols}, {a.N, a.ldy, a.act ? a.ldp : 0, a.lddz}, 2);
  const int64_t cols = ceil_div(a.N, vec ? 512 : 64);
  auto go = [&](auto t, auto d) {
    typedef decltype(t) T;
    typedef decltype(d) D;
    const dim3 grid((unsigned)(cols * a.tiles));
    auto pass = [&](auto width, auto rows) {
      constexpr int V = decltype(width)::value, R = decltype(rows)::value;
      if constexpr (std::is_same<T, f16_t>::value) {
        if (a.row_max || a.col_max) {
          const int64_t words = (a.row_max ? a.M : 0) + (a.col_max ? std::max(1, groups) * nw : 0);
          hipLaunchKernelGGL(k_mm_zero, dim3((unsigned)std::min<int64_t>(ceil_div(words, 256), 2048)), dim3(256), 0, s,
                             a.row_max ? a.row_max : a.col_max, words);
          hipLaunchKernelGGL((k_mm_dz_max<D, V, R>), grid, dim3(256), 0, s, a, (int)cols);
          hipLaunchKernelGGL((k_mm_dz<T, D, V, R, true>), grid, dim3(256), 0, s, a, (int)cols);
          return;
        }
      }
      hipLaunchKernelGGL((k_mm_dz<T, D, V, R, false>), grid, dim3(256), 0, s, a, (int)cols);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 8> eight;
    const std::integral_constant<int, 32> many;
    if (a.M == 0) {
    } else if (a.rows == 8) {
      if (vec) pass(eight, eight);
      else pass(one, eight);
    } else {
      if (vec) pass(eight, many);
      else pass(one, many);
    }
    if (a.dbias)
      hipLaunchKernelGGL((k_mm_dbias<T>), dim3((unsigned)ceil_div(nw, 64), (unsigned)(a.offsets ? a.groups : 1)), dim3(256), 0, s, a);
  };
  if (a.dtype == EFF_DT_BF16) {
    if (a.dy_f32) go(bf16_t{}, float{});
    else go(bf16_t{}, bf16_t{});
  } else {
    if (a.dy_f32) go(f16_t{}, float{});
    else go(f16_t{}, f16_t{});
  }
  return hipGetLastError();
}

}  // namespace eff
