// Dense and grouped products with bias, activation and residual in the epilogue, and their gradients.
//
// Everything is one form, y[m,n] = sum_k x(m,k) w(n,k): the forward product (x, W), dx (dz, W^T) and dw
// (dz^T, x^T) differ in the strides of the two operands.  Products of 16-bit values are exact in fp32 and
// the matrix cores add them in fp32; each output is rounded once.
#include <algorithm>

#include "eff_internal.h"

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

__device__ inline float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
__device__ inline float act_silu(float z) { return z / (1.0f + expf(-z)); }
__device__ inline float act_one(int act, float z) {
  switch (act) {
    case EFF_ACT_SILU: return act_silu(z);
    case EFF_ACT_GELU: return 0.5f * z * erfcf(-z * kInvSqrt2);
    case EFF_ACT_GELU_TANH: return z * sigmoid(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));  // (1 + tanh u) / 2 = sigmoid(2u)
    default: return z;
  }
}
// d silu / dz = s + z s (1 - s).  Where s (1 - s) is 0 its product with a large z is 0 too.
__device__ inline float dact_silu(float z) {
  const float s = sigmoid(z), t = s * (1.0f - s);
  return t > 0.f ? fmaf(z, t, s) : s;
}
__device__ inline float dact_one(int act, float z) {
  switch (act) {
    case EFF_ACT_SILU: return dact_silu(z);
    case EFF_ACT_GELU: {
      const float g = expf(-0.5f * z * z) * kInvSqrt2Pi, p = 0.5f * erfcf(-z * kInvSqrt2);
      return g > 0.f ? fmaf(z, g, p) : p;
    }
    case EFF_ACT_GELU_TANH: {
      const float s = sigmoid(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)), t = s * (1.0f - s);
      return t > 0.f ? fmaf(z * t, 2.0f * kSqrt2OverPi * fmaf(3.0f * kGeluCubic * z, z, 1.0f), s) : s;
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

// The row tile `tile` of the groups' tiles in group order (BM rows each, every group's last one ragged):
// its group and rows, or false past the last.  All threads of the workgroup (NT of them) take part.
template <int BM, int NT>
__device__ inline bool find_tile(const int32_t* offsets, int E, int64_t m, int tile, int* s, int* group, int64_t* row0,
                                 int64_t* row1) {
  // s: NT/64 + 4 ints of LDS
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (E + NT - 1) / NT, e0 = min(E, tid * per), e1 = min(E, e0 + per);
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
  if (tid == 0) s[NT / 64] = -1;
  __syncthreads();
  int before = incl - mine;
  for (int i = 0; i < wave; ++i) before += s[i];
  if (tile >= before && tile < before + mine) {
    int at = before;
    for (int e = e0; e < e1; ++e) {
      int64_t lo, hi;
      group_rows(offsets, e, m, &lo, &hi);
      const int n = (int)((hi - lo + BM - 1) / BM);
      if (tile < at + n) {
        s[NT / 64] = e;
        s[NT / 64 + 1] = (int)(lo + (int64_t)(tile - at) * BM);
        s[NT / 64 + 2] = (int)min(hi, lo + (int64_t)(tile - at + 1) * BM);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  *group = s[NT / 64];
  *row0 = s[NT / 64 + 1];
  *row1 = s[NT / 64 + 2];
  return *group >= 0;
}

template <typename T>
__device__ inline float ld(const void* p, int64_t i) { return (float)reinterpret_cast<const T*>(p)[i]; }

// ---- any strides, any alignment ------------------------------------------------------------------------
// Workgroup = 64 rows x 64 columns (SwiGLU: 32 gate and 32 up columns), 4 waves of 32 x 32, 32 k at a time
// staged through registers with every bound checked.
constexpr int kAnyBM = 64, kAnyBN = 64, kAnyBK = 32, kAnyLD = kAnyBK + 8;

template <typename T, bool GLU>
__global__ void __launch_bounds__(256)
k_mm_any(MmArgs a) {
  typedef typename Vec8<T>::V V8;
  __shared__ T s_x[kAnyBM][kAnyLD], s_w[kAnyBN][kAnyLD];
  __shared__ int s_f[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane >> 4, r = lane & 15;
  constexpr int NC = GLU ? kAnyBN / 2 : kAnyBN;  // output columns of the tile
  const int nt = (int)((a.N + NC - 1) / NC), tile = blockIdx.x / nt;
  const int64_t n0 = (int64_t)(blockIdx.x % nt) * NC;
  int g = 0;
  int64_t m0, m1, k0 = 0, k1 = a.K;
  if (a.mode == MM_ROW_GROUPS) {
    if (!find_tile<kAnyBM, 256>(a.offsets, a.groups, a.M, tile, s_f, &g, &m0, &m1)) return;
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
  for (int64_t kb = k0; kb < k1; kb += kAnyBK) {
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      const int i = z * 256 + tid;
      // consecutive lanes along whichever index is contiguous in memory
      int rr = a.sxk == 1 ? i / kAnyBK : i % kAnyBM, kk = a.sxk == 1 ? i % kAnyBK : i / kAnyBM;
      T v = (T)0.f;
      if (m0 + rr < m1 && kb + kk < k1) v = x[(m0 + rr) * a.sxm + (kb + kk) * a.sxk];
      s_x[rr][kk] = v;
      rr = a.swk == 1 ? i / kAnyBK : i % kAnyBN;
      kk = a.swk == 1 ? i % kAnyBK : i / kAnyBN;
      v = (T)0.f;
      // tile columns: per wave 32, with SwiGLU 16 gate then 16 up
      const int64_t c = GLU ? n0 + (rr >> 5) * 16 + (rr & 15) : n0 + rr;
      const int64_t wr = c + (GLU && (rr & 16) ? a.N : 0);
      if (c < a.N && kb + kk < k1) v = w[wr * a.swn + (kb + kk) * a.swk];
      s_w[rr][kk] = v;
    }
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
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm + i * 16 + r;
    if (m >= m1) continue;
#pragma unroll
    for (int j = 0; j < (GLU ? 1 : 2); ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t n = GLU ? n0 + (wn >> 1) + 4 * q + c : n0 + wn + j * 16 + 4 * q + c;
        if (n >= a.N) continue;
        const int64_t nb = (int64_t)g * (GLU ? 2 * a.N : a.N);
        float z = acc[i][j][c], y;
        if (a.bias) z += ld<T>(a.bias, nb + n);
        if (a.pre) reinterpret_cast<T*>(a.pre)[m * a.ldp + n] = (T)z;
        if (GLU) {
          float u = acc[i][1][c];
          if (a.bias) u += ld<T>(a.bias, nb + a.N + n);
          if (a.pre) reinterpret_cast<T*>(a.pre)[m * a.ldp + a.N + n] = (T)u;
          y = act_silu(z) * u;
        } else {
          y = act_one(a.act, z);
        }
        if (a.residual) y += ld<T>(a.residual, m * a.ldr + n);
        const int64_t o = (a.mode == MM_K_GROUPS ? g * a.syg : 0) + m * a.ldy + n;
        if (a.y_f32) reinterpret_cast<float*>(a.y)[o] = y;
        else reinterpret_cast<T*>(a.y)[o] = (T)y;
      }
  }
}

// ---- dz and dbias --------------------------------------------------------------------------------------

// dz = dy * act'(pre) at (m, n) in fp32; SwiGLU: the gate's and the up's
template <typename T, typename D>
__device__ inline float dz_at(const MmGrad& a, int64_t m, int64_t n, float* up) {
  const float d = ld<D>(a.dy, m * a.ldy + n);
  if (a.act == EFF_ACT_SWIGLU) {
    const float gate = ld<T>(a.pre, m * a.ldp + n), u = ld<T>(a.pre, m * a.ldp + a.N + n);
    *up = d * act_silu(gate);
    return d * u * dact_silu(gate);
  }
  return a.act == EFF_ACT_NONE ? d : d * dact_one(a.act, ld<T>(a.pre, m * a.ldp + n));
}

// grid: (ceil(N / 256), rows).  dz rounded to T: the operand that dx and dw multiply.
template <typename T, typename D>
__global__ void __launch_bounds__(256)
k_mm_dz(MmGrad a) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  T* dz = reinterpret_cast<T*>(a.dz);
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    float up = 0.f;
    const float v = dz_at<T, D>(a, m, n, &up);
    dz[m * a.lddz + n] = (T)v;
    if (a.act == EFF_ACT_SWIGLU) dz[m * a.lddz + a.N + n] = (T)up;
  }
}

// grid: (ceil(N / 64), groups).  Column sums of dz over the group's rows: 4 waves take every fourth row, then
// their sums meet in wave order.
template <typename T, typename D>
__global__ void __launch_bounds__(256)
k_mm_dbias(MmGrad a) {
  __shared__ float s[2][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  int64_t lo = 0, hi = a.M;
  if (a.offsets) group_rows(a.offsets, blockIdx.y, a.M, &lo, &hi);
  float sum = 0.f, sup = 0.f;
  if (n < a.N)
    for (int64_t m = lo + wave; m < hi; m += 4) {
      float up = 0.f;
      sum += dz_at<T, D>(a, m, n, &up);
      sup += up;
    }
  s[0][wave][lane] = sum;
  s[1][wave][lane] = sup;
  __syncthreads();
  if (wave || n >= a.N) return;
  T* db = reinterpret_cast<T*>(a.dbias) + (int64_t)blockIdx.y * (a.act == EFF_ACT_SWIGLU ? 2 * a.N : a.N);
  db[n] = (T)((s[0][0][lane] + s[0][1][lane]) + (s[0][2][lane] + s[0][3][lane]));
  if (a.act == EFF_ACT_SWIGLU) db[a.N + n] = (T)((s[1][0][lane] + s[1][1][lane]) + (s[1][2][lane] + s[1][3][lane]));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// row tiles of BM rows: dense, or at most this many over the groups
int64_t row_tiles(const MmArgs& a, int64_t BM) {
  return a.mode == MM_ROW_GROUPS ? a.M / BM + std::min<int64_t>(a.groups, a.M) : ceil_div(a.M, BM);
}

// workgroups of one launch: their threads stay below 2^32
constexpr int64_t kMaxTiles = (int64_t)1 << 22;

}  // namespace

hipError_t launch_matmul(const MmArgs& a, hipStream_t s) {
  const bool glu = a.act == EFF_ACT_SWIGLU;
  const int64_t tiles = ceil_div(a.N, glu ? kAnyBN / 2 : kAnyBN) * row_tiles(a, kAnyBM);
  if (tiles > kMaxTiles) return hipErrorInvalidConfiguration;
  const dim3 g((unsigned)tiles, a.mode == MM_K_GROUPS ? (unsigned)a.groups : 1u);
  auto go = [&](auto t) {
    typedef decltype(t) T;
    if (glu) hipLaunchKernelGGL((k_mm_any<T, true>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_mm_any<T, false>), g, dim3(256), 0, s, a);
  };
  if (a.dtype == EFF_DT_BF16) go(bf16_t{});
  else go(f16_t{});
  return hipGetLastError();
}

hipError_t launch_matmul_dz(const MmGrad& a, hipStream_t s) {
  auto go = [&](auto t, auto d) {
    typedef decltype(t) T;
    typedef decltype(d) D;
    if (a.dz && a.M > 0)
      hipLaunchKernelGGL((k_mm_dz<T, D>), dim3((unsigned)ceil_div(a.N, 256), (unsigned)std::min<int64_t>(a.M, 65535)), dim3(256),
                         0, s, a);
    if (a.dbias)
      hipLaunchKernelGGL((k_mm_dbias<T, D>), dim3((unsigned)ceil_div(a.N, 64), (unsigned)(a.offsets ? a.groups : 1)), dim3(256), 0,
                         s, a);
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
