// Microscaled 4-bit floats: rows of e2m1 codes with one power of two (e8m0) for 32 values, to and from 16 and 32 bits, and
// the products of such rows.
//
// A row of k values is padded with zeros to whole units of 128, one matrix instruction's worth: 64 bytes of codes (value
// 2i in the low bits of byte i) and 4 bytes of scales each.  Of a block with largest magnitude m the scale is 2^s,
// s = floor(log2 m) - 2 (2 being the exponent of 6, the largest e2m1), within [-127, 127], stored as s + 127; a code is the
// value times 2^-s rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, 6 beyond.  A block with an
// infinity or a NaN gets the scale byte 255 and stands for NaN.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "eff_internal.h"
#include "lds_dma.h"
#include "mm_common.h"

namespace eff {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---- rows to 4 bits and back -----------------------------------------------------------------------------

constexpr int kNaNScale = 255;

// The block exponent's byte from the bits of the largest magnitude (fp32, below infinity).  A subnormal number's exponent
// is below -126, and -127 is the least there is.
__device__ inline int mx4_scale(uint32_t largest) {
  return largest >= 0x7f800000u ? kNaNScale : max((int)(largest >> 23) - 2, 0);
}
// 2^-(scale - 127) for a scale byte up to 252 (no fp32 number has a larger one)
__device__ inline float mx4_inverse(int scale) { return __uint_as_float((uint32_t)(254 - min(scale, 252)) << 23); }

// the e2m1 code of v: nearest, ties to even, 6 beyond
__device__ inline uint32_t mx4_code(float v) {
  const float a = fabsf(v);
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
  return c | (__float_as_uint(v) >> 31 << 3);
}
// the value of a code times 2^(scale - 127); scale 255: NaN
__device__ inline float mx4_value(uint32_t code, int scale) {
  const uint32_t m = code & 7;
  const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126) << 23 | (m & 1) << 22);
  const float v = scale == kNaNScale ? __builtin_nanf("") : mag * (scale ? __uint_as_float((uint32_t)scale << 23) : 0x1p-127f);
  return code & 8 ? -v : v;
}

// 16 threads a unit, 8 consecutive values each, 4 threads a block.  grid: ceil(rows * units / 16).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_mx4_quantize(Mx4Rows a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, u = i >> 4;
  if (u >= a.rows * a.units) return;
  const int64_t row = u / a.units;
  const int unit = (int)(u - row * a.units), part = threadIdx.x & 15;
  if (a.offsets && (a.row0 + row < a.offsets[0] || a.row0 + row >= a.offsets[a.groups])) return;  // rows in no group are not read
  const int64_t k0 = (int64_t)unit * 128 + part * 8;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx + k0;
  float v[8];
  if (VEC && k0 + 8 <= a.k) {
    typedef T V8 __attribute__((ext_vector_type(8)));
    const V8 r = *reinterpret_cast<const V8*>(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)r[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k0 + e < a.k ? (float)x[e] : 0.f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  const int scale = mx4_scale(top);
  const float inv = mx4_inverse(scale);
  uint32_t c = 0;
  if (scale != kNaNScale) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c |= mx4_code(v[e] * inv) << (4 * e);
  }
  *reinterpret_cast<uint32_t*>(a.codes + row * a.ldc + (int64_t)unit * 64 + part * 4) = c;
  if ((part & 3) == 0) a.scales[row * a.lds + (int64_t)unit * 4 + (part >> 2)] = (uint8_t)scale;
}

// the same threads back
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_mx4_dequantize(Mx4Rows a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, u = i >> 4;
  if (u >= a.rows * a.units) return;
  const int64_t row = u / a.units;
  const int unit = (int)(u - row * a.units), part = threadIdx.x & 15;
  const int64_t k0 = (int64_t)unit * 128 + part * 8;
  if (k0 >= a.k) return;
  const uint32_t c = *reinterpret_cast<const uint32_t*>(a.codes + row * a.ldc + (int64_t)unit * 64 + part * 4);
  const int scale = a.scales[row * a.lds + (int64_t)unit * 4 + (part >> 2)];
  T* y = reinterpret_cast<T*>(a.y) + row * a.ldy + k0;
  typedef T V8 __attribute__((ext_vector_type(8)));
  V8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (T)mx4_value(c >> (4 * e) & 15, scale);
  if (VEC && k0 + 8 <= a.k) {
    *reinterpret_cast<V8*>(y) = r;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e < a.k) y[e] = r[e];
  }
}

// ---- products --------------------------------------------------------------------------------------------

// 16 W rows against 16 x rows over 128 k: lane (r, q) holds the 32 values of block q of row r and their scale (the low byte).
// The sums: W rows 4 q .. 4 q + 3 of x row r.
__device__ inline f32x4_t mfma4(i32x4_t w, i32x4_t x, f32x4_t c, int sw, int sx) {
  const i32x8_t a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1), b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, sw, 0, sx);
}

// Workgroup = 64 rows x 64 columns (SwiGLU: 32 gate and 32 up columns), 4 waves of 32 x 32, operands straight from memory.
constexpr int kMxBM = 64, kMxBN = 64;

template <typename T, bool GLU>
__global__ void __launch_bounds__(256)
k_mx4_any(Mx4Args a) {
  __shared__ int s_find[20];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane >> 4, r = lane & 15;
  constexpr int NC = GLU ? kMxBN / 2 : kMxBN;
  const MmArgs& m_ = a.e;
  const int nt = (int)((m_.N + NC - 1) / NC), tile = blockIdx.x / nt;
  const int64_t n0 = (int64_t)(blockIdx.x % nt) * NC;
  int g = 0;
  int64_t m0 = (int64_t)tile * kMxBM, m1 = min(m_.M, m0 + kMxBM);
  if (m_.mode == MM_ROW_GROUPS && !find_tile<kMxBM>(m_.offsets, m_.groups, m_.M, tile, s_find, &g, &m0, &m1)) return;
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  const uint8_t *x[2], *xs[2], *w[2], *ws[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = min(m0 + wm + i * 16 + r, m1 - 1);
    x[i] = a.x + row * a.ldx + q * 16;
    xs[i] = a.xs + row * a.ldxs + q;
    // columns of the wave: 32, with SwiGLU 16 gate then 16 up
    const int64_t c = min(GLU ? n0 + (wn >> 1) + r : n0 + wn + i * 16 + r, m_.N - 1), wr = c + (GLU && i ? m_.N : 0);
    w[i] = a.w + g * a.sw + wr * a.ldw + q * 16;
    ws[i] = a.ws + g * a.sws + wr * a.ldws + q;
  }
  f32x4_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int u = 0; u < a.units; ++u) {
    i32x4_t fx[2], fw[2];
    int sx[2], sw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fx[i] = *reinterpret_cast<const i32x4_t*>(x[i] + (int64_t)u * 64);
      fw[i] = *reinterpret_cast<const i32x4_t*>(w[i] + (int64_t)u * 64);
      sx[i] = xs[i][(int64_t)u * 4];
      sw[i] = ws[i][(int64_t)u * 4];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma4(fw[j], fx[i], acc[i][j], sw[j], sx[i]);
  }
  const int64_t nb = (int64_t)g * (GLU ? 2 * m_.N : m_.N);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm + i * 16 + r;
    if (m >= m1) continue;
#pragma unroll
    for (int j = 0; j < (GLU ? 1 : 2); ++j) {
      const int64_t n = GLU ? n0 + (wn >> 1) + 4 * q : n0 + wn + j * 16 + 4 * q;
      float z[4], u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[c] = acc[i][j][c];
        if (GLU) u[c] = acc[i][1][c];
      }
      mm_finish<T, 4, GLU>(m_, m, n, nb, 0, z, u);
    }
  }
}

}  // namespace

int64_t mx4_units(int64_t k) { return ceil_div(k, 128); }

namespace {

// calls f(type, rows) over parts of the rows that a grid holds (its threads stay below 2^32)
template <typename F>
void over_rows(const Mx4Rows& a, int64_t x_bytes, F f) {
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 27) / a.units);
  for (int64_t r = 0; r < a.rows; r += most) {
    Mx4Rows p = a;
    p.row0 = r, p.rows = std::min(most, a.rows - r);
    if (a.x) p.x = static_cast<const char*>(a.x) + r * a.ldx * x_bytes;
    if (a.y) p.y = static_cast<char*>(a.y) + r * a.ldy * x_bytes;
    p.codes = a.codes + r * a.ldc, p.scales = a.scales + r * a.lds;
    f(p, dim3((unsigned)ceil_div(p.rows * a.units, 16)));
  }
}
template <typename F>
void with_row_type(int dtype, F f) {
  if (dtype == EFF_DT_BF16) f(bf16_t{});
  else if (dtype == EFF_DT_F16) f(f16_t{});
  else f(float{});
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4Rows& a, hipStream_t s) {
  with_row_type(a.dtype, [&](auto t) {
    typedef decltype(t) T;
    const bool vec = (uintptr_t)a.x % (8 * sizeof(T)) == 0 && a.ldx % 8 == 0;  // 8 values at a time
    over_rows(a, sizeof(T), [&](const Mx4Rows& p, dim3 g) {
      if (vec) hipLaunchKernelGGL((k_mx4_quantize<T, true>), g, dim3(256), 0, s, p);
      else hipLaunchKernelGGL((k_mx4_quantize<T, false>), g, dim3(256), 0, s, p);
    });
  });
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4Rows& a, hipStream_t s) {
  with_row_type(a.dtype, [&](auto t) {
    typedef decltype(t) T;
    const bool vec = (uintptr_t)a.y % (8 * sizeof(T)) == 0 && a.ldy % 8 == 0;
    over_rows(a, sizeof(T), [&](const Mx4Rows& p, dim3 g) {
      if (vec) hipLaunchKernelGGL((k_mx4_dequantize<T, true>), g, dim3(256), 0, s, p);
      else hipLaunchKernelGGL((k_mx4_dequantize<T, false>), g, dim3(256), 0, s, p);
    });
  });
  return hipGetLastError();
}

bool mx4_matmul_fits(const Mx4Args& a) {
  const int64_t nw = a.e.act == EFF_ACT_SWIGLU ? 2 * a.e.N : a.e.N;
  const int64_t rows = a.e.mode == MM_ROW_GROUPS ? group_tiles(a.e.M, a.e.groups, kMxBM) : ceil_div(a.e.M, kMxBM);
  return fits(ceil_div(nw, kMxBN) * rows, 256);
}

int64_t mx4_matmul_workspace(const Mx4Args&) { return 0; }

hipError_t launch_mx4_matmul(const Mx4Args& in, void*, hipStream_t s) {
  Mx4Args a = in;
  MmArgs& e = a.e;
  e.vec = aligned16({e.y, e.bias, e.residual, e.pre}, {e.N, e.ldy, e.residual ? e.ldr : 0, e.pre ? e.ldp : 0}, 2);
  const bool glu = e.act == EFF_ACT_SWIGLU;
  const int64_t rows = e.mode == MM_ROW_GROUPS ? group_tiles(e.M, e.groups, kMxBM) : ceil_div(e.M, kMxBM);
  const dim3 g((unsigned)(ceil_div(e.N, glu ? kMxBN / 2 : kMxBN) * rows));
  auto go = [&](auto t) {
    typedef decltype(t) T;
    if (glu) hipLaunchKernelGGL((k_mx4_any<T, true>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_mx4_any<T, false>), g, dim3(256), 0, s, a);
  };
  if (e.dtype == EFF_DT_BF16) go(bf16_t{});
  else go(f16_t{});
  return hipGetLastError();
}

}  // namespace eff
