// Layer norm of token rows and its gradients.
//
// mu = mean x, v = mean (x - mu)^2, r = 1 / sqrt(v + eps), xh = (x - mu) r, y = xh w + b.  With g = dy w:
// dx = r (g - mean g - xh mean(g xh)) + residual, dw = sum over rows of dy xh, db = sum over rows of dy.
//
// A row stays in the registers of TH threads (NV vectors of VEC values each), so it is read once: the mean, then the
// deviations from it, whose own mean corrects the rounding of the first (y of a stream whose offset is far above its spread
// loses nothing; the gradients take xh from the saved mean, one fp32 number: an offset of 2^k spreads shifts their xh by up to
// 2^(k - 24)).  All statistics and sums are fp32; a row whose squares leave its range is scaled by a power of two.
#include <algorithm>
#include <type_traits>

#include "eff_internal.h"
#include "wave.h"

namespace eff {
namespace {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// VEC consecutive values at any place (the hardware takes 16-byte accesses at any address)
template <typename T, int VEC>
struct NormVec {
  typedef T V __attribute__((ext_vector_type(VEC)));
  typedef V Loose __attribute__((aligned(sizeof(T))));
};
template <typename T, int VEC>
__device__ inline void norm_widen(const typename NormVec<T, VEC>::V& v, float* o) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = (float)v[i];
}
// values h .. h + VEC - 1 of a row of H (h < H); WHOLE: H is a multiple of VEC, else zeros past the end
template <typename T, int VEC, bool WHOLE>
__device__ inline typename NormVec<T, VEC>::V norm_load(const void* p, int64_t i, int64_t h, int64_t H) {
  const T* s = reinterpret_cast<const T*>(p) + i + h;
  typename NormVec<T, VEC>::V v = {};
  if (WHOLE || h + VEC <= H) {
    v = *reinterpret_cast<const typename NormVec<T, VEC>::Loose*>(s);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (h + e < H) v[e] = s[e];
  }
  return v;
}
// the same of another type than the rows' (weights): as many 16-byte accesses as they take
template <typename T, int VEC, bool WHOLE>
__device__ inline void norm_get(const void* p, int64_t h, int64_t H, float* o) {
  constexpr int C = VEC * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : VEC;
#pragma unroll
  for (int c = 0; c < VEC; c += C) {
    if (WHOLE || h + c < H) {
      norm_widen<T, C>(norm_load<T, C, WHOLE>(p, 0, h + c, H), o + c);
    } else {
#pragma unroll
      for (int e = 0; e < C; ++e) o[c + e] = 0.f;
    }
  }
}
template <typename T, int VEC, bool WHOLE>
__device__ inline void norm_store(void* p, int64_t i, int64_t h, int64_t H, const float* v) {
  T* d = reinterpret_cast<T*>(p) + i + h;
  if (WHOLE || h + VEC <= H) {
    typename NormVec<T, VEC>::V o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = (T)v[e];
    *reinterpret_cast<typename NormVec<T, VEC>::Loose*>(d) = o;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (h + e < H) d[e] = (T)v[e];
  }
}

// sums of N values over the TH threads of a row (TH = 64: the wave; else the wave's sums meet in LDS, s: [TH / 64][N],
// in wave order).  Every thread of the workgroup takes part.
template <int TH, int N>
__device__ inline void row_sum(float* v, float* s) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TH > 64) {
    const int wave = (threadIdx.x % TH) >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = s[i];
#pragma unroll
    for (int w = 1; w < TH / 64; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += s[w * N + i];
  }
}

// the variance from the deviations' sums (NaN stays: a maximum drops it)
__device__ inline float variance_of(const float* dev, float inv, float more) {
  return fmaxf(dev[1] * inv - more * more, 0.f) + 0.f * dev[1];
}
// A row's squared deviations leave fp32's range where their sum is no finite number, and lose digits where their mean and eps are
// below 2^-100.  Such a row is taken times a power of two that brings the largest magnitude into [1, 4), in the second case only up
// and by 2^110 at most, where eps has room.  What becomes subnormal on the way is nothing next to the largest.
__device__ inline bool out_of_range(float squares, float inv, float eps) {
  return !(squares < __builtin_inff()) || fmaf(squares, inv, eps) < 0x1p-100f;
}
// v's magnitude, infinity for a NaN too (which a maximum drops)
__device__ inline float magnitude(float v) { return fabsf(v) < __builtin_inff() ? fabsf(v) : __builtin_inff(); }
struct Scaled {
  float scale, rstd, mean, value;  // rstd of the scaled deviations; the row's own mean and rstd
  __device__ Scaled(float largest, float squares) {
    const int e = (int)(__float_as_uint(largest) >> 23) - 127, most = squares < __builtin_inff() ? 0 : 126;
    scale = __uint_as_float((uint32_t)(127 - min(max(e, -110), most)) << 23);
  }
  __device__ void finish(const float* dev, float inv, float first, float more, float eps) {
    const float var = variance_of(dev, inv, more);
    rstd = 1.0f / sqrtf(var + eps * scale * scale);
    value = rstd * scale;
    if (scale < 1.f && var == 0.f && eps > 0.f) {  // no spread: eps alone, of which its scaled form keeps nothing
      rstd = fminf(rstd, 0x1.fffffep127f);
      value = 1.0f / sqrtf(eps);
    }
    mean = (first + more) * __uint_as_float((254u << 23) - __float_as_uint(scale));
  }
};

// A row out of range, its outputs written: each of its waves takes the statistics by itself (no barrier, whatever the other rows of
// the workgroup are) and its threads store again what they stored.  8192 x 4096 of nothing but such rows 185 us, of NaN, where
// the first values tell, 26 (22 without the look).
template <typename T, typename W, int VEC, int TH>
__device__ void norm_again(const NormArgs& a, int64_t row, int tid, float squares) {
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
  const int lane = threadIdx.x & 63, H = (int)a.H;
  const float inv = 1.0f / (float)a.H;
  constexpr int N = 8;  // sums of a lane: a value goes through 32 additions of the longest row's
  auto some = [&](int h, auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (h + j * 64 < H) f(j, (float)x[h + j * 64]);
  };
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll 1
    for (int h = lane; h < H; h += 64 * N) some(h, f);
  };
  auto total = [&](float* p) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 1; j < N; ++j) p[0] += p[j];
    return wave_sum(p[0]);
  };
  float top = 0.f, sum[N] = {}, square[N] = {}, dev[2];
#pragma unroll 1
  for (int h0 = 0; h0 < H; h0 += 64 * N) {
    some(h0 + lane, [&](int, float v) __attribute__((always_inline)) { top = fmaxf(top, magnitude(v)); });
    if (__any(top == __builtin_inff())) return;  // an infinity or a NaN among the values: the row is NaN and stays
  }
  Scaled s(wave_max(top), squares);
  each([&](int j, float v) __attribute__((always_inline)) { sum[j] += v * s.scale; });
  const float first = total(sum) * inv;
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j] = 0.f;
  each([&](int j, float v) __attribute__((always_inline)) {
    const float d = v * s.scale - first;
    sum[j] += d;
    square[j] = fmaf(d, d, square[j]);
  });
  dev[0] = total(sum), dev[1] = total(square);
  const float more = dev[0] * inv;
  s.finish(dev, inv, first, more, a.eps);
  if (tid == 0) {
    if (a.mean) a.mean[row] = s.mean;
    if (a.rstd) a.rstd[row] = s.value;
  }
#pragma unroll 1
  for (int i = tid; i * VEC < H; i += TH)
#pragma unroll 1
    for (int h = i * VEC; h < min(H, i * VEC + VEC); ++h) {
      float y = ((float)x[h] * s.scale - first - more) * s.rstd;
      if (a.w) y *= (float)reinterpret_cast<const W*>(a.w)[h];
      if (a.b) y += (float)reinterpret_cast<const W*>(a.b)[h];
      reinterpret_cast<T*>(a.y)[row * a.ldy + h] = (T)y;
    }
}

// grid: ceil(T / R) workgroups of R rows, TH threads each.  Bound by HBM: 8192 x 4096 bf16 30 us, 4.5 TB/s (a plain copy 5.0).
template <typename T, typename W, int VEC, bool WHOLE, int TH, int NV, int R>
__global__ void __launch_bounds__(TH * R)
k_norm(NormArgs a) {
  __shared__ float s_sum[R][2][TH / 64 * 2];
  const int sub = threadIdx.x / TH, tid = threadIdx.x % TH;
  const int64_t row = (int64_t)blockIdx.x * R + sub;
  const bool live = row < a.T;
  const int64_t at = (live ? row : a.T - 1) * a.ldx;
  const float inv = 1.0f / (float)a.H;
  float v[NV][VEC], sum[2] = {0.f, 0.f};
  typename NormVec<T, VEC>::V raw[NV] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t h = (int64_t)(i * TH + tid) * VEC;
    if (h < a.H) raw[i] = norm_load<T, VEC, WHOLE>(a.x, at, h, a.H);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    norm_widen<T, VEC>(raw[i], v[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += v[i][e];
  }
  row_sum<TH, 1>(sum, s_sum[sub][0]);
  const float first = sum[0] * inv;
  float dev[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t h = (int64_t)(i * TH + tid) * VEC;
    if (h < a.H) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = WHOLE || h + e < a.H ? v[i][e] - first : 0.f;
        dev[0] += v[i][e];
        dev[1] = fmaf(v[i][e], v[i][e], dev[1]);
      }
    }
  }
  row_sum<TH, 2>(dev, s_sum[sub][1]);
  const float more = dev[0] * inv;
  const float rstd = 1.0f / sqrtf(variance_of(dev, inv, more) + a.eps);
  if (!live) return;
  if (tid == 0) {
    if (a.mean) a.mean[row] = first + more;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t h = (int64_t)(i * TH + tid) * VEC;
    if (h >= a.H) continue;
    float w[VEC], b[VEC];
    if (a.w) norm_get<W, VEC, WHOLE>(a.w, h, a.H, w);
    if (a.b) norm_get<W, VEC, WHOLE>(a.b, h, a.H, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float y = (v[i][e] - more) * rstd;
      if (a.w) y *= w[e];
      if (a.b) y += b[e];
      v[i][e] = y;
    }
    norm_store<T, VEC, WHOLE>(a.y, row * a.ldy, h, a.H, v[i]);
  }
  if (out_of_range(dev[1], inv, a.eps)) norm_again<T, W, VEC, TH>(a, row, tid, dev[1]);  // behind the stores: before them it cost 3 %
}

// the largest of v >= 0 over the TH threads of a row, as row_sum; s: [TH / 64]
template <int TH>
__device__ inline float row_max(float v, float* s) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) s[(threadIdx.x % TH) >> 6] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < TH / 64; ++w) v = fmaxf(v, s[w]);
  return v;
}

// Rows longer than the registers hold: a workgroup of 1024 threads reads its row three times (the second and third
// from the caches).  grid: T.
constexpr int kLongThreads = 1024;

template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads)
k_norm_long(NormArgs a) {
  __shared__ float s_sum[2][kLongThreads / 64 * 2], s_max[kLongThreads / 64];
  const int64_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
  const float inv = 1.0f / (float)a.H;
  float first, dev[2];
  auto statistics = [&](float scale) __attribute__((always_inline)) {
    float sum = 0.f;
    for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) sum += (float)x[h] * scale;
    row_sum<kLongThreads, 1>(&sum, s_sum[0]);
    first = sum * inv;
    dev[0] = dev[1] = 0.f;
    for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) {
      const float d = (float)x[h] * scale - first;
      dev[0] += d;
      dev[1] = fmaf(d, d, dev[1]);
    }
    row_sum<kLongThreads, 2>(dev, s_sum[1]);
  };
  auto put = [&](float scale, float more, float rstd, float mean, float value) __attribute__((always_inline)) {
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = value;
    }
    for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) {
      float y = ((float)x[h] * scale - first - more) * rstd;
      if (a.w) y *= (float)reinterpret_cast<const W*>(a.w)[h];
      if (a.b) y += (float)reinterpret_cast<const W*>(a.b)[h];
      reinterpret_cast<T*>(a.y)[row * a.ldy + h] = (T)y;
    }
  };
  statistics(1.f);
  float top = __builtin_inff();
  if (__builtin_amdgcn_readfirstlane(out_of_range(dev[1], inv, a.eps))) {
    top = 0.f;
    for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) top = fmaxf(top, magnitude((float)x[h]));
    top = row_max<kLongThreads>(top, s_max);
  }
  if (top == __builtin_inff()) {  // nothing to scale, or an infinity or a NaN among the values: the row is NaN
    const float more = dev[0] * inv, rstd = 1.0f / sqrtf(variance_of(dev, inv, more) + a.eps);
    put(1.f, more, rstd, first + more, rstd);
    return;
  }
  Scaled s(top, dev[1]);
  statistics(s.scale);
  const float more = dev[0] * inv;
  s.finish(dev, inv, first, more, a.eps);
  put(s.scale, more, s.rstd, s.mean, s.value);
}

// ---- gradients -------------------------------------------------------------------------------------------

template <int VEC, bool WHOLE>
__device__ inline void put_f32(float* p, int64_t h, int64_t H, const float* v) {
#pragma unroll
  for (int c = 0; c < VEC; c += 4)
    if (WHOLE || h + c < H) norm_store<float, 4, WHOLE>(p, 0, h + c, H, v + c);
}

// grid: parts workgroups, workgroup p takes rows p R + sub, then parts R further.  dx as rows go by; the columns' sums of
// dy xh and dy stay in the registers of the thread that owns the column, are added over the workgroup's R rows in LDS and
// written as one row of partial sums [parts][2][H], which k_norm_join adds in order.  Bound by HBM: 8192 x 4096 bf16 with a
// residual 49 us, 5.4 TB/s, and the join of 256 parts 4.7.
template <typename T, typename W, int VEC, bool WHOLE, int TH, int NV, int R>
__global__ void __launch_bounds__(TH * R)
k_norm_grad(NormGradArgs a) {
  __shared__ float s_sum[R][2][TH / 64 * 2];
  extern __shared__ float s_col[];  // [TH * VEC] per vector slot, R > 1
  const int sub = threadIdx.x / TH, tid = threadIdx.x % TH;
  const float inv = 1.0f / (float)a.H;
  const bool cols = a.part != nullptr;
  float w[NV][VEC], sw[NV][VEC], sb[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t h = (int64_t)(i * TH + tid) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = 1.f, sw[i][e] = sb[i][e] = 0.f;
    if (a.w && h < a.H) norm_get<W, VEC, WHOLE>(a.w, h, a.H, w[i]);
  }
  // a row is in flight while the one before it is used, where the registers hold both; past the end the last row again, not used
  constexpr bool AHEAD = NV * VEC <= 8;
  typedef typename NormVec<T, VEC>::V V;
  V xn[NV], dn[NV], rn[NV];
  float mean_n = 0.f, rstd_n = 0.f;
  auto fetch = [&](int64_t row) {
    row = min(row, a.T - 1);
    mean_n = a.mean[row], rstd_n = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t h = (int64_t)(i * TH + tid) * VEC, at = h < a.H ? h : 0;
      xn[i] = norm_load<T, VEC, WHOLE>(a.x, row * a.ldx, at, a.H);
      dn[i] = norm_load<T, VEC, WHOLE>(a.dy, row * a.lddy, at, a.H);
      if (a.residual) rn[i] = norm_load<T, VEC, WHOLE>(a.residual, row * a.ldr, at, a.H);
    }
  };
  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * R;
  if (AHEAD) fetch((int64_t)blockIdx.x * R + sub);
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += step, phase ^= 1) {
    const int64_t row = r0 + sub;
    const bool live = row < a.T;
    float xh[NV][VEC], g[NV][VEC], sum[2] = {0.f, 0.f};
    V res[NV];
    if (!AHEAD) fetch(row);
    const float mean = mean_n, rstd = rstd_n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      norm_widen<T, VEC>(xn[i], xh[i]);
      norm_widen<T, VEC>(dn[i], g[i]);
      res[i] = rn[i];
    }
    if (AHEAD) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t h = (int64_t)(i * TH + tid) * VEC;
      if (live && h < a.H) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[i][e] = (xh[i][e] - mean) * rstd;
          if (cols) {
            sw[i][e] = fmaf(g[i][e], xh[i][e], sw[i][e]);
            sb[i][e] += g[i][e];
          }
          g[i][e] *= w[i][e];
          sum[0] += g[i][e];
          sum[1] = fmaf(g[i][e], xh[i][e], sum[1]);
        }
      }
    }
    if (!a.dx) continue;
    row_sum<TH, 2>(sum, s_sum[sub][phase]);  // two buffers: one barrier a row keeps them apart
    const float c1 = sum[0] * inv, c2 = sum[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t h = (int64_t)(i * TH + tid) * VEC;
      if (!live || h >= a.H) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[i][e] = rstd * (g[i][e] - c1 - xh[i][e] * c2);
      if (a.residual) {
        float r[VEC];
        norm_widen<T, VEC>(res[i], r);
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[i][e] += r[e];
      }
      norm_store<T, VEC, WHOLE>(a.dx, row * a.lddx, h, a.H, g[i]);
    }
  }
  if (!cols) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t h = (int64_t)(i * TH + tid) * VEC;
      if constexpr (R > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) s_col[(sub * VEC + e) * TH + tid] = k ? sb[i][e] : sw[i][e];
        __syncthreads();
        if (sub == 0 && h < a.H) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float v = s_col[e * TH + tid];
#pragma unroll
            for (int r = 1; r < R; ++r) v += s_col[(r * VEC + e) * TH + tid];
            (k ? sb : sw)[i][e] = v;
          }
          put_f32<VEC, WHOLE>(part + k * a.H, h, a.H, (k ? sb : sw)[i]);
        }
      } else if (h < a.H) {
        put_f32<VEC, WHOLE>(part + k * a.H, h, a.H, (k ? sb : sw)[i]);
      }
    }
}

// dx of rows longer than the registers hold, grid: T
template <typename T, typename W>
__global__ void __launch_bounds__(kLongThreads)
k_norm_grad_long(NormGradArgs a) {
  __shared__ float s_sum[kLongThreads / 64 * 2];
  const int64_t row = blockIdx.x;
  const T *x = reinterpret_cast<const T*>(a.x) + row * a.ldx, *dy = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
  const W* w = reinterpret_cast<const W*>(a.w);
  const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / (float)a.H;
  float sum[2] = {0.f, 0.f};
  for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) {
    const float g = w ? (float)dy[h] * (float)w[h] : (float)dy[h];
    sum[0] += g;
    sum[1] = fmaf(g, ((float)x[h] - mean) * rstd, sum[1]);
  }
  row_sum<kLongThreads, 2>(sum, s_sum);
  const float c1 = sum[0] * inv, c2 = sum[1] * inv;
  for (int64_t h = threadIdx.x; h < a.H; h += kLongThreads) {
    const float g = w ? (float)dy[h] * (float)w[h] : (float)dy[h];
    float d = rstd * (g - c1 - ((float)x[h] - mean) * rstd * c2);
    if (a.residual) d += (float)reinterpret_cast<const T*>(a.residual)[row * a.ldr + h];
    reinterpret_cast<T*>(a.dx)[row * a.lddx + h] = (T)d;
  }
}

// the columns' sums of such rows over part p's rows, grid: (ceil(H / 256), parts)
template <typename T>
__global__ void __launch_bounds__(256)
k_norm_cols_long(NormGradArgs a) {
  const int64_t h = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (a.T + gridDim.y - 1) / gridDim.y;
  if (h >= a.H) return;
  const int64_t r1 = min(a.T, (blockIdx.y + 1) * per);
  float sw = 0.f, sb = 0.f;
  for (int64_t r = blockIdx.y * per; r < r1; ++r) {
    const float d = (float)reinterpret_cast<const T*>(a.dy)[r * a.lddy + h];
    sw = fmaf(d, ((float)reinterpret_cast<const T*>(a.x)[r * a.ldx + h] - a.mean[r]) * a.rstd[r], sw);
    sb += d;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.H;
  part[h] = sw;
  part[a.H + h] = sb;
}

// grid: (64 columns from h0 on each, 2).  The partial sums of 64 columns of dw (y = 0) or db: 16 waves take every 16th part, their
// sums are added in wave order.
constexpr int kJoinThreads = 1024;

template <typename W>
__global__ void __launch_bounds__(kJoinThreads)
k_norm_join(const float* __restrict__ part, int64_t parts, int64_t H, int64_t h0, void* dw, void* db) {
  __shared__ float s_sum[16][64];
  W* out = reinterpret_cast<W*>(blockIdx.y ? db : dw);
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t h = h0 + (int64_t)blockIdx.x * 64 + lane;
  const float* p = part + blockIdx.y * H + h;
  float sum = 0.f;
  if (h < H) {
#pragma unroll 8
    for (int64_t i = wave; i < parts; i += 16) sum += p[i * 2 * H];
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave || h >= H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) sum += s_sum[i][lane];
  out[h] = (W)sum;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int TH, int NV, int R>
struct NormShape {
  static constexpr int th = TH, nv = NV, r = R;
};

// calls f with the shape for rows of n vectors, or g where the registers hold no such row
template <typename F, typename G>
void with_shape(int64_t n, F f, G g) {
  if (n <= 64) f(NormShape<64, 1, 4>{});
  else if (n <= 128) f(NormShape<64, 2, 4>{});
  else if (n <= 256) f(NormShape<256, 1, 2>{});
  else if (n <= 512) f(NormShape<256, 2, 2>{});
  else if (n <= 1024) f(NormShape<256, 4, 2>{});
  else if (n <= 2048) f(NormShape<1024, 2, 1>{});
  else g();
}
// the same for the gradients, whose threads hold the columns' sums besides
template <typename F, typename G>
void with_grad_shape(int64_t n, F f, G g) {
  if (n <= 64) f(NormShape<64, 1, 4>{});
  else if (n <= 128) f(NormShape<128, 1, 4>{});
  else if (n <= 256) f(NormShape<256, 1, 2>{});
  else if (n <= 512) f(NormShape<512, 1, 2>{});
  else if (n <= 1024) f(NormShape<1024, 1, 1>{});
  else if (n <= 2048) f(NormShape<1024, 2, 1>{});
  else g();
}

// calls f with the rows' and the weights' types
template <typename F>
void with_types(int dtype, int w_dtype, F f) {
  const bool same = dtype == w_dtype;
  if (dtype == EFF_DT_BF16) same ? f(bf16_t{}, bf16_t{}) : f(bf16_t{}, float{});
  else if (dtype == EFF_DT_F16) same ? f(f16_t{}, f16_t{}) : f(f16_t{}, float{});
  else f(float{}, float{});
}

}  // namespace

int64_t norm_at_once(int threads, int64_t per) { return most_workgroups(threads) * per; }
int64_t norm_columns_at_once() { return most_workgroups(kJoinThreads) * 64; }

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  with_types(a.dtype, a.w_dtype, [&](auto t, auto wt) {
    typedef decltype(t) T;
    typedef decltype(wt) W;
    constexpr int VEC = 16 / (int)sizeof(T);
    auto rows = [&](auto launch, int threads, int64_t per) {  // per: rows of a workgroup
      const int64_t most = norm_at_once(threads, per);
      for (int64_t t0 = 0; t0 < a.T; t0 += most) {
        NormArgs p = a;
        p.T = std::min(most, a.T - t0);
        p.x = reinterpret_cast<const T*>(a.x) + t0 * a.ldx;
        p.y = reinterpret_cast<T*>(a.y) + t0 * a.ldy;
        if (a.mean) p.mean = a.mean + t0;
        if (a.rstd) p.rstd = a.rstd + t0;
        launch(p, dim3((unsigned)cdiv(p.T, per)));
      }
    };
    auto go = [&](auto sh, auto whole) {
      typedef decltype(sh) S;
      rows([&](const NormArgs& p, dim3 g) {
        hipLaunchKernelGGL((k_norm<T, W, VEC, decltype(whole)::value, S::th, S::nv, S::r>), g, dim3(S::th * S::r), 0, s, p);
      }, S::th * S::r, S::r);
    };
    with_shape(cdiv(a.H, VEC), [&](auto sh) { a.H % VEC ? go(sh, std::false_type{}) : go(sh, std::true_type{}); }, [&] {
      rows([&](const NormArgs& p, dim3 g) { hipLaunchKernelGGL((k_norm_long<T, W>), g, dim3(kLongThreads), 0, s, p); }, kLongThreads, 1);
    });
  });
  return hipGetLastError();
}

// Parts of the columns' sums, a workgroup's each: as many as fill the chip with 16 waves a CU.
int64_t norm_parts(int64_t T, int64_t H) { return std::min<int64_t>(T, H <= 512 ? 1024 : H <= 2048 ? 512 : 256); }

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  const int64_t parts = norm_parts(a.T, a.H);
  with_types(a.dtype, a.w_dtype, [&](auto t, auto wt) {
    typedef decltype(t) T;
    typedef decltype(wt) W;
    constexpr int VEC = 16 / (int)sizeof(T);
    int64_t written = parts;  // rows of partial sums that the pass writes
    auto lengthy = [&] {
      const int64_t most = norm_at_once(kLongThreads, 1);
      for (int64_t t0 = 0; a.dx && t0 < a.T; t0 += most) {
        NormGradArgs p = a;
        p.T = std::min(most, a.T - t0);
        p.x = reinterpret_cast<const T*>(a.x) + t0 * a.ldx;
        p.dy = reinterpret_cast<const T*>(a.dy) + t0 * a.lddy;
        if (a.residual) p.residual = reinterpret_cast<const T*>(a.residual) + t0 * a.ldr;
        p.mean = a.mean + t0, p.rstd = a.rstd + t0, p.dx = reinterpret_cast<T*>(a.dx) + t0 * a.lddx;
        hipLaunchKernelGGL((k_norm_grad_long<T, W>), dim3((unsigned)p.T), dim3(kLongThreads), 0, s, p);
      }
      if (a.part) hipLaunchKernelGGL((k_norm_cols_long<T>), dim3((unsigned)cdiv(a.H, 256), (unsigned)parts), dim3(256), 0, s, a);
    };
    auto go = [&](auto sh, auto whole) {
      typedef decltype(sh) S;
      written = std::min(parts, cdiv(a.T, S::r));
      const int lds = S::r > 1 ? S::r * S::th * VEC * 4 : 0;
      hipLaunchKernelGGL((k_norm_grad<T, W, VEC, decltype(whole)::value, S::th, S::nv, S::r>), dim3((unsigned)written), dim3(S::th * S::r),
                         lds, s, a);
    };
    if (a.T > 0) with_grad_shape(cdiv(a.H, VEC), [&](auto sh) { a.H % VEC ? go(sh, std::false_type{}) : go(sh, std::true_type{}); }, lengthy);
    for (int64_t h0 = 0; (a.dw || a.db) && h0 < a.H; h0 += norm_columns_at_once())
      hipLaunchKernelGGL((k_norm_join<W>), dim3((unsigned)cdiv(std::min(norm_columns_at_once(), a.H - h0), 64), 2), dim3(kJoinThreads), 0, s,
                         a.part, a.T > 0 ? written : 0, a.H, h0, a.dw, a.db);
  });
  return hipGetLastError();
}

}  // namespace eff
