// The router's losses over a batch, with the experts' counts, and the gradient at the logits.
//
// p[t] = softmax(l[t]), lse[t] = log sum exp l[t].  A token is live if its mask is set and some logit is above -inf; n is
// their number.  f[e] = (live tokens' pairs with id e) / (n K);  P[e] = mean of p[t,e];
//   balance = E sum f P,  z = mean of lse^2  (means over the live tokens; 0 where there is none).
// f counts and has no gradient, so with a = g0 E / n, b = 2 g1 / n, S[t] = sum f p[t]:
//   dl[t,j] = p[t,j] (a (f[j] - S[t]) + b lse[t]) + sum over k with ids[t,k] = j of w[t,k] (dw[t,k] - sum w[t] dw[t]),
// the last term being the softmax over the selected logits that gave the weights w.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "eff_internal.h"
#include "wave.h"

namespace eff {
namespace {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// A wave takes a row; waves of a workgroup, 16 where the registers of so many hold it.
template <int VEC, int NV>
constexpr int waves_of() { return VEC * NV <= 16 ? 16 : 4; }
constexpr int waves_for(int E) { return E <= 16 * 64 ? 16 : 4; }  // the same: VEC NV is the number of columns of a lane
constexpr int kGradWaves = 4;
constexpr float kInf = __builtin_inff();

// VEC consecutive logits at any place (the hardware takes 16-byte accesses at any address)
template <typename T, int VEC>
struct LogitVec {
  typedef T V __attribute__((ext_vector_type(VEC)));
  typedef V Loose __attribute__((aligned(sizeof(T))));
};

// A lane's values of a row of E logits: columns (i * 64 + lane) * VEC + e.  WHOLE: E is a multiple of VEC.
template <typename T, int VEC, bool WHOLE, int NV>
struct LogitRow {
  typename LogitVec<T, VEC>::V raw[NV];
  __device__ void load(const T* p, int E, int lane) {  // past the end the row's first values, which are not used
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * 64 + lane) * VEC;
      if (WHOLE || E >= VEC) {  // a vector that ends past the row is read from where it ends with it, and moved
        const int at = j + VEC <= E ? j : j < E ? E - VEC : 0;
        raw[i] = *reinterpret_cast<const typename LogitVec<T, VEC>::Loose*>(p + at);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) raw[i][e] = p[min(e, E - 1)];
      }
    }
  }
  __device__ void widen(int E, int lane, float (*v)[VEC]) const {  // past the end -infinity
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * 64 + lane) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = j + e < E ? (float)raw[i][e] : -kInf;
      if (!WHOLE && E >= VEC && j < E && j + VEC > E) {
        const int shift = j + VEC - E;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float from = -kInf;
#pragma unroll
          for (int o = 1; o < VEC; ++o)
            if (o == shift && e + o < VEC) from = (float)raw[i][e + o];
          v[i][e] = from;
        }
      }
    }
  }
};

// e^x to about 2 units in the last place and 0 below 2^-126, for x <= 0 or NaN.  With log2 e = a + b, a its nearest float: t = fl(x a)
// leaves d = (x a - t) + x b, and e^x = 2^t 2^d, where 2^d = 1 + d ln 2 to fp32, |d| being below 2^-16.
__device__ inline float exp_down(float x) {
  constexpr double log2e = 1.4426950408889634074;  // 1 / ln 2
  constexpr float a = (float)log2e, b = (float)(log2e - (double)a), ln2 = (float)(1.0 / log2e);
  x = x < -104.f ? -104.f : x;
  const float t = x * a, d = fmaf(x, b, fmaf(x, a, -t));
  return __builtin_amdgcn_exp2f(t) * fmaf(d, ln2, 1.0f);
}

// A copy that stays one: the value is taken out of the register that the next load goes to before that load is issued (else the
// copies stand at the end of the loop, behind a wait for everything under way).
template <typename V>
__device__ inline void keep(V& v) { asm volatile("" : "+v"(v)); }

// LDS writes of this wave before, reads of its other lanes after (a wave's LDS accesses complete in order)
__device__ inline void wave_order() {
  asm volatile("" : : : "memory");
  __builtin_amdgcn_wave_barrier();
}

// sum: over the experts of their sum of p times their count; z: the sum of lse^2
__device__ inline void put_losses(const BalanceArgs& a, double sum, double z, int live) {
  const double n = (double)live;
  a.losses[0] = live ? (float)(sum * a.E / (n * n * a.K)) : 0.f;
  a.losses[1] = live ? (float)(z / n) : 0.f;
}

// grid: parts.  Wave w of part p takes rows p W + w, then parts W further (W waves); the part's sums of p and of lse^2 and
// its counts go to one row of the workspace.  2048 x 256 fp32 4.9 us: the way to memory and back, two rows a wave.
// One part alone finishes by itself.
template <typename T, int VEC, bool WHOLE, int NV>
__global__ void __launch_bounds__(64 * (waves_of<VEC, NV>()))
k_balance(BalanceArgs a) {
  constexpr int W = waves_of<VEC, NV>();
  extern __shared__ int s_count[];  // [E + 1], the last: live tokens
  __shared__ float s_p[W][64 * VEC], s_z[W];
  __shared__ double s_share[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), E = a.E, K = a.K;
  for (int e = threadIdx.x; e <= E; e += 64 * W) s_count[e] = 0;
  __syncthreads();
  float sum[NV][VEC], z = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[i][e] = 0.f;
  // a row is in flight while the one before it is used, masked or not; past the end the last row again, which is not used
  const int64_t step = (int64_t)gridDim.x * W;
  LogitRow<T, VEC, WHOLE, NV> next;
  int next_id = -1, next_set = 1;
  auto fetch = [&](int64_t t) {
    t = min(t, a.T - 1);
    if (a.mask) next_set = a.mask[t];
    next.load(reinterpret_cast<const T*>(a.logits) + t * a.ld, E, lane);
    next_id = a.ids[t * K + min(lane, K - 1)];
  };
  int64_t t = (int64_t)blockIdx.x * W + wave;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += step) {
    float v[NV][VEC], top = -kInf;
    const int set = next_set;
    int id = next_id;
    next.widen(E, lane, v);
    keep(id);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) keep(v[i][e]);
    fetch(t + step);
    if (!set) {
      if (lane == 0) a.lse[t] = -kInf;
      continue;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) top = fmaxf(top, v[i][e]);
    top = wave_max(top);
    if (top == -kInf) top = 0.f;  // no logit above -inf: the sum is 0, or NaN where one is NaN
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = exp_down(v[i][e] - top);
        total += v[i][e];
      }
    total = wave_sum(total);
    const float lse = total == 0.f ? -kInf : top + logf(total);
    if (lane == 0) a.lse[t] = lse;
    if (total == 0.f) continue;
    const float inv = 1.0f / total;
    z = fmaf(lse, lse, z);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[i][e] = fmaf(v[i][e], inv, sum[i][e]);
    if (lane < K && id >= 0 && id < E) atomicAdd(&s_count[id], 1);
    if (lane == 0) atomicAdd(&s_count[E], 1);
  }
  if (lane == 0) s_z[wave] = z;
  const bool alone = gridDim.x == 1;
  double share = 0.0;  // alone: of the sum of f P
  int2* part = a.part + (int64_t)blockIdx.x * (E + 1);
#pragma unroll
  for (int i = 0; i < NV; ++i) {  // the waves' sums in wave order, 64 VEC columns at a time
#pragma unroll
    for (int e = 0; e < VEC; ++e) s_p[wave][lane * VEC + e] = sum[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < 64 * VEC; c += 64 * W) {
      const int j = i * 64 * VEC + c;
      float v = s_p[0][c];
#pragma unroll
      for (int w = 1; w < W; ++w) v += s_p[w][c];
      if (j >= E) continue;
      if (alone) {
        share += (double)v * (double)s_count[j];
        a.counts[j] = s_count[j];
      } else {
        part[j] = make_int2(__float_as_int(v), s_count[j]);
      }
    }
    __syncthreads();
  }
  if (alone) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) share += __shfl_xor(share, o);
    if (lane == 0) s_share[wave] = share;
    __syncthreads();
  }
  if (threadIdx.x) return;
  for (int w = 1; w < W; ++w) z += s_z[w];
  if (!alone) {
    part[E] = make_int2(__float_as_int(z), s_count[E]);
    return;
  }
  for (int w = 1; w < W; ++w) share += s_share[w];
  a.counts[E] = s_count[E];
  put_losses(a, share, z, s_count[E]);
}

// Column sums over the parts, in double and in order: many columns or parts are added up by many workgroups first
// (k_balance_columns, grid: ceil((E + 1) / 64), one row left, rounded to fp32), the rest by the one that computes the losses.  One
// workgroup for all of 64 parts of 257 columns takes 5 us, five and a last one to finish 10.  Three launches for 512 x 4096 take
// 35 us, for 16384 x 512 19.
constexpr int kJoin = 1024, kParts = 256;

__global__ void __launch_bounds__(kJoin)
k_balance_columns(const int2* __restrict__ part, int parts, int E, int2* __restrict__ out) {
  __shared__ double s_p[kJoin / 64][64];
  __shared__ int s_c[kJoin / 64][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  double p = 0.0;
  int c = 0;
  if (e <= E) {
    constexpr int MOST = kParts / (kJoin / 64);  // all of a wave's parts at once; past the last one the last again, not used
    int2 v[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) v[i] = part[(int64_t)min(wave + i * (kJoin / 64), parts - 1) * (E + 1) + e];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      if (wave + i * (kJoin / 64) >= parts) continue;
      p += (double)__int_as_float(v[i].x);
      c += v[i].y;
    }
  }
  s_p[wave][lane] = p;
  s_c[wave][lane] = c;
  __syncthreads();
  if (wave || e > E) return;
  for (int w = 1; w < kJoin / 64; ++w) {
    p += s_p[w][lane];
    c += s_c[w][lane];
  }
  out[e] = make_int2(__float_as_int((float)p), c);
}

__global__ void __launch_bounds__(kJoin)
k_balance_join(BalanceArgs a, const int2* __restrict__ part, int parts) {
  __shared__ double s_p[kJoin];
  __shared__ int s_c[kJoin];
  __shared__ double s_sum[kJoin / 64], s_z;
  __shared__ int s_n;
  const int tid = threadIdx.x, E = a.E;
  const int per = min(kJoin, (E + 64) / 64 * 64), slices = kJoin / per;  // threads of a slice of the parts, a column each
  const int slice = tid / per, lane_col = tid - slice * per;
  double sum = 0.0;
  for (int c0 = 0; c0 <= E; c0 += per) {
    const int e = c0 + lane_col;
    double p = 0.0;
    int c = 0;
    if (slice < slices && e <= E) {
      constexpr int B = 24;  // parts under way at once; past the last one the last again, not used
      for (int i0 = slice; i0 < parts; i0 += B * slices) {
        int2 v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) v[b] = part[(int64_t)min(i0 + b * slices, parts - 1) * (E + 1) + e];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (i0 + b * slices >= parts) continue;
          p += (double)__int_as_float(v[b].x);
          c += v[b].y;
        }
      }
    }
    s_p[tid] = p;
    s_c[tid] = c;
    __syncthreads();
    if (slice == 0 && e <= E) {
      for (int s = 1; s < slices; ++s) {
        p += s_p[s * per + lane_col];
        c += s_c[s * per + lane_col];
      }
      a.counts[e] = c;
      if (e < E) sum += p * (double)c;
      else s_z = p, s_n = c;
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
  __syncthreads();
  if (tid) return;
  for (int w = 1; w < kJoin / 64; ++w) sum += s_sum[w];
  put_losses(a, sum, s_z, s_n);
}

// grid: as many workgroups as fill the chip; a wave per row.  f of the lane's columns stays in registers.  Bound by HBM:
// 16384 x 512 fp32 with top-10 weights 16 us, 4.2 TB/s.
template <typename T, int VEC, bool WHOLE, int NV>
__global__ void __launch_bounds__(64 * kGradWaves)
k_balance_grad(BalanceGradArgs a) {
  constexpr int W = kGradWaves;
  extern __shared__ __attribute__((aligned(16))) float s_pairs[];  // [W][E rounded up to 64 VEC NV], with w
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), E = a.E, K = a.K;
  const float n = (float)a.counts[E];
  const float ga = a.dlosses && n > 0 ? a.dlosses[0] * ((float)E / n) : 0.f, gb = a.dlosses && n > 0 ? a.dlosses[1] * (2.f / n) : 0.f;
  const float per = n > 0 ? 1.f / (n * (float)K) : 0.f;
  float f[NV][VEC];
  int count[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) count[i][e] = a.counts[min((i * 64 + lane) * VEC + e, E - 1)];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[i][e] = (i * 64 + lane) * VEC + e < E ? (float)count[i][e] * per : 0.f;
  float* mine = s_pairs + wave * (64 * VEC * NV);
  if (a.w) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) mine[(i * 64 + lane) * VEC + e] = 0.f;
  }
  // a row is in flight while the one before it is used, live or not; past the end the last row again, which is not used
  const int64_t step = (int64_t)gridDim.x * W;
  LogitRow<T, VEC, WHOLE, NV> next;
  float next_lse = -kInf, next_w = 0.f, next_dw = 0.f;
  int next_id = -1;
  auto fetch = [&](int64_t t) {
    t = min(t, a.T - 1);
    next_lse = a.lse[t];
    if (a.dlosses) next.load(reinterpret_cast<const T*>(a.logits) + t * a.ld, E, lane);
    if (a.w) {
      const int64_t at = t * K + min(lane, K - 1);
      next_id = a.ids[at];
      next_w = a.w[at];
      next_dw = a.dw[at];
    }
  };
  int64_t t = (int64_t)blockIdx.x * W + wave;
  fetch(t);
  for (; t < a.T; t += step) {
    T* out = reinterpret_cast<T*>(a.dlogits) + t * a.ldd;
    const float lse = next_lse;
    float w_k = next_w, dw_k = next_dw, v[NV][VEC];
    int id = next_id;
    if (a.dlosses) next.widen(E, lane, v);
    keep(w_k), keep(dw_k), keep(id);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) keep(v[i][e]);
    fetch(t + step);
    if (lse == -kInf) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
    } else {
      if (a.dlosses) {
        // the softmax anew and not exp(l - lse): far from 0 the saved lse has lost digits that p needs
        float top = -kInf, both[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) top = fmaxf(top, v[i][e]);
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            v[i][e] = exp_down(v[i][e] - top);
            both[0] += v[i][e];
            both[1] = fmaf(f[i][e], v[i][e], both[1]);
          }
        const float inv = 1.0f / wave_sum(both[0]), s = wave_sum(both[1]) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] *= inv * fmaf(ga, f[i][e] - s, gb * lse);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      }
      if (a.w) {
        const bool ok = lane < K && id >= 0 && id < E;
        const float w = ok ? w_k : 0.f, dw = ok ? dw_k : 0.f;
        const float g = w * (dw - wave_sum(w * dw));
        float sum = 0.f;  // of the pairs with this pair's id, in order of k
        for (int k = 0; k < K; ++k) {
          const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), k));
          if (__builtin_amdgcn_readlane(id, k) == id) sum += o;
        }
        if (ok) mine[id] = sum;
        wave_order();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += mine[(i * 64 + lane) * VEC + e];
        wave_order();
        if (ok) mine[id] = 0.f;
        wave_order();
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * 64 + lane) * VEC;
      if (j >= E) continue;
      if (WHOLE || j + VEC <= E) {
        typename LogitVec<T, VEC>::V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = (T)v[i][e];
        *reinterpret_cast<typename LogitVec<T, VEC>::Loose*>(out + j) = o;
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (j + e < E) out[j + e] = (T)v[i][e];
      }
    }
  }
}

// calls f with the logits' type, the vector width, whether it divides E, and the vectors of a lane
template <typename T, int VEC, typename W, typename F>
void with_vectors(int E, W whole, F f) {
  const std::integral_constant<int, VEC> v;
  const int n = (E + 64 * VEC - 1) / (64 * VEC);
  if (n <= 1) f(T{}, v, whole, std::integral_constant<int, 1>{});
  else if (n <= 2) f(T{}, v, whole, std::integral_constant<int, 2>{});
  else if (n <= 4) f(T{}, v, whole, std::integral_constant<int, 4>{});
  else if (n <= 8) f(T{}, v, whole, std::integral_constant<int, 8>{});
  else if constexpr (VEC < 8) f(T{}, v, whole, std::integral_constant<int, 16>{});
}
template <typename F>
void with_logits(int dtype, int E, F f) {
  auto go = [&](auto t) {
    typedef decltype(t) T;
    constexpr int VEC = 16 / (int)sizeof(T);
    E % VEC ? with_vectors<T, VEC>(E, std::false_type{}, f) : with_vectors<T, VEC>(E, std::true_type{}, f);
  };
  if (dtype == EFF_DT_F32) go(float{});
  else if (dtype == EFF_DT_BF16) go(bf16_t{});
  else go(f16_t{});
}

}  // namespace

// Workgroups of the pass over the logits: one per CU, fewer where its waves would have fewer than two rows each, and one alone, which
// needs no second launch, for up to four rows a wave: 64 x 256 fp32 9.0 us and not 11.6, 128 rows 10.7 and 11.6, 256 rows 18 and 11.7
// (so it ends somewhat below where the two meet).
int64_t balance_parts(int64_t T, int E) {
  const int W = waves_for(E);
  return T <= 4 * W ? 1 : std::min<int64_t>(kParts, (T + 2 * W - 1) / (2 * W));
}

int64_t balance_workspace(int64_t T, int E) { return ((balance_parts(T, E) + 1) * (E + 1) * 8 + 255) / 256 * 256; }

hipError_t launch_balance(BalanceArgs a, void* workspace, hipStream_t s) {
  int parts = (int)balance_parts(a.T, a.E);
  a.part = static_cast<int2*>(workspace);
  with_logits(a.dtype, a.E, [&](auto t, auto vec, auto whole, auto nv) {
    constexpr int V = decltype(vec)::value, N = decltype(nv)::value;
    hipLaunchKernelGGL((k_balance<decltype(t), V, decltype(whole)::value, N>), dim3(parts), dim3(64 * waves_of<V, N>()), (a.E + 1) * 4, s, a);
  });
  if (parts == 1) return hipGetLastError();
  const int2* part = a.part;
  if ((int64_t)parts * (a.E + 1) > 65536) {
    int2* out = a.part + (int64_t)parts * (a.E + 1);
    hipLaunchKernelGGL(k_balance_columns, dim3((a.E + 64) / 64), dim3(kJoin), 0, s, part, parts, a.E, out);
    part = out, parts = 1;
  }
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(kJoin), 0, s, a, part, parts);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s) {
  const int grid = (int)std::min<int64_t>(1024, (a.T + kGradWaves - 1) / kGradWaves);
  with_logits(a.dtype, a.E, [&](auto t, auto vec, auto whole, auto nv) {
    constexpr int V = decltype(vec)::value, N = decltype(nv)::value;
    hipLaunchKernelGGL((k_balance_grad<decltype(t), V, decltype(whole)::value, N>), dim3(grid), dim3(64 * kGradWaves), a.w ? kGradWaves * 64 * V * N * 4 : 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace eff
