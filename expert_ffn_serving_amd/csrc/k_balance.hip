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

constexpr int kWaves = 4;  // a wave per row
constexpr float kInf = __builtin_inff();

template <typename T, int VEC>
struct LogitVec {
  typedef T V __attribute__((ext_vector_type(VEC)));
};
template <typename T>
struct LogitVec<T, 1> {
  typedef T V;
};

// A lane's values of a row of E logits: columns (i * 64 + lane) * VEC + e.
template <typename T, int VEC, int NV>
struct LogitRow {
  typename LogitVec<T, VEC>::V raw[NV];
  __device__ void load(const T* p, int E, int lane) {  // past the end the row's first values, which are not used
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * 64 + lane) * VEC;
      raw[i] = *reinterpret_cast<const typename LogitVec<T, VEC>::V*>(p + (j < E ? j : 0));
    }
  }
  __device__ void widen(int E, int lane, float (*v)[VEC]) const {  // past the end -infinity
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if constexpr (VEC == 1) v[i][e] = (i * 64 + lane) * VEC < E ? (float)raw[i] : -kInf;
        else v[i][e] = (i * 64 + lane) * VEC < E ? (float)raw[i][e] : -kInf;
      }
  }
};

// LDS writes of this wave before, reads of its other lanes after (a wave's LDS accesses complete in order)
__device__ inline void wave_order() {
  asm volatile("" : : : "memory");
  __builtin_amdgcn_wave_barrier();
}
// grid: parts.  Wave w of part p takes rows p kWaves + w, then parts kWaves further; the part's sums of p and of lse^2 and
// its counts go to one row of the workspace each.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(64 * kWaves)
k_balance(BalanceArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
  int* s_count = reinterpret_cast<int*>(s_dyn);         // [E + 1], the last: live tokens
  float* s_p = reinterpret_cast<float*>(s_dyn) + a.E + 1;  // [E]
  __shared__ float s_z[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, K = a.K;
  for (int e = threadIdx.x; e <= E; e += 64 * kWaves) s_count[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;  // k_balance_join counts its workgroups from here
  __syncthreads();
  float sum[NV][VEC], z = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[i][e] = 0.f;
  // a row is in flight while the one before it is used; a masked token's is not read, past the end the last row is
  const int64_t step = (int64_t)gridDim.x * kWaves;
  LogitRow<T, VEC, NV> next;
  int next_id = -1;
  bool next_set = false;
  auto fetch = [&](int64_t t) {
    t = min(t, a.T - 1);
    next_set = !a.mask || a.mask[t];
    if (!next_set) return;
    next.load(reinterpret_cast<const T*>(a.logits) + t * a.ld, E, lane);
    next_id = lane < K ? a.ids[t * K + lane] : -1;
  };
  int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += step) {
    float v[NV][VEC], top = -kInf;
    const bool set = next_set;
    const int id = next_id;
    if (set) next.widen(E, lane, v);
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
        v[i][e] = expf(v[i][e] - top);
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
    if (id >= 0 && id < E) atomicAdd(&s_count[id], 1);
    if (lane == 0) atomicAdd(&s_count[E], 1);
  }
  if (lane == 0) s_z[wave] = z;
  for (int w = 0; w < kWaves; ++w) {  // the waves' sums in wave order
    __syncthreads();
    if (wave == w) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = (i * 64 + lane) * VEC + e;
          if (j < E) s_p[j] = w == 0 ? sum[i][e] : s_p[j] + sum[i][e];
        }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += 64 * kWaves)
    a.part[(int64_t)blockIdx.x * (E + 1) + e] = make_int2(__float_as_int(e < E ? s_p[e] : (s_z[0] + s_z[1]) + (s_z[2] + s_z[3])), s_count[e]);
}

// grid: ceil((E + 1) / 64).  Columns' sums over the parts: 16 waves take every 16th part, sums in double, in order.  The
// workgroup that finishes last adds up the losses (in order of e, so which one it is changes nothing).
constexpr int kJoin = 1024, kParts = 256;

__global__ void __launch_bounds__(kJoin)
k_balance_join(BalanceArgs a, int parts) {
  __shared__ double s_p[kJoin / 64][64];
  __shared__ int s_c[kJoin / 64][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, e = blockIdx.x * 64 + lane;
  double p = 0.0;
  int c = 0;
  if (e <= E) {
    constexpr int MOST = kParts / (kJoin / 64);  // all of a wave's parts at once; past the last one the last again, not used
    int2 v[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) v[i] = a.part[(int64_t)min(wave + i * (kJoin / 64), parts - 1) * (E + 1) + e];
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
  if (wave == 0 && e <= E) {
    for (int w = 1; w < kJoin / 64; ++w) {
      p += s_p[w][lane];
      c += s_c[w][lane];
    }
    a.total_p[e] = p;
    a.counts[e] = c;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const volatile double* tp = a.total_p;
  const volatile int32_t* tc = a.counts;
  double sum = 0.0;
  for (int i = threadIdx.x; i < E; i += kJoin) sum += tp[i] * (double)tc[i];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) s_p[wave][0] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < kJoin / 64; ++w) sum += s_p[w][0];
  const double n = (double)tc[E];
  a.losses[0] = n > 0 ? (float)(sum * E / (n * n * a.K)) : 0.f;
  a.losses[1] = n > 0 ? (float)(tp[E] / n) : 0.f;
}

// grid: as many workgroups as fill the chip; a wave per row.  f of the lane's columns stays in registers.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(64 * kWaves)
k_balance_grad(BalanceGradArgs a) {
  extern __shared__ __attribute__((aligned(16))) float s_pairs[];  // [kWaves][E rounded up to 64 VEC NV], with w
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, K = a.K;
  const float n = (float)a.counts[E];
  const float ga = a.dlosses && n > 0 ? a.dlosses[0] * ((float)E / n) : 0.f, gb = a.dlosses && n > 0 ? a.dlosses[1] * (2.f / n) : 0.f;
  const float per = n > 0 ? 1.f / (n * (float)K) : 0.f;
  float f[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int j = (i * 64 + lane) * VEC + e;
      f[i][e] = j < E ? (float)a.counts[j] * per : 0.f;
    }
  float* mine = s_pairs + wave * (64 * VEC * NV);
  if (a.w) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) mine[(i * 64 + lane) * VEC + e] = 0.f;
  }
  // a row is in flight while the one before it is used; one that is not live is not read, past the end the last row is
  const int64_t step = (int64_t)gridDim.x * kWaves;
  LogitRow<T, VEC, NV> next;
  float next_lse = -kInf, next_w = 0.f, next_dw = 0.f;
  int next_id = -1;
  auto fetch = [&](int64_t t, float lse) {
    t = min(t, a.T - 1);
    next_lse = lse;
    if (lse == -kInf) return;
    if (a.dlosses) next.load(reinterpret_cast<const T*>(a.logits) + t * a.ld, E, lane);
    if (a.w && lane < K) {
      next_id = a.ids[t * K + lane];
      next_w = a.w[t * K + lane];
      next_dw = a.dw[t * K + lane];
    }
  };
  int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  float after = -kInf;  // the lse of the row after the next
  if (t < a.T) {
    fetch(t, a.lse[t]);
    after = a.lse[min(t + step, a.T - 1)];
  }
  for (; t < a.T; t += step) {
    T* out = reinterpret_cast<T*>(a.dlogits) + t * a.ldd;
    const float lse = next_lse, w_k = next_w, dw_k = next_dw;
    const int id = next_id;
    float v[NV][VEC];
    if (lse != -kInf && a.dlosses) next.widen(E, lane, v);
    fetch(t + step, after);
    after = a.lse[min(t + 2 * step, a.T - 1)];
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
            v[i][e] = expf(v[i][e] - top);
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
      typename LogitVec<T, VEC>::V o;
      if constexpr (VEC == 1) {
        o = (T)v[i][0];
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = (T)v[i][e];
      }
      *reinterpret_cast<typename LogitVec<T, VEC>::V*>(out + j) = o;
    }
  }
}

// calls f with the logits' type, the vector width and the vectors of a lane
template <typename T, int VEC, typename F>
void with_vectors(int E, F f) {
  const int n = (E + 64 * VEC - 1) / (64 * VEC);
  if (n <= 1) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 1>{});
  else if (n <= 2) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 2>{});
  else if (n <= 4) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 4>{});
  else if (n <= 8) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 8>{});
  else if constexpr (VEC < 8) {
    if (n <= 16) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 16>{});
    else if constexpr (VEC == 1) f(T{}, std::integral_constant<int, VEC>{}, std::integral_constant<int, 64>{});
  }
}
template <typename F>
void with_logits(int dtype, bool vec, int E, F f) {
  if (dtype == EFF_DT_F32) vec ? with_vectors<float, 4>(E, f) : with_vectors<float, 1>(E, f);
  else if (dtype == EFF_DT_BF16) vec ? with_vectors<bf16_t, 8>(E, f) : with_vectors<bf16_t, 1>(E, f);
  else vec ? with_vectors<f16_t, 8>(E, f) : with_vectors<f16_t, 1>(E, f);
}
bool rows_of_vectors(int dtype, int E, const void* p, int64_t ld, const void* q, int64_t ldq) {
  const int64_t b = dtype == EFF_DT_F32 ? 4 : 2;
  return E * b % 16 == 0 && (uintptr_t)p % 16 == 0 && ld * b % 16 == 0 && (uintptr_t)q % 16 == 0 && ldq * b % 16 == 0;
}

}  // namespace

// Workgroups of the pass over the logits: one per CU, fewer where each wave would have fewer than four rows.
int64_t balance_parts(int64_t T) { return std::max<int64_t>(1, std::min<int64_t>(kParts, (T + 4 * kWaves - 1) / (4 * kWaves))); }

int64_t balance_workspace(int64_t T, int E) {
  const int64_t row = balance_parts(T) * (E + 1);
  return ((E + 1) * 8 + 8 + row * 8 + 255) / 256 * 256;
}

hipError_t launch_balance(BalanceArgs a, void* workspace, hipStream_t s) {
  const int parts = (int)balance_parts(a.T);
  a.total_p = static_cast<double*>(workspace);
  a.done = reinterpret_cast<int32_t*>(a.total_p + a.E + 1);
  a.part = reinterpret_cast<int2*>(a.done + 2);
  with_logits(a.dtype, rows_of_vectors(a.dtype, a.E, a.logits, a.ld, nullptr, 0), a.E, [&](auto t, auto vec, auto nv) {
    hipLaunchKernelGGL((k_balance<decltype(t), decltype(vec)::value, decltype(nv)::value>), dim3(parts), dim3(64 * kWaves),
                       (2 * a.E + 1) * 4, s, a);
  });
  hipLaunchKernelGGL(k_balance_join, dim3((a.E + 64) / 64), dim3(kJoin), 0, s, a, parts);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s) {
  const int grid = (int)std::min<int64_t>(2048, (a.T + kWaves - 1) / kWaves);
  with_logits(a.dtype, rows_of_vectors(a.dtype, a.E, a.logits, a.ld, a.dlogits, a.ldd), a.E, [&](auto t, auto vec, auto nv) {
    constexpr int V = decltype(vec)::value, N = decltype(nv)::value;
    hipLaunchKernelGGL((k_balance_grad<decltype(t), V, N>), dim3(grid), dim3(64 * kWaves), a.w ? kWaves * 64 * V * N * 4 : 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace eff
