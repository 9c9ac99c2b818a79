// Tokens sorted by expert and back: a stable counting sort of the (token, k) pairs, the copy of token
// rows into expert order, the weighted sum back to tokens, and both gradients.
//
// A pair whose id is outside [0, E) is unrouted (the -1 of a pair that another processor computes): it
// gets no place, its weight and rows are never read, and rows behind the last place stay as they were.
#include <algorithm>

#include "eff_internal.h"

namespace eff {
namespace {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// ---- sort ------------------------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortCounters = 32768;      // (wave, expert) counters in LDS: 128 KiB

// waves that count and place pairs, each over a contiguous part (the other waves only help scan)
__host__ __device__ inline int sort_waves(int E) {
  const int w = kSortCounters / E;
  return w < kSortThreads / 64 ? w : kSortThreads / 64;
}

// exclusive prefix of v over the workgroup's threads; *total the sum.  s: kSortThreads/64 ints of LDS.
__device__ inline int block_exclusive(int v, int* s, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) s[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSortThreads / 64; ++i) {
    const int c = s[i];
    before += i < wave ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// this wave's part [lo, hi) of [b0, b1): parts of whole 64-pair chunks in wave order
__device__ inline void wave_part(int64_t b0, int64_t b1, int nw, int wave, int64_t* lo, int64_t* hi) {
  const int64_t chunks = (b1 - b0 + 63) / 64, per = (chunks + nw - 1) / nw;
  *lo = min(b1, b0 + wave * per * 64);
  *hi = min(b1, b0 + (wave + 1) * per * 64);
}

// counts of this block's pairs into cnt[wave][E] (LDS, zeroed here)
__device__ inline void count_pairs(const int32_t* ids, int64_t b0, int64_t b1, int E, int nw, int* cnt) {
  for (int i = threadIdx.x; i < nw * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave < nw) {
    int64_t lo, hi;
    wave_part(b0, b1, nw, wave, &lo, &hi);
    for (int64_t i = lo + lane; i < hi; i += 64) {
      const int id = ids[i];
      if (id >= 0 && id < E) atomicAdd(&cnt[wave * E + id], 1);
    }
  }
  __syncthreads();
}

// places of this block's pairs: cnt[wave][e] holds the next place of expert e in this wave's part.
// The lanes of a chunk with the same id are found by one ballot per id bit; the lowest of them takes
// the counter forward for all, so a pair's place is its rank in pair order whatever the timing.
__device__ inline void place_pairs(const int32_t* ids, int64_t b0, int64_t b1, int E, int nw, int bits, int* cnt,
                                   int32_t* order, int32_t* pos) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave >= nw) return;
  int64_t lo, hi;
  wave_part(b0, b1, nw, wave, &lo, &hi);
  int next = lo + lane < hi ? ids[lo + lane] : -1;
  for (int64_t c = lo; c < hi; c += 64) {
    const int64_t i = c + lane;
    const int id = next;
    next = i + 64 < hi ? ids[i + 64] : -1;  // in flight while this chunk is ranked
    const bool ok = id >= 0 && id < E;
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= ((id >> b) & 1) ? m : ~m;
    }
    int base = 0;
    const int leader = ok ? __ffsll((unsigned long long)same) - 1 : lane;
    if (ok && lane == leader) base = atomicAdd(&cnt[wave * E + id], __popcll(same));
    base = __shfl(base, leader);
    if (i < hi) {
      int p = -1;
      if (ok) {
        p = base + __popcll(same & ((1ull << lane) - 1));
        order[p] = (int32_t)i;
      }
      pos[i] = p;
    }
  }
}

// Counting and placing by waves over contiguous parts keeps the order of equal ids without a sort.  Bound by latency: 160
// pairs over 512 experts 4.6 us in one workgroup; 49152 over 256 in 32 parts 4 + 10 us (in 64 parts, whose counts come in
// four trips and not one, 4 + 19).  One workgroup per part of the pairs.  hist null: the whole sort in one workgroup.  Otherwise hist
// [parts][E] holds every part's counts (k_sort_count), and each workgroup sums the columns it needs.
__global__ void __launch_bounds__(kSortThreads)
k_sort_place(const int32_t* __restrict__ ids, int64_t n, int E, int bits, int64_t part, const int32_t* __restrict__ hist,
             int32_t* __restrict__ offsets, int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  extern __shared__ int s_dyn[];
  __shared__ int s_scan[kSortThreads / 64];
  int* cnt = s_dyn;
  const int nw = sort_waves(E), tid = threadIdx.x, parts = gridDim.x, me = blockIdx.x;
  const int64_t b0 = me * part, b1 = min(n, b0 + part);
  count_pairs(ids, b0, b1, E, nw, cnt);
  // experts in rounds of one per thread; `run` carries the places of earlier rounds
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    int total = 0, before = 0;
    if (e < E) {
      if (hist) {
#pragma unroll 32
        for (int p = 0; p < parts; ++p) {
          const int c = hist[(int64_t)p * E + e];
          total += c;
          before += p < me ? c : 0;
        }
      } else {
        for (int w = 0; w < nw; ++w) total += cnt[w * E + e];
      }
    }
    int all;
    const int at = run + block_exclusive(total, s_scan, &all);
    if (e < E) {
      if (me == 0) offsets[e] = at;
      int next = at + before;
      for (int w = 0; w < nw; ++w) {
        const int c = cnt[w * E + e];
        cnt[w * E + e] = next;
        next += c;
      }
    }
    run += all;
  }
  if (me == 0 && tid == 0) offsets[E] = run;
  for (int64_t i = b0 + tid; i < b1; i += kSortThreads)  // places behind the last routed pair
    if (i >= run) order[i] = -1;
  __syncthreads();
  place_pairs(ids, b0, b1, E, nw, bits, cnt, order, pos);
}

__global__ void __launch_bounds__(kSortThreads)
k_sort_count(const int32_t* __restrict__ ids, int64_t n, int E, int64_t part, int32_t* __restrict__ hist) {
  extern __shared__ int s_dyn[];
  const int nw = sort_waves(E);
  const int64_t b0 = blockIdx.x * part, b1 = min(n, b0 + part);
  count_pairs(ids, b0, b1, E, nw, s_dyn);
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int c = 0;
    for (int w = 0; w < nw; ++w) c += s_dyn[w * E + e];
    hist[(int64_t)blockIdx.x * E + e] = c;
  }
}

// ---- rows ------------------------------------------------------------------------------------------

// VEC consecutive values of a row in fp32 (16 bytes per access with VEC * sizeof(T) == 16)
template <typename T, int VEC>
struct Pack {
  typedef T V __attribute__((ext_vector_type(VEC)));
};
template <typename T>
struct Pack<T, 1> {
  typedef T V;
};

template <typename T, int VEC>
__device__ inline void load_f32(const T* p, float* o) {
  const typename Pack<T, VEC>::V v = *reinterpret_cast<const typename Pack<T, VEC>::V*>(p);
  if constexpr (VEC == 1) {
    o[0] = (float)v;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = (float)v[i];
  }
}
template <typename T, int VEC>
__device__ inline void store_f32(T* p, const float* o) {
  typename Pack<T, VEC>::V v;
  if constexpr (VEC == 1) {
    v = (T)o[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (T)o[i];
  }
  *reinterpret_cast<typename Pack<T, VEC>::V*>(p) = v;
}

// vectors of one thread, 256 apart: rows that are no whole vectors move value by value, four in flight
template <int VEC>
constexpr int columns() { return VEC == 1 ? 4 : 1; }

// grid: (ceil(H / (256 U VEC)), T).  A token's row is read once and written to its K places (read once per place, most
// reads would hit L2, but a token's workgroup needs its positions only once this way).  8192 tokens x 6 x 4096: 430 MB in
// 84 us, 5.1 TB/s; a plain copy moves 5.0.  Stores past the caches changed nothing.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
k_dispatch(const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ pos, int K, int64_t H, T* __restrict__ xs,
           int64_t ldxs, int64_t rows) {
  constexpr int U = columns<VEC>();
  typedef typename Pack<T, VEC>::V V;
  const int64_t t = blockIdx.y, h0 = ((int64_t)blockIdx.x * U * 256 + threadIdx.x) * VEC;
  if (h0 >= H) return;
  V v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const V*>(x + t * ldx + min(h0 + u * 256 * VEC, H - VEC));
  for (int k = 0; k < K; ++k) {
    const int64_t p = pos[t * K + k];
    if (p < 0 || p >= rows) continue;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * 256 * VEC < H) *reinterpret_cast<V*>(xs + p * ldxs + h0 + u * 256 * VEC) = v[u];
  }
}

constexpr int kAhead = 4;

// grid: (ceil(H / (256 U VEC)), T).  out = residual + sum_k w * ys[pos], k ascending in fp32; w null: weights of 1.  8192
// tokens x 6 x 4096 with the residual: 497 MB in 95 us, 5.2 TB/s (one pair's row at a time: the same).
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
k_combine_rows(const T* __restrict__ ys, int64_t ldys, int64_t rows, const int32_t* __restrict__ pos,
               const float* __restrict__ w, int K, int64_t H, const T* residual, int64_t ldr, T* out, int64_t ldo) {
  constexpr int U = columns<VEC>();
  typedef typename Pack<T, VEC>::V V;
  const int64_t t = blockIdx.y, h0 = ((int64_t)blockIdx.x * U * 256 + threadIdx.x) * VEC;
  if (h0 >= H) return;
  int64_t h[U];   // past the end the row's last values, which are not stored
#pragma unroll
  for (int u = 0; u < U; ++u) h[u] = min(h0 + u * 256 * VEC, H - VEC);
  float acc[U][VEC];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (residual) {
      load_f32<T, VEC>(residual + t * ldr + h[u], acc[u]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[u][i] = 0.f;
    }
  }
  // kAhead pairs' rows are loaded before the first is added; a pair without a row loads nothing
  for (int k0 = 0; k0 < K; k0 += kAhead) {
    V v[kAhead][U];
    float wk[kAhead];
    bool ok[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = t * K + min(k0 + i, K - 1);
      const int64_t p = pos[at];
      ok[i] = k0 + i < K && p >= 0 && p < rows;
      if (ok[i]) {
        wk[i] = w ? w[at] : 1.f;
#pragma unroll
        for (int u = 0; u < U; ++u) v[i][u] = *reinterpret_cast<const V*>(ys + p * ldys + h[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!ok[i]) continue;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (VEC == 1) {
          acc[u][0] = fmaf(wk[i], (float)v[i][u], acc[u][0]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[u][e] = fmaf(wk[i], (float)v[i][u][e], acc[u][e]);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (h0 + u * 256 * VEC < H) store_f32<T, VEC>(out + t * ldo + h[u], acc[u]);
}

// grid: T workgroups of 4 waves; wave w takes the pairs k = w, w+4, ...: dys = w * dout and, with dw, the
// dot product of dout and ys (64 lane sums in column order, folded pairwise).  dout is read from HBM once, by the other
// pairs from L2.  4096 tokens x 8 x 2048: 286 MB in 50 us on the same rows again, 64 on others, 4.5 TB/s.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
k_combine_grad(const T* __restrict__ dout, int64_t ldd, const T* __restrict__ ys, int64_t ldys, int64_t rows,
               const int32_t* __restrict__ pos, const float* __restrict__ w, int K, int64_t H, T* __restrict__ dys,
               int64_t lddys, float* __restrict__ dw) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const T* d = dout + t * ldd;
  for (int k = threadIdx.x >> 6; k < K; k += 4) {
    const int64_t p = pos[t * K + k];
    const bool ok = p >= 0 && p < rows;
    float sum = 0.f;
    if (ok) {
      const float wk = w[t * K + k];
      constexpr int U = VEC == 1 ? 8 : 2;  // vectors in flight; past the end the row's last one, which is not used
      for (int64_t h0 = lane * VEC; h0 < H; h0 += 64 * VEC * U) {
        float dv[U][VEC], yv[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t h = min(h0 + u * 64 * VEC, H - VEC);
          load_f32<T, VEC>(d + h, dv[u]);
          if (dw) load_f32<T, VEC>(ys + p * ldys + h, yv[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t h = h0 + u * 64 * VEC;
          if (h >= H) break;
          if (dw) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum = fmaf(dv[u][i], yv[u][i], sum);
          }
#pragma unroll
          for (int i = 0; i < VEC; ++i) dv[u][i] *= wk;
          store_f32<T, VEC>(dys + p * lddys + h, dv[u]);
        }
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    }
    if (dw && lane == 0) dw[t * K + k] = sum;
  }
}

bool vec16(int bytes, int64_t H, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  if (H * bytes % 16) return false;
  for (const void* p : ptrs)
    if ((uintptr_t)p % 16) return false;
  for (int64_t l : lds)
    if (l * bytes % 16) return false;
  return true;
}

// calls f with a value of the row type and the vector width (16 bytes, or single values)
template <typename F>
hipError_t with_type(int dtype, bool v, F f) {
  switch (dtype) {
    case EFF_DT_BF16: return v ? f(bf16_t{}, std::integral_constant<int, 8>{}) : f(bf16_t{}, std::integral_constant<int, 1>{});
    case EFF_DT_F16: return v ? f(f16_t{}, std::integral_constant<int, 8>{}) : f(f16_t{}, std::integral_constant<int, 1>{});
    default: return v ? f(float{}, std::integral_constant<int, 4>{}) : f(float{}, std::integral_constant<int, 1>{});
  }
}

constexpr int64_t kGridX = 1 << 23;  // workgroups of 256 threads: a grid's threads stay below 2^32
constexpr int64_t kGridY = 65535;  // tokens per launch of the two-dimensional grids

}  // namespace

// Up to kSortOne pairs one workgroup does the whole sort (one launch): in us, one workgroup and 32 parts, 4096 pairs over 256
// experts 10.1 and 12.7, over 4096 19 and 30; 8192 14.3 and 12.9, 27 and 30; 16384 22.7 and 13.0, 45 and 31.
constexpr int64_t kSortOne = 8192;
// Parts beyond: 32, whose counts are read in one go, and 128 above 256K pairs.  32 and 128: 49152 pairs over 256 14.4 and 24.7,
// 256K 22 and 27, over 4096 51 and 84; 512K 32 and 30, 72 and 91; 1M 52 and 35, 124 and 106; 4M 200 and 80, 426 and 181.
constexpr int64_t kSortParts = 128;
int64_t sort_parts(int64_t n) { return n <= (int64_t)1 << 18 ? 32 : kSortParts; }

int64_t sort_workspace(int64_t n, int E) {
  if (n <= kSortOne) return 0;
  return (sort_parts(n) * E * 4 + 255) / 256 * 256;
}

hipError_t launch_sort_tokens(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                              int32_t* hist, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  const size_t lds = (size_t)sort_waves(E) * E * 4;
  if (n <= kSortOne) {
    hipLaunchKernelGGL(k_sort_place, dim3(1), dim3(kSortThreads), lds, s, ids, n, E, bits, n, nullptr, offsets, order, pos);
    return hipGetLastError();
  }
  const int64_t want = sort_parts(n), part = ((n + want - 1) / want + 63) / 64 * 64;
  const int parts = (int)((n + part - 1) / part);
  hipLaunchKernelGGL(k_sort_count, dim3(parts), dim3(kSortThreads), lds, s, ids, n, E, part, hist);
  hipLaunchKernelGGL(k_sort_place, dim3(parts), dim3(kSortThreads), lds, s, ids, n, E, bits, part, hist, offsets, order, pos);
  return hipGetLastError();
}

hipError_t launch_dispatch_tokens(int dtype, const void* x, int64_t ldx, const int32_t* pos, int64_t T, int K, int64_t H,
                                  void* xs, int64_t ldxs, int64_t rows, hipStream_t s) {
  const bool v = vec16(dtype == EFF_DT_F32 ? 4 : 2, H, {x, xs}, {ldx, ldxs});
  return with_type(dtype, v, [&](auto t, auto vec) {
    typedef decltype(t) E;
    constexpr int V = decltype(vec)::value, W = 256 * V * columns<V>();
    for (int64_t t0 = 0; t0 < T; t0 += kGridY) {
      const dim3 g((unsigned)((H + W - 1) / W), (unsigned)std::min(kGridY, T - t0));
      hipLaunchKernelGGL((k_dispatch<E, V>), g, dim3(256), 0, s, (const E*)x + t0 * ldx, ldx, pos + t0 * K, K, H, (E*)xs,
                         ldxs, rows);
    }
    return hipGetLastError();
  });
}

hipError_t launch_combine_tokens(int dtype, const void* ys, int64_t ldys, int64_t rows, const int32_t* pos, const float* w,
                                 int64_t T, int K, int64_t H, const void* residual, int64_t ldr, void* out, int64_t ldo,
                                 hipStream_t s) {
  const bool v = vec16(dtype == EFF_DT_F32 ? 4 : 2, H, {ys, residual, out}, {ldys, residual ? ldr : 0, ldo});
  return with_type(dtype, v, [&](auto t, auto vec) {
    typedef decltype(t) E;
    constexpr int V = decltype(vec)::value, W = 256 * V * columns<V>();
    for (int64_t t0 = 0; t0 < T; t0 += kGridY) {
      const dim3 g((unsigned)((H + W - 1) / W), (unsigned)std::min(kGridY, T - t0));
      hipLaunchKernelGGL((k_combine_rows<E, V>), g, dim3(256), 0, s, (const E*)ys, ldys, rows, pos + t0 * K,
                         w ? w + t0 * K : nullptr, K, H, residual ? (const E*)residual + t0 * ldr : nullptr, ldr,
                         (E*)out + t0 * ldo, ldo);
    }
    return hipGetLastError();
  });
}

hipError_t launch_combine_tokens_grad(int dtype, const void* dout, int64_t ldd, const void* ys, int64_t ldys, int64_t rows,
                                      const int32_t* pos, const float* w, int64_t T, int K, int64_t H, void* dys,
                                      int64_t lddys, float* dw, hipStream_t s) {
  const bool v = vec16(dtype == EFF_DT_F32 ? 4 : 2, H, {dout, dw ? ys : nullptr, dys}, {ldd, dw ? ldys : 0, lddys});
  return with_type(dtype, v, [&](auto t, auto vec) {
    typedef decltype(t) E;
    constexpr int V = decltype(vec)::value;
    for (int64_t t0 = 0; t0 < T; t0 += kGridX)
      hipLaunchKernelGGL((k_combine_grad<E, V>), dim3((unsigned)std::min(kGridX, T - t0)), dim3(256), 0, s,
                         (const E*)dout + t0 * ldd, ldd, (const E*)ys, ldys, rows, pos + t0 * K, w + t0 * K, K, H, (E*)dys, lddys,
                         dw ? dw + t0 * K : nullptr);
    return hipGetLastError();
  });
}

// Per device, once: the sort kernels' counters take up to 128 KiB of dynamic LDS.
hipError_t tokens_setup() {
  const void* fs[] = {reinterpret_cast<const void*>(&k_sort_place), reinterpret_cast<const void*>(&k_sort_count)};
  for (const void* f : fs) {
    const hipError_t err = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kSortCounters * 4);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace eff
