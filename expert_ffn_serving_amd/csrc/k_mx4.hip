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
#include <cmath>
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
typedef bf16_t bf16x2_t __attribute__((ext_vector_type(2)));
typedef f16_t f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <>
struct Vec8<float> { typedef f32x8_t V; };

// 8 values at any place (the hardware takes 16-byte accesses at any address)
template <typename T>
struct Loose8 {
  typedef typename Vec8<T>::V V __attribute__((aligned(sizeof(T))));
};

// the largest of v over the 4 lanes of a quad
__device__ inline uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}
// the scale byte of a block from the largest magnitude of this lane's 8 values; the 4 lanes of a quad hold a block.  The
// magnitudes of 16-bit values are compared as integers, two at a time.  A subnormal fp32 number's exponent is below -126,
// and -127 is the least there is.
__device__ inline int mx4_scale(uint32_t bits) {  // of the largest magnitude in fp32
  return bits >= 0x7f800000u ? kNaNScale : max((int)(bits >> 23) - 2, 0);
}
template <typename V>
__device__ inline uint32_t top_of_16(const V& v) {
  struct Pairs { u16x2_t p[4]; };
  const Pairs w = __builtin_bit_cast(Pairs, v);
  u16x2_t m = w.p[0] & (uint16_t)0x7fff;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, w.p[i] & (uint16_t)0x7fff);
  return max((uint32_t)m[0], (uint32_t)m[1]);
}
// the magnitude's bits in fp32
__device__ inline uint32_t bits_of_16(const bf16x8_t&, uint32_t top) { return top << 16; }
__device__ inline uint32_t bits_of_16(const f16x8_t&, uint32_t top) {
  const uint16_t t = (uint16_t)top;
  return __float_as_uint((float)__builtin_bit_cast(f16_t, t));
}
__device__ inline int block_scale(const bf16x8_t& v) { return mx4_scale(bits_of_16(v, quad_max(top_of_16(v)))); }
__device__ inline int block_scale(const f16x8_t& v) { return mx4_scale(bits_of_16(v, quad_max(top_of_16(v)))); }
__device__ inline int block_scale(const f32x8_t& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return mx4_scale(quad_max(m));
}
// 2^(scale - 127) as the conversions take it: they look at the exponent, of which 0 is 2^-127
__device__ inline float scale_value(int scale) { return __uint_as_float((uint32_t)scale << 23); }

// 8 values to codes: v_cvt_scalef32_pk_fp4_* rounds to nearest, ties to even, and gives 6 beyond 6
__device__ inline uint32_t to_codes(const bf16x8_t& v, float s) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0, bf16x2_t{v[0], v[1]}, s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2_t{v[2], v[3]}, s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2_t{v[4], v[5]}, s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2_t{v[6], v[7]}, s, 3);
}
__device__ inline uint32_t to_codes(const f16x8_t& v, float s) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(0, f16x2_t{v[0], v[1]}, s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f16x2_t{v[2], v[3]}, s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f16x2_t{v[4], v[5]}, s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f16x2_t{v[6], v[7]}, s, 3);
}
__device__ inline uint32_t to_codes(const f32x8_t& v, float s) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
}
// and back, rounded once to T
__device__ inline void from_codes(uint32_t c, float s, bf16x8_t* v) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
  *v = bf16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
__device__ inline void from_codes(uint32_t c, float s, f32x8_t* v) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  *v = f32x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
__device__ inline void from_codes(uint32_t c, float s, f16x8_t* v) {
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1);
  const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3);
  *v = f16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// Pieces of 8 values, 4 a block and 16 a unit.  A workgroup takes 1024 consecutive ones, a thread 4 of them 256 apart, whose
// loads are all under way before the first is used.  FLAT: the rows of both sides follow each other without a gap, so that
// the number of a piece is its place.  Bound by HBM: 65536 x 4096 bf16 to codes 143 us, 4.7 TB/s, and back 104 us, 6.5 TB/s.
constexpr int kPieces = 4;

// where a piece is: its row and first value in the row
__device__ inline void piece_at(const Mx4Rows& a, uint32_t i, int64_t* row, int64_t* k0, int64_t* unit) {
  const uint32_t u = i >> 4, r = u / (uint32_t)a.units;
  *row = r;
  *unit = u - r * (uint32_t)a.units;
  *k0 = *unit * 128 + (i & 15) * 8;
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(256)
k_mx4_quantize(Mx4Rows a) {
  typedef typename Vec8<T>::V V8;
  const uint32_t i0 = blockIdx.x * (256 * kPieces) + threadIdx.x;
  uint32_t lo = 0, hi = (uint32_t)(a.rows * a.units * 16);
  if (a.offsets) {  // rows in no group are not read
    const int64_t per = a.units * 16;
    lo = (uint32_t)(min(max((int64_t)a.offsets[0] - a.row0, (int64_t)0), a.rows) * per);
    hi = (uint32_t)(min(max((int64_t)a.offsets[a.groups] - a.row0, (int64_t)0), a.rows) * per);
  }
  if (lo >= hi) return;
  const T* x = reinterpret_cast<const T*>(a.x);
  V8 v[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const uint32_t i = min(max(i0 + p * 256, lo), hi - 1);  // outside: the nearest piece again, which is not used
    v[p] = V8{};
    if constexpr (FLAT) {
      v[p] = *reinterpret_cast<const typename Loose8<T>::V*>(x + (int64_t)i * 8);
    } else {
      int64_t row, k0, unit;
      piece_at(a, i, &row, &k0, &unit);
      const T* at = x + row * a.ldx + k0;
      if (k0 + 8 <= a.k) {
        v[p] = *reinterpret_cast<const typename Loose8<T>::V*>(at);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k0 + e < a.k) v[p][e] = at[e];
      }
    }
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const uint32_t i = i0 + p * 256;
    const int scale = block_scale(v[p]);  // lo, hi and the end are multiples of 16: a quad is inside or not
    const uint32_t c = scale == kNaNScale ? 0u : to_codes(v[p], scale_value(scale));
    if (i < lo || i >= hi) continue;
    if constexpr (FLAT) {
      *reinterpret_cast<uint32_t*>(a.codes + (int64_t)i * 4) = c;
      if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = (uint8_t)scale;
    } else {
      int64_t row, k0, unit;
      piece_at(a, i, &row, &k0, &unit);
      *reinterpret_cast<uint32_t*>(a.codes + row * a.ldc + unit * 64 + (i & 15) * 4) = c;
      if ((threadIdx.x & 3) == 0) a.scales[row * a.lds + unit * 4 + ((i & 15) >> 2)] = (uint8_t)scale;
    }
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(256)
k_mx4_dequantize(Mx4Rows a) {
  typedef typename Vec8<T>::V V8;
  const uint32_t i0 = blockIdx.x * (256 * kPieces) + threadIdx.x, hi = (uint32_t)(a.rows * a.units * 16);
  uint32_t c[kPieces];
  int scale[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const uint32_t i = min(i0 + p * 256, hi - 1);
    if constexpr (FLAT) {
      c[p] = *reinterpret_cast<const uint32_t*>(a.codes + (int64_t)i * 4);
      scale[p] = a.scales[i >> 2];
    } else {
      int64_t row, k0, unit;
      piece_at(a, i, &row, &k0, &unit);
      c[p] = *reinterpret_cast<const uint32_t*>(a.codes + row * a.ldc + unit * 64 + (i & 15) * 4);
      scale[p] = a.scales[row * a.lds + unit * 4 + ((i & 15) >> 2)];
    }
  }
  T* y = reinterpret_cast<T*>(a.y);
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const uint32_t i = i0 + p * 256;
    if (i >= hi) continue;
    V8 v;
    from_codes(c[p], scale_value(scale[p]), &v);
    if (scale[p] == kNaNScale) v = (V8)(T)__builtin_nanf("");
    if constexpr (FLAT) {
      *reinterpret_cast<typename Loose8<T>::V*>(y + (int64_t)i * 8) = v;
    } else {
      int64_t row, k0, unit;
      piece_at(a, i, &row, &k0, &unit);
      T* at = y + row * a.ldy + k0;
      if (k0 + 8 <= a.k) {
        *reinterpret_cast<typename Loose8<T>::V*>(at) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k0 + e < a.k) at[e] = v[e];
      }
    }
  }
}

// ---- products --------------------------------------------------------------------------------------------

// A block of 32 16-bit values in one lane: its codes and scale.
template <typename V8>
__device__ inline i32x4_t quantise_block(const V8* v, int* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, top_of_16(v[i]));
  *scale = mx4_scale(bits_of_16(v[0], top));
  const float s = scale_value(*scale);
  i32x4_t c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = *scale == kNaNScale ? 0 : (int)to_codes(v[i], s);
  return c;
}

// 16 W rows against 16 x rows over 128 k: lane (r, q) holds 32 values of row r, the q-th of 4 blocks, and their scale in byte
// B of sw and sx.  The sums: W rows 4 q .. 4 q + 3 of x row r.
template <int B>
__device__ inline f32x4_t mfma4(i32x4_t w, i32x4_t x, f32x4_t c, int sw, int sx) {
  const i32x8_t a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1), b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, B, sw, B, sx);
}

// ---- tiles through LDS ----------------------------------------------------------------------------------
//
// Workgroup = BM rows x BN columns, WM x WN waves, steps of 256 k: 128 bytes of codes a row, which go to LDS by direct 16-byte
// copies as those of 64 16-bit values do (k_mm_tile in k_matmul.hip: the same tiles, chunk places and epilogue; C::BK counts 2-byte
// units).  A matrix instruction takes 128 k; which 32 of them a lane holds is free as long as x and W agree, so the lane
// of block pair q takes blocks 2 q and 2 q + 1 of a step, one for each of its two instructions: its two scale bytes
// lie side by side and are read as one 16-bit value, whose byte the instruction picks.
//
// Scales come to LDS for two steps at a time, 16 bytes a row (one line of a row holds those of 16 steps: fetched step by step
// it would be requested as often as the codes' lines): [buffer][row][16], x rows first.
//
// 256 x 256 (AHEAD): 8192 x 8192 x 8192 270 us, 4.1 PFLOP/s, 8192 x 2 x 4096 x 4096 SwiGLU 155 us, 3.5; the instructions alone, on
// random codes in registers, reach 6.1 (8.7 on zeros: the clock gives way to the power drawn).  By the fit at plan_mx4 the steps run at
// 5.2 and a tile spends 12 us outside them; what takes those has not been measured.  Its workgroups, one a CU, take tile
// after tile where the sums are stored from registers, the next tile's first step on its way meanwhile: 162 -> 157,
// 277 -> 271 us.  64 x 128 for groups: 12288 rows over 256 experts, 4096 -> 2 x 2048, 470 us, 4.9 TB/s of W; with a row a group
// (512 groups, 2560 -> 2 x 640, 138 us) W comes at 6.5 through the same LDS.
template <int BM, int BN, int WM, int WN, int S, bool AHEAD>
using MxCfg = TileCfg<BM, BN, WM, WN, 64, S, AHEAD>;


// Buffers of two steps' scales: step t + S - 1 is copied while step t is used, so its buffer's last steps are behind t.
constexpr int scale_buffers(int S) { return (S + 2) / 2; }

template <typename T, class C, bool GLU>
__global__ void __launch_bounds__(C::TH)
k_mx4_tile(Mx4Args a) {
  constexpr int BM = C::BM, BN = C::BN, S = C::S, TH = C::TH, CK = 8;
  constexpr int TM = BM / C::WM, TN = BN / C::WN, MT = TM / 16, NT = TN / 16;
  constexpr int HALVES = GLU ? 2 : 1, NTH = NT / HALVES, TNH = TN / HALVES, BNH = BN / HALVES, RUN = NTH * 4;
  constexpr int XB = BM * 128, WB = BN * 128, STEP = XB + WB, SCALES = (BM + BN) * 16, SB = scale_buffers(S);
  // copies of one thread per step, and of scales every other one; where x has fewer rows than that, by the first waves alone
  constexpr int SX = (BM * CK + TH - 1) / TH, SW = BN * CK / TH, SCX = (BM * 4 + TH - 1) / TH, SCW = BN * 4 / TH;
  constexpr bool ALL_X = BM * CK % TH == 0, ALL_XS = BM * 4 % TH == 0;
  constexpr int CP = (ALL_X ? SX : 0) + SW;  // at least
  static_assert(C::BK == 64 && BN * CK % TH == 0 && BN * 4 % TH == 0 && (ALL_X || SX == 1) && (ALL_XS || SCX == 1) && TNH % 16 == 0 && NT % HALVES == 0, "tile");
  extern __shared__ __attribute__((aligned(128))) uint8_t s_tile[];
  int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const MmArgs& e = a.e;

  const int nt = (int)((e.N + BNH - 1) / BNH);
  int g = 0, nt_i, job = blockIdx.x;
  int64_t m0, m1, n0;
  // an XCD's workgroups take a contiguous part of the tiles, in bands of 8 row tiles, as in k_mm_tile
  auto locate = [&]() __attribute__((always_inline)) {
    const int all = a.tiles, xcd = job & 7, id = xcd * (all >> 3) + min(xcd, all & 7) + (job >> 3);
    const int mts = all / nt, band = id / (8 * nt), in_band = id - band * 8 * nt, height = min(8, mts - band * 8);
    nt_i = in_band / height;
    m0 = (int64_t)(band * 8 + in_band % height) * BM;
    m1 = min(e.M, m0 + BM);
    n0 = (int64_t)nt_i * BNH;
  };
  if (e.mode == MM_ROW_GROUPS) {
    nt_i = blockIdx.x % nt;
    if (!find_tile<BM>(e.offsets, e.groups, e.M, blockIdx.x / nt, reinterpret_cast<int*>(s_tile), &g, &m0, &m1)) return;
    n0 = (int64_t)nt_i * BNH;
  } else {
    locate();
  }

  const int64_t up_codes = GLU ? e.N * a.ldw : 0, up_scales = GLU ? e.N * a.ldws : 0;
  const int bytes = a.units * 64;
  // This thread's copies: byte offsets from uniform addresses that advance with the steps (plan_mx4 keeps them < 2^32), of the
  // first one and of the tile's last row; the others are a fixed number of rows further and end there.
  const uint8_t *bx, *bw, *bxs, *bws;
  uint32_t ox, ow, osx, osw, endx, endw, endsx, endsw;
  constexpr int PER = TH / CK, PERS = TH / 4;  // LDS rows of a copy
  static_assert((PER % TNH == 0 || TNH % PER == 0) && (PERS % TNH == 0 || TNH % PERS == 0), "copies of rows side by side");
  auto w_at = [](int row) { return (row / TN) * TNH + row % TNH; };
  // the chunk of every copy
  auto chunk_x = [&] { return (tid % CK) ^ swz_rows<64, 1>(tid / CK); };
  auto chunk_w = [&] { return (tid % CK) ^ swz_rows<64, RUN>(tid / CK); };
  static_assert(PER % 8 == 0 && PER % (2 * RUN) == 0, "copies PER rows apart have the same chunk");
  auto aim = [&]() __attribute__((always_inline)) {
    const int64_t lx = m1 - 1 - m0, lw = e.N - 1 - n0;
    ox = (uint32_t)(tid / CK * a.ldx) + chunk_x() * 16, endx = (uint32_t)(lx * a.ldx) + chunk_x() * 16;
    ow = (uint32_t)(w_at(tid / CK) * a.ldw) + chunk_w() * 16, endw = (uint32_t)(min(lw, (int64_t)BN - 1) * a.ldw) + chunk_w() * 16;
    osx = (uint32_t)(tid / 4 * a.ldxs) + (tid & 3) * 4, endsx = (uint32_t)(lx * a.ldxs) + (tid & 3) * 4;
    osw = (uint32_t)(w_at(tid / 4) * a.ldws) + (tid & 3) * 4, endsw = (uint32_t)(min(lw, (int64_t)BN - 1) * a.ldws) + (tid & 3) * 4;
    bx = a.x + m0 * a.ldx, bw = a.w + g * a.sw + n0 * a.ldw;
    bxs = a.xs + m0 * a.ldxs, bws = a.ws + g * a.sws + n0 * a.ldws;
  };
  aim();
  const uint32_t lds0 = lds_address(s_tile), lds_s = lds0 + S * STEP;
  const int steps = (a.units + 1) / 2;

  // Where a row ends inside a step its last unit (or the first one, of the scales) is copied once more; drop() takes it out.
  auto issue = [&](int t) __attribute__((always_inline)) {
    const uint32_t base = lds0 + (t % S) * STEP + wave * 1024;
    const int left = min(128, bytes - t * 128);
    const uint8_t *sx = bx + (int64_t)t * 128, *sw = bw + (int64_t)t * 128;
    // a wave copies whole rows, on one side of a tile's gate and up rows
    auto side = [&](int i) { return GLU && ((i * TH + wave * 64) / CK) % TN >= TNH ? sw + up_codes : sw; };
    const uint32_t back_x = left < 128 && chunk_x() >= 4 ? 64 : 0, back_w = left < 128 && chunk_w() >= 4 ? 64 : 0;
#pragma unroll
    for (int i = 0; i < SX; ++i)
      if (ALL_X || wave * 64 < BM * CK) lds_copy16(sx, min(ox + i * PER * (uint32_t)a.ldx, endx) - back_x, base + i * (TH * 16));
#pragma unroll
    for (int i = 0; i < SW; ++i) lds_copy16(side(i), min(ow + w_at(i * PER) * (uint32_t)a.ldw, endw) - back_w, base + XB + i * (TH * 16));
    if (t % 2 == 0) {  // the scales of steps t and t + 1, 4 units: a wave's copy has 16 rows of 4 times 4 bytes
      const uint32_t at = lds_s + (t / 2 % SB) * SCALES + wave * 256;
      const int units = a.units - t * 2;
      const uint8_t *sxs = bxs + (int64_t)t * 8, *sws = bws + (int64_t)t * 8;
      const uint32_t back = (tid & 3) < units ? 0 : (tid & 3) * 4;
#pragma unroll
      for (int i = 0; i < SCX; ++i)
        if (ALL_XS || wave * 64 < BM * 4) lds_copy4(sxs, min(osx + i * PERS * (uint32_t)a.ldxs, endsx) - back, at + i * (TH * 4));
#pragma unroll
      for (int i = 0; i < SCW; ++i)
        lds_copy4(GLU && (i * (TH / 4) + wave * 16) % TN >= TNH ? sws + up_scales : sws, min(osw + w_at(i * PERS) * (uint32_t)a.ldws, endsw) - back, at + BM * 16 + i * (TH * 4));
    }
  };

#pragma unroll
  for (int t = 0; t < S - 1; ++t)
    if (t < steps) issue(t);
  while (true) {
    if (C::AHEAD) asm volatile("" : "+v"(tid));  // what depends on it is computed again and holds no registers from tile to tile
    const int lane = tid & 63, q = lane >> 4, r = lane & 15;
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto x_row = [&](int i) { return wm * TM + i * 16 + r; };
    auto w_row = [&](int j) { return wn * TN + (j / NTH) * TNH + (r >> 2) * RUN + (j % NTH) * 4 + (r & 3); };
    auto frag_x = [&](const uint8_t* b, int i, int ks) __attribute__((always_inline)) {
      const int row = x_row(i);
      return *reinterpret_cast<const i32x4_t*>(b + row * 128 + (((2 * q + ks) ^ swz_rows<64, 1>(row)) << 4));
    };
    auto frag_w = [&](const uint8_t* b, int j, int ks) __attribute__((always_inline)) {
      const int row = w_row(j);
      return *reinterpret_cast<const i32x4_t*>(b + XB + row * 128 + (((2 * q + ks) ^ swz_rows<64, RUN>(row)) << 4));
    };
    auto scale_of = [&](int t, int row) -> int {
      return *reinterpret_cast<const uint16_t*>(s_tile + S * STEP + (t / 2 % SB) * SCALES + row * 16 + (t & 1) * 8 + q * 2);
    };
    auto buffer = [&](int t) { return s_tile + (t % S) * STEP; };

    // this wave's operands of a step's instruction ks
    i32x4_t fw[2][NT], fx[MT];
    int sw[NT], sx[MT];
    auto read_w = [&](int into, int t, int ks) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fw[into][j] = frag_w(buffer(t), j, ks);
    };
    auto products = [&](auto ks, int i) __attribute__((always_inline)) {
      constexpr int B = decltype(ks)::value;
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma4<B>(fw[B][j], fx[i], acc[i][j], sw[j], sx[i]);
      if constexpr (C::AHEAD) {
        // the products stay on this side of the barrier and of the branches around it (no instruction, only a use of the sums),
        // and an operand is read again behind them, not into a second register
#pragma unroll
        for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // the last step's second unit where there is none: zeros on W's side, for the lanes q >= 2 that hold it
    const bool odd = a.units & 1;
    auto drop = [&](int set) __attribute__((always_inline)) {
      if (odd && q >= 2) {
#pragma unroll
        for (int j = 0; j < NT; ++j) fw[set][j] = i32x4_t{0, 0, 0, 0}, sw[j] = 0;
      }
    };
    const std::integral_constant<int, 0> first;
    const std::integral_constant<int, 1> second;
    if constexpr (C::AHEAD) {
      // as in k_mm_tile: an x operand is read again as soon as its products are issued, the w operands half a step ahead into a
      // second set, and the barrier of a step stands inside the last half's products
      static_assert(S == 2, "two buffers");
      constexpr int LATE = 2;  // x operands whose products stand before the barrier
      vm_wait<0>();
      meet();
      if (steps > 1) issue(1);
      read_w(0, 0, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j) sw[j] = scale_of(0, BM + w_row(j));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sx[i] = scale_of(0, x_row(i));
        fx[i] = frag_x(buffer(0), i, 0);
      }
      for (int t = 0; t < steps - 1; ++t) {
        read_w(1, t, 1);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          products(first, i);
          fx[i] = frag_x(buffer(t), i, 1);
        }
#pragma unroll
        for (int i = 0; i < LATE; ++i) products(second, i);
        vm_wait<0>();
        meet();  // step t + 1 is in LDS and step t in registers
        if (t + 2 < steps) issue(t + 2);
        read_w(0, t + 1, 0);
        int next[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) next[j] = scale_of(t + 1, BM + w_row(j));
#pragma unroll
        for (int i = 0; i < LATE; ++i) {
          sx[i] = scale_of(t + 1, x_row(i));
          fx[i] = frag_x(buffer(t + 1), i, 0);
        }
#pragma unroll
        for (int i = LATE; i < MT; ++i) {
          products(second, i);
          sx[i] = scale_of(t + 1, x_row(i));
          fx[i] = frag_x(buffer(t + 1), i, 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) sw[j] = next[j];
      }
      read_w(1, steps - 1, 1);
      drop(0);
      drop(1);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        products(first, i);
        fx[i] = frag_x(buffer(steps - 1), i, 1);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) products(second, i);
    } else {
      for (int t = 0; t < steps; ++t) {
        // copies issued after step t's: at least CP for every later step (scales beside, which only makes the wait stricter)
        if (t + S - 1 > steps) vm_wait<0>();
        else vm_wait<(S - 2) * CP>();
        meet();
        if (t + S - 1 < steps) issue(t + S - 1);
#pragma unroll
        for (int i = 0; i < MT; ++i) sx[i] = scale_of(t, x_row(i));
#pragma unroll
        for (int j = 0; j < NT; ++j) sw[j] = scale_of(t, BM + w_row(j));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          read_w(ks, t, ks);
          if (t == steps - 1) drop(ks);
#pragma unroll
          for (int i = 0; i < MT; ++i) fx[i] = frag_x(buffer(t), i, ks);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            if (ks == 0) products(first, i);
            else products(second, i);
          }
        }
      }
    }
    if (!e.simple) {
      // through LDS where there is more to do than SwiGLU and a residual, whose code would stand there for every piece
      if constexpr (C::BM < 64) store_regs<T, C, GLU, false>(e, acc, g, m0, m1, n0);
      else store_tile<T, C, true, GLU>(e, acc, s_tile, g, m0, m1, n0);
      return;
    }
    const int64_t done0 = m0, done1 = m1, done_n = n0;
    bool more = false;
    if constexpr (C::AHEAD) {  // the next tile's first step is on its way while this one's sums are stored
      job += gridDim.x;
      more = e.mode != MM_ROW_GROUPS && job < a.tiles;
      if (more) {
        asm volatile("" : "+v"(tid));
        locate();
        aim();
        meet();  // every wave has read the last step
        issue(0);
      }
    }
    store_regs<T, C, GLU, true>(e, acc, g, done0, done1, done_n);
    if (!more) return;
  }
}

// ---- few rows --------------------------------------------------------------------------------------------
//
// Up to 16 MT rows of x against 16 rows of W per workgroup (SwiGLU: 8 gate and 8 up rows), the k split over its waves, as
// k_mm_few does for 16 bits: every wave keeps U chunks of 256 k (2 KiB of W each) in flight in registers, nothing waits for a
// barrier before the end, where the waves' sums meet in LDS in wave order.
//
// RAW: x comes in 16 bits and every wave quantises what it multiplies, a lane its own blocks: for 16 rows, whose x
// is small next to W (16 rows, 4096 -> 2 x 2048: 8.5 us and not 12.3 for two launches and their workspace), and for more
// where there is little to compute (mx4_takes_raw).
template <int MT>
constexpr int mx4_unroll() { return MT >= 4 ? 1 : 2; }

template <typename T, int MT, bool GLU, bool RAW>
__global__ void __launch_bounds__(1024)
k_mx4_few(Mx4Args a, int slices) {
  constexpr int U = mx4_unroll<MT>(), BM = 16 * MT;
  typedef typename Vec8<T>::V V8;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_few[];
  f32x4_t* s_acc = reinterpret_cast<f32x4_t*>(s_few);  // [waves][MT][64]
  const MmArgs& e = a.e;
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int64_t tile = blockIdx.x / slices, n0 = (int64_t)(blockIdx.x % slices) * (GLU ? 8 : 16);
  int g = 0;
  int64_t m0 = tile * BM, m1 = min(e.M, m0 + BM);
  if (e.mode == MM_ROW_GROUPS && !find_tile<BM>(e.offsets, e.groups, e.M, (int)tile, reinterpret_cast<int*>(s_few), &g, &m0, &m1)) return;
  const int chunks = (a.units + 1) / 2;
  const int64_t col = min(n0 + (GLU ? r & 7 : r), e.N - 1), wr = col + (GLU && r >= 8 ? e.N : 0);
  const uint8_t *w = a.w + g * a.sw + wr * a.ldw + q * 32, *ws = a.ws + g * a.sws + wr * a.ldws + q * 2;
  const uint8_t *x[MT], *xs[MT];  // RAW: x the row's first value
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = min(m0 + i * 16 + r, m1 - 1);
    x[i] = RAW ? a.x + row * a.ldx * 2 : a.x + row * a.ldx + q * 32;
    xs[i] = a.xs + row * a.ldxs + q * 2;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  i32x4_t fw[U][2], fx[U][MT][2];
  V8 raw[U][MT][RAW ? 8 : 1];
  int sw[U], sx[U][MT];
  const int K = (int)e.K;
  const bool odd = a.units & 1;  // the last chunk has one unit: lanes q >= 2 have nothing there
  // chunk c of this wave's into slot s; past the end the first chunk again (not used)
  auto load = [&](int c, int s) {
    const bool none = c >= chunks || (odd && c == chunks - 1 && q >= 2);
    const int64_t at = none ? -(int64_t)q * 32 : (int64_t)c * 128, as = none ? -(int64_t)q * 2 : (int64_t)c * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fw[s][h] = *reinterpret_cast<const i32x4_t*>(w + at + h * 16);
      if constexpr (!RAW) {
#pragma unroll
        for (int i = 0; i < MT; ++i) fx[s][i][h] = *reinterpret_cast<const i32x4_t*>(x[i] + at + h * 16);
      }
    }
    sw[s] = *reinterpret_cast<const uint16_t*>(ws + as);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if constexpr (RAW) {  // 8 values at a time, k being a multiple of 8; past its end the row's first ones
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int k = c * 256 + q * 64 + p * 8;
          raw[s][i][p] = *reinterpret_cast<const typename Loose8<T>::V*>(reinterpret_cast<const T*>(x[i]) + (c < chunks && k < K ? k : 0));
        }
      } else {
        sx[s][i] = *reinterpret_cast<const uint16_t*>(xs[i] + as);
      }
    }
  };
  auto use = [&](int c, int s) {
    if (c >= chunks) return;
    if constexpr (RAW) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (c == chunks - 1) {
#pragma unroll
          for (int p = 0; p < 8; ++p)
            if (c * 256 + q * 64 + p * 8 >= K) raw[s][i][p] = V8{};
        }
        int first, second;
        fx[s][i][0] = quantise_block(raw[s][i], &first);
        fx[s][i][1] = quantise_block(raw[s][i] + 4, &second);
        sx[s][i] = first | second << 8;
      }
    }
    if (odd && c == chunks - 1 && q >= 2) {  // zeros, whatever scales
      fw[s][0] = fw[s][1] = i32x4_t{0, 0, 0, 0};
      sw[s] = 0;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fx[s][i][0] = fx[s][i][1] = i32x4_t{0, 0, 0, 0};
        sx[s][i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      acc[i] = mfma4<0>(fw[s][0], fx[s][i][0], acc[i], sw[s], sx[s][i]);
      acc[i] = mfma4<1>(fw[s][1], fx[s][i][1], acc[i], sw[s], sx[s][i]);
    }
  };
#pragma unroll
  for (int s = 0; s < U; ++s) load(wave + s * waves, s);
  const int64_t nb = (int64_t)g * (GLU ? 2 * e.N : e.N);
  Extra<4> extra;
  if (wave < MT && m0 + wave * 16 + r < m1 && n0 + 4 * q < e.N && (!GLU || q < 2))
    mm_fetch<T, 4, GLU>(e, m0 + wave * 16 + r, n0 + 4 * q, nb, &extra);
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
    for (int k = 0; k < 4; ++k) {
      z[k] = sum[k];
      if (GLU) u[k] = __shfl_down(z[k], 32);
    }
    if (m < m1 && n < e.N && (!GLU || q < 2)) {
      if (i != wave) mm_fetch<T, 4, GLU>(e, m, n, nb, &extra);
      mm_apply<T, 4, GLU>(e, m, n, 0, z, u, extra);
    }
  }
}

}  // namespace

int64_t mx4_units(int64_t k) { return ceil_div(k, 128); }

namespace {

// calls f(rows, grid, flat) over parts of the rows that a grid and 32 bits hold; ldv: of the 16-bit or fp32 side
template <typename F>
void over_rows(const Mx4Rows& a, int64_t ldv, int64_t bytes, F f) {
  const bool flat = a.k % 128 == 0 && (a.rows == 1 || (ldv == a.k && a.ldc == a.units * 64 && a.lds == a.units * 4));
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 27) / a.units);
  for (int64_t r = 0; r < a.rows; r += most) {
    Mx4Rows p = a;
    p.row0 = r, p.rows = std::min(most, a.rows - r);
    if (a.x) p.x = static_cast<const char*>(a.x) + r * a.ldx * bytes;
    if (a.y) p.y = static_cast<char*>(a.y) + r * a.ldy * bytes;
    p.codes = a.codes + r * a.ldc, p.scales = a.scales + r * a.lds;
    const dim3 g((unsigned)ceil_div(p.rows * a.units * 16, 256 * kPieces));
    flat ? f(p, g, std::true_type{}) : f(p, g, std::false_type{});
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
    over_rows(a, a.ldx, sizeof(T), [&](const Mx4Rows& p, dim3 g, auto flat) {
      hipLaunchKernelGGL((k_mx4_quantize<T, decltype(flat)::value>), g, dim3(256), 0, s, p);
    });
  });
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4Rows& a, hipStream_t s) {
  with_row_type(a.dtype, [&](auto t) {
    typedef decltype(t) T;
    over_rows(a, a.ldy, sizeof(T), [&](const Mx4Rows& p, dim3 g, auto flat) {
      hipLaunchKernelGGL((k_mx4_dequantize<T, decltype(flat)::value>), g, dim3(256), 0, s, p);
    });
  });
  return hipGetLastError();
}

namespace {

// ---- which kernel ----------------------------------------------------------------------------------------

typedef MxCfg<256, 256, 2, 4, 2, true> MxBig;
typedef MxCfg<128, 128, 2, 2, 2, false> MxMid;
typedef MxCfg<64, 128, 1, 4, 3, false> MxLow;
typedef MxCfg<16, 128, 1, 4, 4, false> MxThin;

int64_t mx4_rows(const MmArgs& e, int64_t BM) { return e.mode == MM_ROW_GROUPS ? group_tiles(e.M, e.groups, BM) : ceil_div(e.M, BM); }

// An estimate of each kernel's time in us, with constants fitted to what they take forced everywhere (warm, 256 CUs).
// Streamed, 16, 32 or 64 rows at a time: a launch and the way to memory, and W once per row tile from the caches.  4096 ->
// 4096, 16 / 32 / 64 rows at a time and 64 x 128 tiles: 1 row 5.6, 5.8, 6.4, 11; 16 rows 6.6, 6.9, 7.4, 13; 32 rows 9.3, 8.0,
// 8.4, 13; 64 rows -, 12.1, 10.8, 13.4; 128 rows -, 20, -, 13.5.  2563 -> 520, 256 rows -, 7.4, 6.3, 10.3; 512 rows -, 9.3, 8.9,
// 10.3; 1024 rows -, -, 11.5, 10.5.  A k split over workgroups and joined never won (4096 -> 4096, 64 rows, 4 parts 12.3).
// Tiles: rounds of workgroups (`occ` on a CU, slower each when they share it) of so many steps and a start and end.  64 x 128,
// 128 x 128 and 256 x 256: 4096 -> 4096, 1024 rows 19.4, 21.3, 36; 2048 rows 35, 30, 38; 4096 rows 66, 56, 43; 256 experts of 16,
// 48, 64, 96 and 128 rows, 4096 -> 2 x 2048: 388, 486, 669; 457, 513, 683; 539, 526, 690; 647, 600, 709; 776, 740, 729.
// Groups of up to 8 rows stream W in 16 x 128 tiles, four steps of it in LDS: 512 groups, 2560 -> 2 x 640, a row each 134 and
// 138 (64 x 128); 4 rows 155 and 160; 16 rows 203 and 177.
// Of groups the host knows M and their number alone: every row counts as routed and every group as an average one.  The tiles' part
// has no term for W's bytes, so it tells tiles apart and not how long they take where W bounds them: for 64 rows a group it has 286 and
// 456 us for the 539 and 526 above, and takes the former.
int plan_mx4(const Mx4Args& a, double* us = nullptr) {
  const MmArgs& e = a.e;
  const bool grouped = e.mode == MM_ROW_GROUPS;
  const int64_t n = e.act == EFF_ACT_SWIGLU ? 2 * e.N : e.N, groups = grouped ? std::min<int64_t>(e.groups, std::max<int64_t>(1, e.M)) : 1;
  const int64_t rows = e.M / groups, steps = ceil_div(a.units, 2);
  int best = MX_FEW4;  // any size
  double least = 0;
  auto offer = [&](int kind, double us) {
    if (least == 0 || us < least) least = us, best = kind;
  };
  const double mb = (double)n * a.units * 68e-6;  // W of a group, as it lies in memory
  const struct { int kind; int64_t rows; double us; } few[] = {{MX_FEW1, 16, 0.40}, {MX_FEW2, 32, 0.56}, {MX_FEW4, 64, 0.88}};
  for (const auto& f : few) offer(f.kind, 3.0 + f.us * mb * groups * ceil_div(std::max<int64_t>(1, rows), f.rows));
  // a tile's lanes hold unsigned 32-bit byte offsets from its first row
  const int64_t far = std::max(std::max(a.ldx, a.ldw), std::max(a.ldxs, a.ldws));
  const struct { int kind; int64_t bm, bn; int occ; double alone, step, fixed; } tiles[] = {
      {MX_BIG, MxBig::BM, MxBig::BN, 1, 1.65, 1.65, 12}, {MX_MID, MxMid::BM, MxMid::BN, 2, 1.05, 1.5, 4.5},
      {MX_LOW, MxLow::BM, MxLow::BN, 2, 0.62, 0.9, 3.5}, {MX_THIN, MxThin::BM, MxThin::BN, 2, 0.45, 0.7, 3.3}};
  for (const auto& t : tiles) {
    if (far > 0xffffffffll / std::max(t.bm, t.bn) || (t.kind == MX_THIN && (!grouped || rows > 8))) continue;
    const double rt = grouped ? std::max<double>((double)ceil_div(rows, t.bm) * groups, e.M / (double)t.bm) : (double)ceil_div(e.M, t.bm);
    const double count = rt * ceil_div(n, t.bn), full = std::floor(count / (256.0 * t.occ)), rest = count - full * 256 * t.occ;
    offer(t.kind, full * (t.step * steps + t.fixed) + (rest > 0 ? (rest <= 256 ? t.alone : t.step) * steps + t.fixed : 0));
  }
  if (us) *us = least;
  return best;
}

template <typename T, class C, bool GLU>
hipError_t launch_mx4_tile(const Mx4Args& a, hipStream_t s) {
  const int64_t tiles = ceil_div(a.e.N, GLU ? C::BN / 2 : C::BN) * mx4_rows(a.e, C::BM);
  constexpr int lds = (C::S * 128 + scale_buffers(C::S) * 16) * (C::BM + C::BN);
  auto* fn = &k_mx4_tile<T, C, GLU>;
  static std::atomic<uint64_t> done{0};
  const hipError_t set = allow_lds(reinterpret_cast<const void*>(fn), lds, &done);
  if (set != hipSuccess) return set;
  Mx4Args p = a;
  p.tiles = (int)tiles;
  // one workgroup a CU that goes on to the next tile, where the sums go out of registers
  const int64_t grid = C::AHEAD && a.e.simple && a.e.mode != MM_ROW_GROUPS ? std::min<int64_t>(tiles, 256) : tiles;
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(C::TH), lds, s, p);
  return hipGetLastError();
}

template <typename T, int MT, bool GLU, bool RAW>
hipError_t launch_mx4_few(const Mx4Args& a, hipStream_t s) {
  const int64_t slices = ceil_div(a.e.N, GLU ? 8 : 16), jobs = slices * mx4_rows(a.e, 16 * MT);
  // waves per workgroup: up to 32 per CU over the launch, each with at least two chunks of k, their sums within 64 KiB of LDS
  int waves = 16;
  while (waves > 1 && (jobs * waves > 8192 || waves * 4 > a.units + 3)) waves /= 2;
  hipLaunchKernelGGL((k_mx4_few<T, MT, GLU, RAW>), dim3((unsigned)jobs), dim3(64 * waves), waves * MT * 1024, s, a, (int)slices);
  return hipGetLastError();
}

template <typename T, bool GLU>
hipError_t launch_mx4_kind(const Mx4Args& a, int kind, hipStream_t s) {
  switch (kind) {
    case MX_FEW1: return a.xs ? launch_mx4_few<T, 1, GLU, false>(a, s) : launch_mx4_few<T, 1, GLU, true>(a, s);
    case MX_FEW2: return launch_mx4_few<T, 2, GLU, false>(a, s);
    case MX_FEW4: return launch_mx4_few<T, 4, GLU, false>(a, s);
    case MX_BIG: return launch_mx4_tile<T, MxBig, GLU>(a, s);
    case MX_MID: return launch_mx4_tile<T, MxMid, GLU>(a, s);
    case MX_LOW: return launch_mx4_tile<T, MxLow, GLU>(a, s);
    default: return launch_mx4_tile<T, MxThin, GLU>(a, s);
  }
}

}  // namespace

int mx4_choice(const Mx4Args& a) { return plan_mx4(a); }

// Quantising in every workgroup of 16 rows and 16 W rows against once, in a launch of its own, and the kernel planned then.  us of
// both in a row (and of the calls, bound by the host beyond): 256 x 1024, 256 rows 4.8, 7.8 (7.4, 11.2); 256 x 4096, 256 rows 8.8, 12.9;
// 2 x 640 x 2560, 48 rows 7.0, 8.8, 128 rows 13.6, 9.4; 1024 x 2048, 64 rows 5.9, 9.0, 256 rows 13.3, 9.4; 2048 x 4096, 32 rows
// 8.5, 9.6, 64 rows 13.5, 12.3; 4096 x 4096, 16 rows 8.9, 8.3 (8.8, 11.9), 32 rows 14.1, 9.6.  Fitted to up to 1024 rows.
bool mx4_takes_raw(const Mx4Args& a) {
  const MmArgs& e = a.e;
  double coded;
  const int kind = plan_mx4(a, &coded);
  const int64_t jobs = ceil_div(e.N, e.act == EFF_ACT_SWIGLU ? 8 : 16) * mx4_rows(e, 16);
  if (e.K % 8 || e.M > 1024 || !fits(jobs, 1024)) return false;
  const double raw = 3.5 + (0.2 + 1.2e-3 * (double)e.K) * (double)ceil_div(jobs, 256);
  // the second launch, a long k's way through few workgroups, x read and its codes written
  const double first = 3.5 + 5e-4 * (double)e.K + 5e-7 * (double)e.M * (double)e.K;
  return raw <= coded + first || (kind == MX_FEW1 && e.M <= 16);
}

// whether the launch holds the problem (a grid's threads stay below 2^32)
bool mx4_matmul_fits(const Mx4Args& a) {
  const int64_t nw = a.e.act == EFF_ACT_SWIGLU ? 2 * a.e.N : a.e.N;
  const int kind = plan_mx4(a);
  if (kind <= MX_FEW4) return fits(ceil_div(nw, 16) * mx4_rows(a.e, kind == MX_FEW1 ? 16 : kind == MX_FEW2 ? 32 : 64), 1024);
  return fits(ceil_div(nw, 128) * mx4_rows(a.e, kind == MX_THIN ? 16 : 64), 512);
}

hipError_t launch_mx4_matmul(const Mx4Args& in, hipStream_t s) {
  Mx4Args a = in;
  MmArgs& e = a.e;
  e.vec = aligned16({e.y, e.bias, e.residual, e.pre}, {e.N, e.ldy, e.residual ? e.ldr : 0, e.pre ? e.ldp : 0}, 2);
  e.stream = e.M * e.N * (e.y_f32 ? 4 : 2) > (int64_t)256 << 20;  // past the caches, as launch_matmul
  e.simple = e.vec && !e.bias && !e.pre && !e.y_f32 && (e.act == EFF_ACT_NONE || e.act == EFF_ACT_SWIGLU);
  const int kind = a.xs ? plan_mx4(a) : MX_FEW1;  // the other kernels take no 16-bit x
  const bool glu = e.act == EFF_ACT_SWIGLU;
  if (e.dtype == EFF_DT_BF16) return glu ? launch_mx4_kind<bf16_t, true>(a, kind, s) : launch_mx4_kind<bf16_t, false>(a, kind, s);
  return glu ? launch_mx4_kind<f16_t, true>(a, kind, s) : launch_mx4_kind<f16_t, false>(a, kind, s);
}

}  // namespace eff
