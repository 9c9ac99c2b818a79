// C entry points of the operators that need no engine: products with their epilogue and gradients, tokens
// sorted by expert and back, layer norm, the router's losses, 4-bit rows and their products.  Argument checks, workspace
// layout and launches; the kernels are in k_matmul.hip, k_tokens.hip, k_norm.hip, k_balance.hip and k_mx4.hip.
#include <algorithm>
#include <mutex>

#include "eff_internal.h"

using namespace eff;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int kMaxDevices = 64;

int bad(const char* fn, const char* why) { return fail(EFF_EINVAL, std::string(fn) + ": " + why); }

// kernel attributes, once per device
int setup(const char* fn) {
  static std::once_flag once[kMaxDevices];
  static hipError_t result[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return fail(EFF_EHIP, std::string(fn) + ": no HIP device");
  std::call_once(once[dev], [&] { result[dev] = tokens_setup(); });
  if (result[dev] != hipSuccess) return fail(EFF_EHIP, std::string(fn) + ": " + hipGetErrorString(result[dev]));
  return EFF_OK;
}

int launched(const char* fn, hipError_t err) {
  return err == hipSuccess ? EFF_OK : fail(EFF_EHIP, std::string(fn) + ": " + hipGetErrorString(err));
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// nullptr if the description is sound, else what is wrong with it
const char* check_desc(const eff_matmul_desc* d) {
  if (!d) return "the description is NULL";
  if (d->dtype != EFF_DT_BF16 && d->dtype != EFF_DT_F16) return "dtype must be EFF_DT_BF16 or EFF_DT_F16";
  if (d->out_dtype != d->dtype && d->out_dtype != EFF_DT_F32) return "out_dtype must be dtype or EFF_DT_F32";
  if (d->act < EFF_ACT_NONE || d->act > EFF_ACT_SWIGLU) return "unknown activation";
  if (d->groups < 0 || d->groups > kMaxExperts) return "groups must be in [0, 4096]";
  if (d->m < 0 || d->m >= kMaxDim || d->n < 1 || d->k < 1 || d->k >= kMaxDim) return "m >= 0, n >= 1, k >= 1, each below 2^31";
  const int64_t nw = d->act == EFF_ACT_SWIGLU ? 2 * d->n : d->n;
  if (nw >= kMaxDim) return "W's rows must be below 2^31";
  return nullptr;
}

int64_t w_rows(const eff_matmul_desc* d) { return d->act == EFF_ACT_SWIGLU ? 2 * d->n : d->n; }
bool inputs_ld_bad(int64_t ld) { return ld < 0; }

// The products of a description: the forward one, and the two of the backward pass (pointers unset).
MmArgs forward_args(const eff_matmul_desc* d) {
  MmArgs a = {};
  a.dtype = d->dtype, a.y_f32 = d->out_dtype == EFF_DT_F32, a.act = d->act, a.groups = d->groups;
  a.mode = d->groups ? MM_ROW_GROUPS : MM_DENSE;
  a.xk = 1, a.sxm = d->ld_x, a.sxk = 1;
  a.wk = 1, a.swn = d->ld_w, a.swk = 1, a.swg = d->groups ? d->stride_w : 0;
  a.M = d->m, a.N = d->n, a.K = d->k;
  a.ldr = d->ld_residual, a.ldy = d->ld_y, a.ldp = d->ld_pre;
  return a;
}
// The backward pass materialises dz unless it is dy itself, in rows that can be read as 16-byte vectors.
int64_t dz_ld(const eff_matmul_desc* d) { return (w_rows(d) + 7) / 8 * 8; }
bool needs_dz(const eff_matmul_desc* d) {
  return d->act != EFF_ACT_NONE || d->out_dtype != d->dtype || d->n % 8 || d->ld_y % 8;
}
// In fp16 dz is scaled into its range where it is rounded, by rows for dx and by columns for dw: a copy for each, and the
// largest magnitude of every row and of every column of a group.
bool scales_dz(const eff_matmul_desc* d) { return d->dtype == EFF_DT_F16 && (d->act != EFF_ACT_NONE || d->out_dtype != d->dtype); }
int64_t dz_bytes(const eff_matmul_desc* d) { return needs_dz(d) ? align256(d->m * dz_ld(d) * 2) : 0; }  // of one copy
int64_t dz_copies(const eff_matmul_desc* d) { return scales_dz(d) ? 2 : 1; }
int64_t max_bytes(const eff_matmul_desc* d) { return scales_dz(d) ? align256((d->m + std::max(1, d->groups) * w_rows(d)) * 4) : 0; }
int64_t part_bytes(const eff_matmul_desc* d) { return align256(matmul_dz_tiles(d->m, d->n, d->groups) * w_rows(d) * 4); }
// dx[m,k] = sum over W's rows n of dz[m,n] w[n,k]
MmArgs dx_args(const eff_matmul_desc* d) {
  MmArgs a = {};
  a.dtype = d->dtype, a.groups = d->groups;
  a.mode = d->groups ? MM_ROW_GROUPS : MM_DENSE;
  a.xk = 1, a.sxm = needs_dz(d) ? dz_ld(d) : d->ld_y, a.sxk = 1, a.x_padded = needs_dz(d);
  a.swn = 1, a.swk = d->ld_w, a.swg = d->groups ? d->stride_w : 0;
  a.M = d->m, a.N = d->k, a.K = w_rows(d);
  a.ldy = d->ld_dx;
  return a;
}
// dw[n,k] = sum over rows m of dz[m,n] x[m,k]
MmArgs dw_args(const eff_matmul_desc* d) {
  MmArgs a = {};
  a.dtype = d->dtype, a.groups = d->groups;
  a.mode = d->groups ? MM_K_GROUPS : MM_DENSE;
  a.sxm = 1, a.sxk = needs_dz(d) ? dz_ld(d) : d->ld_y, a.x_padded = needs_dz(d);
  a.swn = 1, a.swk = d->ld_x;
  a.M = w_rows(d), a.N = d->k, a.K = d->m;
  a.ldy = d->ld_dw, a.syg = d->groups ? d->stride_dw : 0;
  return a;
}

int check_ws(const char* fn, int64_t need, const void* ws, size_t bytes) {
  if (need <= 0) return EFF_OK;
  if (!ws || (int64_t)bytes < need) return fail(EFF_EINVAL, std::string(fn) + ": needs " + std::to_string(need) + " bytes of workspace");
  if ((uintptr_t)ws % 256) return bad(fn, "the workspace must be 256-byte aligned");
  return EFF_OK;
}

const char* check_rows(int dtype, int64_t T, int K, int64_t H, int64_t rows) {
  if (dtype < EFF_DT_BF16 || dtype > EFF_DT_F32) return "unknown dtype";
  if (T < 0 || K < 1 || K > kMaxTopK || T * K >= kMaxDim || T >= kMaxDim) return "T >= 0, 1 <= K <= 32, T*K below 2^31";
  if (H < 1 || H >= kMaxDim || rows < 0 || rows >= kMaxDim) return "H >= 1, rows >= 0, each below 2^31";
  return nullptr;
}

const char* check_norm(int dtype, int w_dtype, int64_t T, int64_t H) {
  if (dtype < EFF_DT_BF16 || dtype > EFF_DT_F32) return "unknown dtype";
  if (w_dtype != dtype && w_dtype != EFF_DT_F32) return "w_dtype must be dtype or EFF_DT_F32";
  if (T < 0 || T >= kMaxDim || H < 1 || H >= kMaxDim) return "T >= 0, H >= 1, each below 2^31";
  return nullptr;
}

const char* check_balance(int dtype, int64_t T, int K, int num_experts) {
  if (dtype < EFF_DT_BF16 || dtype > EFF_DT_F32) return "unknown dtype";
  if (num_experts < 1 || num_experts > kMaxExperts) return "num_experts must be in [1, 4096]";
  if (T < 0 || K < 1 || K > kMaxTopK || T >= kMaxDim || T * K >= kMaxDim) return "T >= 0, 1 <= K <= 32, T*K below 2^31";
  return nullptr;
}

// rows of codes and scales
const char* check_mx4(int dtype, int64_t rows, int64_t k, const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales) {
  if (dtype < EFF_DT_BF16 || dtype > EFF_DT_F32) return "unknown dtype";
  if (rows < 0 || rows >= kMaxDim || k < 1 || k >= kMaxDim) return "rows >= 0, k >= 1, each below 2^31";
  if ((uintptr_t)codes % 16 || (uintptr_t)scales % 4 || (rows > 1 && (ld_codes % 16 || ld_scales % 4 || ld_codes < 0 || ld_scales < 0)))
    return "rows of codes must begin at multiples of 16 bytes, of scales at multiples of 4";
  return nullptr;
}

const char* check_mx4_desc(const eff_mx4_desc* d) {
  if (!d) return "the description is NULL";
  if (d->dtype != EFF_DT_BF16 && d->dtype != EFF_DT_F16) return "dtype must be EFF_DT_BF16 or EFF_DT_F16";
  if (d->x_dtype != EFF_DT_MX4 && d->x_dtype != d->dtype) return "x_dtype must be EFF_DT_MX4 or dtype";
  if (d->out_dtype != d->dtype && d->out_dtype != EFF_DT_F32) return "out_dtype must be dtype or EFF_DT_F32";
  if (d->act < EFF_ACT_NONE || d->act > EFF_ACT_SWIGLU) return "unknown activation";
  if (d->groups < 0 || d->groups > kMaxExperts) return "groups must be in [0, 4096]";
  if (d->reserved) return "reserved must be 0";
  if (d->m < 0 || d->m >= kMaxDim || d->n < 1 || d->n >= kMaxDim || d->k < 1 || d->k >= kMaxDim) return "m >= 0, n >= 1, k >= 1, each below 2^31";
  if (d->act == EFF_ACT_SWIGLU && 2 * d->n >= kMaxDim) return "W's rows must be below 2^31";
  return nullptr;
}

Mx4Args mx4_args(const eff_mx4_desc* d) {
  Mx4Args a = {};
  MmArgs& e = a.e;
  e.dtype = d->dtype, e.y_f32 = d->out_dtype == EFF_DT_F32, e.act = d->act, e.groups = d->groups;
  e.mode = d->groups ? MM_ROW_GROUPS : MM_DENSE;
  e.M = d->m, e.N = d->n, e.K = d->k;
  e.ldr = d->ld_residual, e.ldy = d->ld_y, e.ldp = d->ld_pre;
  a.units = (int)mx4_units(d->k);
  const bool coded = d->x_dtype == EFF_DT_MX4;
  a.ldx = coded ? d->ld_x : a.units * (int64_t)64, a.ldxs = coded ? d->ld_xs : a.units * (int64_t)4;
  a.ldw = d->ld_w, a.ldws = d->ld_ws;
  a.sw = d->groups ? d->stride_w : 0, a.sws = d->groups ? d->stride_ws : 0;
  return a;
}
// the workspace: x in 4 bits, where it comes in 16 and the kernel does not quantise it itself
int64_t x_code_bytes(const eff_mx4_desc* d) { return align256(d->m * mx4_units(d->k) * 64); }
int64_t x_scale_bytes(const eff_mx4_desc* d) { return align256(d->m * mx4_units(d->k) * 4); }

}  // namespace

MmChoice eff::matmul_choice(const eff_matmul_desc& d, int product) {
  return matmul_choice(product == 0 ? forward_args(&d) : product == 1 ? dx_args(&d) : dw_args(&d));
}

int eff::mx4_choice(const eff_mx4_desc& d) { return mx4_choice(mx4_args(&d)); }

extern "C" {

int64_t eff_matmul_workspace(const eff_matmul_desc* d, int backward) {
  if (const char* why = check_desc(d)) return bad("eff_matmul_workspace", why);
  if (d->m == 0) return 0;
  if (!backward) return align256(matmul_workspace(forward_args(d)));
  return dz_copies(d) * dz_bytes(d) + max_bytes(d) + part_bytes(d) + align256(std::max(matmul_workspace(dx_args(d)), matmul_workspace(dw_args(d))));
}

int eff_matmul(const eff_matmul_desc* d, const void* x, const void* w, const void* bias, const void* residual,
               const int32_t* offsets, void* y, void* pre, void* workspace, size_t workspace_bytes, eff_stream_t stream) {
  const char* fn = "eff_matmul";
  if (const char* why = check_desc(d)) return bad(fn, why);
  if (d->m == 0) return EFF_OK;
  if (!x || !w || !y) return bad(fn, "x, w and y are needed");
  if ((d->groups > 0) != (offsets != nullptr)) return bad(fn, "offsets go with groups");
  const int64_t nw = w_rows(d);
  if (inputs_ld_bad(d->ld_x) || inputs_ld_bad(d->ld_w) || inputs_ld_bad(d->ld_residual) || d->stride_w < 0) return bad(fn, "negative stride");
  if (d->m > 1 && (d->ld_y < d->n || (pre && d->ld_pre < nw))) return bad(fn, "rows of an output overlap");
  if (residual == y && (d->out_dtype != d->dtype || (d->m > 1 && d->ld_residual != d->ld_y)))
    return bad(fn, "y may be the residual only with its type and ld");
  if (int rc = check_ws(fn, eff_matmul_workspace(d, 0), workspace, workspace_bytes)) return rc;
  MmArgs a = forward_args(d);
  if (!matmul_fits(a)) return bad(fn, "too many output tiles for one launch");
  a.x = x, a.w = w, a.offsets = offsets, a.bias = bias, a.residual = residual, a.y = y, a.pre = pre;
  return launched(fn, launch_matmul(a, workspace, (hipStream_t)stream));
}

int eff_matmul_backward(const eff_matmul_desc* d, const void* dy, const void* x, const void* w, const void* pre,
                        const int32_t* offsets, void* dx, void* dw, void* dbias, void* workspace, size_t workspace_bytes,
                        eff_stream_t stream) {
  const char* fn = "eff_matmul_backward";
  if (const char* why = check_desc(d)) return bad(fn, why);
  const bool rows = d->m > 0;
  if ((d->groups > 0) != (offsets != nullptr)) return bad(fn, "offsets go with groups");
  if (rows && (!dy || (dx && !w) || (dw && !x))) return bad(fn, "dy is needed, w for dx, x for dw");
  if (rows && d->act != EFF_ACT_NONE && !pre) return bad(fn, "pre is needed with an activation");
  const int64_t nw = w_rows(d);
  if (inputs_ld_bad(d->ld_x) || inputs_ld_bad(d->ld_w) || inputs_ld_bad(d->ld_y) || inputs_ld_bad(d->ld_pre) || d->stride_w < 0)
    return bad(fn, "negative stride");
  if ((dx && d->m > 1 && d->ld_dx < d->k) || (dw && nw > 1 && d->ld_dw < d->k) ||
      (dw && d->groups > 1 && d->stride_dw < (nw - 1) * std::max(d->ld_dw, d->k) + d->k))
    return bad(fn, "rows of an output overlap");
  if (int rc = check_ws(fn, eff_matmul_workspace(d, 1), workspace, workspace_bytes)) return rc;
  if ((rows && dx && !matmul_fits(dx_args(d))) || (dw && !matmul_fits(dw_args(d))) ||
      ((rows || dbias) && !matmul_dz_fits(d->m, d->n, d->groups)))
    return bad(fn, "too many output tiles for one launch");
  hipStream_t s = (hipStream_t)stream;
  MmGrad g = {};
  g.dtype = d->dtype, g.dy_f32 = d->out_dtype == EFF_DT_F32, g.act = d->act;
  g.M = d->m, g.N = d->n;
  g.dy = dy, g.ldy = d->ld_y, g.pre = pre, g.ldp = d->ld_pre;
  g.offsets = offsets, g.groups = d->groups;
  g.dbias = dbias;
  const void *dz = dy, *dz_w = dy;  // for dx and for dw
  char* ws = static_cast<char*>(workspace);
  if (needs_dz(d) && (dx || dw)) {
    dz = dz_w = g.dz = ws, g.lddz = dz_ld(d);
    if (rows && scales_dz(d)) {
      uint32_t* largest = reinterpret_cast<uint32_t*>(ws + 2 * dz_bytes(d));
      if (dx) g.row_max = largest, largest += d->m;
      else g.dz = nullptr;
      if (dw) g.col_max = largest, dz_w = g.dz_cols = ws + dz_bytes(d);
    }
  }
  if (ws) ws += dz_copies(d) * dz_bytes(d) + max_bytes(d);
  if (dbias) g.part = reinterpret_cast<float*>(ws);
  if (g.dz || g.dz_cols || dbias)
    if (int rc = launched(fn, launch_matmul_dz(g, s))) return rc;
  if (ws) ws += part_bytes(d);
  if (dx && rows) {
    MmArgs a = dx_args(d);
    a.x = dz, a.w = w, a.y = dx, a.offsets = offsets, a.row_max = g.row_max;
    if (int rc = launched(fn, launch_matmul(a, ws, s))) return rc;
  }
  if (dw) {
    MmArgs a = dw_args(d);
    a.x = dz_w, a.w = x, a.y = dw, a.offsets = offsets, a.row_max = g.col_max;
    if (int rc = launched(fn, launch_matmul(a, ws, s))) return rc;
  }
  return EFF_OK;
}

int64_t eff_sort_tokens_workspace(int64_t n, int num_experts) {
  if (n < 0 || n >= kMaxDim || num_experts < 1 || num_experts > kMaxExperts)
    return bad("eff_sort_tokens_workspace", "0 <= n < 2^31, 1 <= num_experts <= 4096");
  return sort_workspace(n, num_experts);
}

int eff_sort_tokens(const int32_t* ids, int64_t n, int num_experts, int32_t* offsets, int32_t* order, int32_t* pos,
                    void* workspace, size_t workspace_bytes, eff_stream_t stream) {
  const char* fn = "eff_sort_tokens";
  const int64_t need = eff_sort_tokens_workspace(n, num_experts);
  if (need < 0) return (int)need;
  if (!offsets || (n > 0 && (!ids || !order || !pos))) return bad(fn, "ids, offsets, order and pos are needed");
  if (int rc = check_ws(fn, need, workspace, workspace_bytes)) return rc;
  if (int rc = setup(fn)) return rc;
  return launched(fn, launch_sort_tokens(ids, n, num_experts, offsets, order, pos, (int32_t*)workspace, (hipStream_t)stream));
}

int eff_dispatch_tokens(int dtype, const void* x, int64_t ld_x, const int32_t* pos, int64_t T, int K, int64_t H, void* xs,
                        int64_t ld_xs, int64_t rows, eff_stream_t stream) {
  const char* fn = "eff_dispatch_tokens";
  if (const char* why = check_rows(dtype, T, K, H, rows)) return bad(fn, why);
  if (T == 0 || rows == 0) return EFF_OK;
  if (!x || !pos || !xs) return bad(fn, "x, pos and xs are needed");
  if (ld_x < 0 || (rows > 1 && ld_xs < H)) return bad(fn, "negative stride, or rows of an output overlap");
  return launched(fn, launch_dispatch_tokens(dtype, x, ld_x, pos, T, K, H, xs, ld_xs, rows, (hipStream_t)stream));
}

int eff_dispatch_tokens_backward(int dtype, const void* dxs, int64_t ld_dxs, int64_t rows, const int32_t* pos, int64_t T, int K,
                                 int64_t H, void* dx, int64_t ld_dx, eff_stream_t stream) {
  const char* fn = "eff_dispatch_tokens_backward";
  if (const char* why = check_rows(dtype, T, K, H, rows)) return bad(fn, why);
  if (T == 0) return EFF_OK;
  if ((!dxs && rows > 0) || !pos || !dx) return bad(fn, "dxs, pos and dx are needed");
  if (ld_dxs < 0 || (T > 1 && ld_dx < H)) return bad(fn, "negative stride, or rows of an output overlap");
  return launched(fn, launch_combine_tokens(dtype, dxs, ld_dxs, rows, pos, nullptr, T, K, H, nullptr, 0, dx, ld_dx, (hipStream_t)stream));
}

int eff_combine_tokens(int dtype, const void* ys, int64_t ld_ys, int64_t rows, const int32_t* pos, const float* w, int64_t T,
                       int K, int64_t H, const void* residual, int64_t ld_residual, void* out, int64_t ld_out,
                       eff_stream_t stream) {
  const char* fn = "eff_combine_tokens";
  if (const char* why = check_rows(dtype, T, K, H, rows)) return bad(fn, why);
  if (T == 0) return EFF_OK;
  if ((!ys && rows > 0) || !pos || !w || !out) return bad(fn, "ys, pos, w and out are needed");
  if (ld_ys < 0 || ld_residual < 0 || (T > 1 && ld_out < H)) return bad(fn, "negative stride, or rows of an output overlap");
  if (residual == out && T > 1 && ld_residual != ld_out) return bad(fn, "out may be the residual only with its ld");
  return launched(fn, launch_combine_tokens(dtype, ys, ld_ys, rows, pos, w, T, K, H, residual, ld_residual, out, ld_out, (hipStream_t)stream));
}

int eff_combine_tokens_backward(int dtype, const void* dout, int64_t ld_dout, const void* ys, int64_t ld_ys, int64_t rows,
                                const int32_t* pos, const float* w, int64_t T, int K, int64_t H, void* dys, int64_t ld_dys,
                                float* dw, eff_stream_t stream) {
  const char* fn = "eff_combine_tokens_backward";
  if (const char* why = check_rows(dtype, T, K, H, rows)) return bad(fn, why);
  if (T == 0) return EFF_OK;
  if (!dout || !pos || !w || (rows > 0 && (!dys || (dw && !ys)))) return bad(fn, "dout, pos, w and dys are needed, ys for dw");
  if (ld_dout < 0 || ld_ys < 0 || (rows > 1 && ld_dys < H)) return bad(fn, "negative stride, or rows of an output overlap");
  return launched(fn, launch_combine_tokens_grad(dtype, dout, ld_dout, ys, ld_ys, rows, pos, w, T, K, H, dys, ld_dys, dw, (hipStream_t)stream));
}

// ---- layer norm ------------------------------------------------------------------------------------------

int eff_layer_norm(int dtype, int w_dtype, const void* x, int64_t ld_x, const void* w, const void* b, float eps, int64_t T,
                   int64_t H, void* y, int64_t ld_y, float* mean, float* rstd, eff_stream_t stream) {
  const char* fn = "eff_layer_norm";
  if (const char* why = check_norm(dtype, w_dtype, T, H)) return bad(fn, why);
  if (!(eps >= 0.f) || eps > 3.4e38f) return bad(fn, "eps must be a number of at least 0");
  if (T == 0) return EFF_OK;
  if (!x || !y) return bad(fn, "x and y are needed");
  if (ld_x < 0 || (T > 1 && ld_y < H)) return bad(fn, "negative stride, or rows of an output overlap");
  NormArgs a = {};
  a.dtype = dtype, a.w_dtype = w_dtype, a.x = x, a.ldx = ld_x, a.w = w, a.b = b, a.eps = eps, a.T = T, a.H = H;
  a.y = y, a.ldy = T > 1 ? ld_y : H, a.mean = mean, a.rstd = rstd;
  return launched(fn, launch_norm(a, (hipStream_t)stream));
}

int64_t eff_layer_norm_backward_workspace(int64_t T, int64_t H) {
  if (const char* why = check_norm(EFF_DT_F32, EFF_DT_F32, T, H)) return bad("eff_layer_norm_backward_workspace", why);
  return align256(norm_parts(T, H) * 2 * H * 4);
}

int eff_layer_norm_backward(int dtype, int w_dtype, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, const void* w,
                            const float* mean, const float* rstd, const void* residual, int64_t ld_residual, int64_t T,
                            int64_t H, void* dx, int64_t ld_dx, void* dw, void* db, void* workspace, size_t workspace_bytes,
                            eff_stream_t stream) {
  const char* fn = "eff_layer_norm_backward";
  if (const char* why = check_norm(dtype, w_dtype, T, H)) return bad(fn, why);
  if (T > 0 && (!dy || !x || !mean || !rstd)) return bad(fn, "dy, x, mean and rstd are needed");
  if (ld_dy < 0 || ld_x < 0 || ld_residual < 0 || (dx && T > 1 && ld_dx < H)) return bad(fn, "negative stride, or rows of an output overlap");
  if (dw || db)
    if (int rc = check_ws(fn, eff_layer_norm_backward_workspace(T, H), workspace, workspace_bytes)) return rc;
  if (!dw && !db && (!dx || T == 0)) return EFF_OK;
  NormGradArgs a = {};
  a.dtype = dtype, a.w_dtype = w_dtype, a.dy = dy, a.lddy = ld_dy, a.x = x, a.ldx = ld_x, a.w = w, a.mean = mean, a.rstd = rstd;
  a.residual = residual, a.ldr = ld_residual, a.T = T, a.H = H, a.dx = dx, a.lddx = T > 1 ? ld_dx : H, a.dw = dw, a.db = db;
  a.part = dw || db ? static_cast<float*>(workspace) : nullptr;
  return launched(fn, launch_norm_grad(a, (hipStream_t)stream));
}

// ---- the router's losses -----------------------------------------------------------------------------------

int64_t eff_balance_loss_workspace(int64_t T, int num_experts) {
  if (const char* why = check_balance(EFF_DT_F32, T, 1, num_experts)) return bad("eff_balance_loss_workspace", why);
  return balance_workspace(T, num_experts);
}

int eff_balance_loss(int dtype, const void* logits, int64_t ld_logits, const int32_t* ids, const uint8_t* mask, int64_t T, int K,
                     int num_experts, int32_t* counts, float* lse, float* losses, void* workspace, size_t workspace_bytes,
                     eff_stream_t stream) {
  const char* fn = "eff_balance_loss";
  if (const char* why = check_balance(dtype, T, K, num_experts)) return bad(fn, why);
  if (!counts || !losses || (T > 0 && (!logits || !ids || !lse))) return bad(fn, "logits, ids, counts, lse and losses are needed");
  if (ld_logits < 0) return bad(fn, "negative stride");
  if (int rc = check_ws(fn, balance_workspace(T, num_experts), workspace, workspace_bytes)) return rc;
  BalanceArgs a = {};
  a.dtype = dtype, a.logits = logits, a.ld = ld_logits, a.ids = ids, a.mask = mask, a.T = T, a.K = K, a.E = num_experts;
  a.counts = counts, a.lse = lse, a.losses = losses;
  return launched(fn, launch_balance(a, workspace, (hipStream_t)stream));
}

int eff_balance_loss_backward(int dtype, const void* logits, int64_t ld_logits, const int32_t* ids, const int32_t* counts,
                              const float* lse, const float* dlosses, const float* w, const float* dw, int64_t T, int K,
                              int num_experts, void* dlogits, int64_t ld_dlogits, eff_stream_t stream) {
  const char* fn = "eff_balance_loss_backward";
  if (const char* why = check_balance(dtype, T, K, num_experts)) return bad(fn, why);
  if (!w != !dw) return bad(fn, "w and dw go together");
  if (T == 0) return EFF_OK;
  if (!logits || !ids || !counts || !lse || !dlogits) return bad(fn, "logits, ids, counts, lse and dlogits are needed");
  if (ld_logits < 0 || (T > 1 && ld_dlogits < num_experts)) return bad(fn, "negative stride, or rows of an output overlap");
  BalanceGradArgs a = {};
  a.dtype = dtype, a.logits = logits, a.ld = ld_logits, a.ids = ids, a.counts = counts, a.lse = lse, a.dlosses = dlosses;
  a.w = w, a.dw = dw, a.T = T, a.K = K, a.E = num_experts, a.dlogits = dlogits, a.ldd = T > 1 ? ld_dlogits : num_experts;
  return launched(fn, launch_balance_grad(a, (hipStream_t)stream));
}

// ---- 4-bit rows and their products -------------------------------------------------------------------------

int64_t eff_mx4_code_bytes(int64_t k) {
  return k < 1 || k >= kMaxDim ? bad("eff_mx4_code_bytes", "k >= 1, below 2^31") : mx4_units(k) * 64;
}
int64_t eff_mx4_scale_bytes(int64_t k) {
  return k < 1 || k >= kMaxDim ? bad("eff_mx4_scale_bytes", "k >= 1, below 2^31") : mx4_units(k) * 4;
}

int eff_mx4_quantize(int dtype, const void* x, int64_t ld_x, int64_t rows, int64_t k, uint8_t* codes, int64_t ld_codes,
                     uint8_t* scales, int64_t ld_scales, eff_stream_t stream) {
  const char* fn = "eff_mx4_quantize";
  if (const char* why = check_mx4(dtype, rows, k, codes, ld_codes, scales, ld_scales)) return bad(fn, why);
  if (rows == 0) return EFF_OK;
  if (!x || !codes || !scales) return bad(fn, "x, codes and scales are needed");
  if (ld_x < 0 || (rows > 1 && (ld_codes < mx4_units(k) * 64 || ld_scales < mx4_units(k) * 4)))
    return bad(fn, "negative stride, or rows of an output overlap");
  Mx4Rows a = {};
  a.dtype = dtype, a.x = x, a.ldx = ld_x, a.rows = rows, a.k = k, a.units = mx4_units(k);
  a.codes = codes, a.ldc = ld_codes, a.scales = scales, a.lds = ld_scales;
  return launched(fn, launch_mx4_quantize(a, (hipStream_t)stream));
}

int eff_mx4_dequantize(int dtype, const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales, int64_t rows,
                       int64_t k, void* y, int64_t ld_y, eff_stream_t stream) {
  const char* fn = "eff_mx4_dequantize";
  if (const char* why = check_mx4(dtype, rows, k, codes, ld_codes, scales, ld_scales)) return bad(fn, why);
  if (rows == 0) return EFF_OK;
  if (!y || !codes || !scales) return bad(fn, "codes, scales and y are needed");
  if (rows > 1 && ld_y < k) return bad(fn, "rows of an output overlap");
  Mx4Rows a = {};
  a.dtype = dtype, a.y = y, a.ldy = rows > 1 ? ld_y : k, a.rows = rows, a.k = k, a.units = mx4_units(k);
  a.codes = const_cast<uint8_t*>(codes), a.ldc = ld_codes, a.scales = const_cast<uint8_t*>(scales), a.lds = ld_scales;
  return launched(fn, launch_mx4_dequantize(a, (hipStream_t)stream));
}

int64_t eff_mx4_matmul_workspace(const eff_mx4_desc* d) {
  if (const char* why = check_mx4_desc(d)) return bad("eff_mx4_matmul_workspace", why);
  if (d->m == 0 || d->x_dtype == EFF_DT_MX4 || mx4_takes_raw(mx4_args(d))) return 0;
  return x_code_bytes(d) + x_scale_bytes(d);
}

int eff_mx4_matmul(const eff_mx4_desc* d, const void* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, const void* bias,
                   const void* residual, const int32_t* offsets, void* y, void* pre, void* workspace, size_t workspace_bytes,
                   eff_stream_t stream) {
  const char* fn = "eff_mx4_matmul";
  if (const char* why = check_mx4_desc(d)) return bad(fn, why);
  if (d->m == 0) return EFF_OK;
  const bool coded = d->x_dtype == EFF_DT_MX4;
  if (!x || !w || !ws || !y || coded != (xs != nullptr)) return bad(fn, "x, w, ws and y are needed, xs with EFF_DT_MX4 alone");
  if ((d->groups > 0) != (offsets != nullptr)) return bad(fn, "offsets go with groups");
  const int64_t nw = d->act == EFF_ACT_SWIGLU ? 2 * d->n : d->n;
  if (d->ld_x < 0 || d->ld_xs < 0 || d->ld_w < 0 || d->ld_ws < 0 || d->ld_residual < 0 || d->stride_w < 0 || d->stride_ws < 0)
    return bad(fn, "negative stride");
  if (const char* why = check_mx4(EFF_DT_F32, nw, d->k, w, d->ld_w, ws, d->ld_ws)) return bad(fn, why);
  if (d->groups > 1 && (d->stride_w % 16 || d->stride_ws % 4)) return bad(fn, "groups of codes must begin at multiples of 16 bytes, of scales 4");
  if (coded)
    if (const char* why = check_mx4(EFF_DT_F32, d->m, d->k, static_cast<const uint8_t*>(x), d->ld_x, xs, d->ld_xs)) return bad(fn, why);
  if (d->m > 1 && (d->ld_y < d->n || (pre && d->ld_pre < nw))) return bad(fn, "rows of an output overlap");
  if (residual == y && (d->out_dtype != d->dtype || (d->m > 1 && d->ld_residual != d->ld_y)))
    return bad(fn, "y may be the residual only with its type and ld");
  if (int rc = check_ws(fn, eff_mx4_matmul_workspace(d), workspace, workspace_bytes)) return rc;
  Mx4Args a = mx4_args(d);
  if (!mx4_matmul_fits(a)) return bad(fn, "too many output tiles for one launch");
  a.e.offsets = offsets, a.e.bias = bias, a.e.residual = residual, a.e.y = y, a.e.pre = pre;
  a.w = w, a.ws = ws, a.x = static_cast<const uint8_t*>(x), a.xs = xs;
  uint8_t* tmp = static_cast<uint8_t*>(workspace);
  if (!coded && mx4_takes_raw(a)) {
    a.ldx = d->ld_x, a.xs = nullptr;
  } else if (!coded) {
    Mx4Rows q = {};
    q.dtype = d->dtype, q.x = x, q.ldx = d->ld_x, q.rows = d->m, q.k = d->k, q.units = a.units, q.offsets = offsets, q.groups = d->groups;
    q.codes = tmp, q.ldc = a.ldx, q.scales = tmp + x_code_bytes(d), q.lds = a.ldxs;
    if (int rc = launched(fn, launch_mx4_quantize(q, (hipStream_t)stream))) return rc;
    a.x = q.codes, a.xs = q.scales;
  }
  return launched(fn, launch_mx4_matmul(a, (hipStream_t)stream));
}

}  // extern "C"
