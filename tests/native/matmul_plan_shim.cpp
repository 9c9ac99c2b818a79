// Test shim: which kernel the library takes for a product, asked of the built library without a GPU.  Compiled by
// tests/test_matmul_plan.py and linked against it.
#include "../../expert_ffn_serving_amd/csrc/eff_internal.h"

// product: 0 forward, 1 dx, 2 dw.  out: kind (KIND_*), parts of k, elements between the rows of both operands.
extern "C" void shim_matmul_choice(const eff_matmul_desc* d, int product, int64_t* out) {
  const eff::MmChoice c = eff::matmul_choice(*d, product);
  out[0] = c.kind, out[1] = c.splits, out[2] = c.ld_x, out[3] = c.ld_w;
}
