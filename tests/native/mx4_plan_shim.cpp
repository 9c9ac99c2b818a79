// Test shim: which kernel the library takes for a product of 4-bit operands, asked of the built library without a GPU.  Compiled
// by tests/test_mx4_plan.py and linked against it.
#include "../../expert_ffn_serving_amd/csrc/eff_internal.h"

extern "C" int shim_mx4_choice(const eff_mx4_desc* d) { return eff::mx4_choice(*d); }
