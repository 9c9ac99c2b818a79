// Test shim: rows and columns that one launch of layer norm or its gradients takes, asked of the built library without a GPU.  Compiled by
// tests/test_norm_plan.py and linked against it.
#include "../../expert_ffn_serving_amd/csrc/eff_internal.h"

extern "C" int64_t shim_norm_at_once(int threads, int64_t per) { return eff::norm_at_once(threads, per); }
extern "C" int64_t shim_norm_columns_at_once() { return eff::norm_columns_at_once(); }
