// ftd_prefix_tc.cuh -- selection of the tensor-core kernel over a shared prefix (ftd_prefix_tc_kernel.cuh).
#pragma once

#include "ftd_prefix.cuh"

namespace ftd {
// Cache type, head dimension, and whether q is kept as a pair of 16-bit numbers.
PrefixKernel select_prefix_tc(bool bf16, int D, bool pair_q);
// INT8 caches: q's own type where it is no pair (bf16, else fp16); a pair is of bf16 numbers.
PrefixKernel select_prefix_tc_i8(bool q_bf16, int D, bool pair_q);
}  // namespace ftd
