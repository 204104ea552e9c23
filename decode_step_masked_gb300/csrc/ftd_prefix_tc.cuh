// ftd_prefix_tc.cuh -- selection of the tensor-core kernel over a shared prefix (ftd_prefix_tc.cu).
#pragma once

#include "ftd_prefix.cuh"

namespace ftd {
// Cache type, head dimension, and whether q and the weights are kept as pairs.
PrefixKernel select_prefix_tc(bool bf16, int D, bool pair);
}  // namespace ftd
