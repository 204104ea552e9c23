// ftd_prefix_tc.cu -- the tensor-core kernel over a shared prefix for fp16 and bf16 caches.
#include "ftd_prefix_tc_kernel.cuh"

namespace ftd {

namespace {
template <typename CT, int D>
PrefixKernel pick(bool pair_q) {
    return pair_q ? ptc::kernel_of<CT, D, true, false>() : ptc::kernel_of<CT, D, false, false>();
}
}  // namespace

PrefixKernel select_prefix_tc(bool bf16, int D, bool pair_q) {
    if (bf16) return D == 64 ? pick<__nv_bfloat16, 64>(pair_q) : pick<__nv_bfloat16, 128>(pair_q);
    return D == 64 ? pick<__half, 64>(pair_q) : pick<__half, 128>(pair_q);
}

}  // namespace ftd
