// ftd_prefix_tc.cu -- the tensor-core kernel over a shared prefix for fp16 and bf16 caches.
#include "ftd_prefix_tc_kernel.cuh"

namespace ftd {

namespace {
template <typename CT, int D>
PrefixKernel pick(int pairs) {
    return pairs == 2   ? ptc::kernel_of<CT, D, true, true, false>()
           : pairs == 1 ? ptc::kernel_of<CT, D, true, false, false>()
                        : ptc::kernel_of<CT, D, false, false, false>();
}
}  // namespace

PrefixKernel select_prefix_tc(bool bf16, int D, int pairs) {
    if (bf16) return D == 64 ? pick<__nv_bfloat16, 64>(pairs) : pick<__nv_bfloat16, 128>(pairs);
    return D == 64 ? pick<__half, 64>(pairs) : pick<__half, 128>(pairs);
}

}  // namespace ftd
