// ftd_prefix_tc_i8.cu -- the tensor-core kernel over a shared prefix for INT8 caches.
#include "ftd_prefix_tc_kernel.cuh"

namespace ftd {

namespace {
template <int D>
PrefixKernel pick(bool q_bf16, int pairs) {
    return pairs == 2   ? ptc::kernel_of<__nv_bfloat16, D, true, true, true>()
           : pairs == 1 ? ptc::kernel_of<__nv_bfloat16, D, true, false, true>()
           : q_bf16     ? ptc::kernel_of<__nv_bfloat16, D, false, false, true>()
                        : ptc::kernel_of<__half, D, false, false, true>();
}
}  // namespace

PrefixKernel select_prefix_tc_i8(bool q_bf16, int D, int pairs) { return D == 64 ? pick<64>(q_bf16, pairs) : pick<128>(q_bf16, pairs); }

}  // namespace ftd
