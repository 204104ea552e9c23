// ftd_inst_cross_tc.cu -- tensor-core cross-attention kernels.
#include "ftd_decode_wide_tc.cuh"

namespace ftd {
template <typename CT, bool MQ>
static TcKernelInfo pick(int G) {
    if (G == 64) return wide_kernel_info<CT, 64, MQ, kCross>();
    if (G == 32) return wide_kernel_info<CT, 32, MQ, kCross>();
    return G == 16 ? tc_kernel_info<CT, 16, MQ, kCross>() : tc_kernel_info<CT, 8, MQ, kCross>();
}

TcKernelInfo select_tc_cross(bool bf16, int G, bool multi_token) {
    if (bf16) return multi_token ? pick<__nv_bfloat16, true>(G) : pick<__nv_bfloat16, false>(G);
    return multi_token ? pick<__half, true>(G) : pick<__half, false>(G);
}

TcKernelInfo select_tc_i8_cross(bool multi_token) {
    return multi_token ? tc_kernel_info<int8_t, 8, true, kCross>() : tc_kernel_info<int8_t, 8, false, kCross>();
}
}  // namespace ftd
