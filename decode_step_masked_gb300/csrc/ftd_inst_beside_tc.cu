// ftd_inst_beside_tc.cu -- tensor-core decode kernels beside a shared prefix.
#include "ftd_decode_wide_tc.cuh"

namespace ftd {
template <typename CT, bool MQ>
static TcKernelInfo pick(int D, int G) {
    if (D == 64) return G == 16 ? tc_kernel_info<CT, 16, MQ, kBeside, 64>() : tc_kernel_info<CT, 8, MQ, kBeside, 64>();
    if (G == 64) return wide_kernel_info<CT, 64, MQ, kBeside>();
    if (G == 32) return wide_kernel_info<CT, 32, MQ, kBeside>();
    return G == 16 ? tc_kernel_info<CT, 16, MQ, kBeside>() : tc_kernel_info<CT, 8, MQ, kBeside>();
}

TcKernelInfo select_tc_beside(bool bf16, int D, int G, bool multi_token) {
    if (bf16) return multi_token ? pick<__nv_bfloat16, true>(D, G) : pick<__nv_bfloat16, false>(D, G);
    return multi_token ? pick<__half, true>(D, G) : pick<__half, false>(D, G);
}

TcKernelInfo select_tc_i8_beside(int D, bool multi_token) {
    if (D == 64) return multi_token ? tc_kernel_info<int8_t, 8, true, kBeside, 64>() : tc_kernel_info<int8_t, 8, false, kBeside, 64>();
    return multi_token ? tc_kernel_info<int8_t, 8, true, kBeside>() : tc_kernel_info<int8_t, 8, false, kBeside>();
}
}  // namespace ftd
