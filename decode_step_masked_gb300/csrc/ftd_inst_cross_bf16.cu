// ftd_inst_cross_bf16.cu -- CUDA-core cross-attention kernels, bf16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_bf16_cross(int D, int G) { return select_kernel<__nv_bfloat16, kCross>(D, G); }
}  // namespace ftd
