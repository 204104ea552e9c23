// ftd_inst_cross_f16.cu -- CUDA-core cross-attention kernels, f16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f16_cross(int D, int G) { return select_kernel<__half, kCross>(D, G); }
}  // namespace ftd
