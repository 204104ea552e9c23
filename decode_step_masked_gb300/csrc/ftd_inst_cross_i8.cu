// ftd_inst_cross_i8.cu -- CUDA-core cross-attention kernels, i8 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_i8_cross(int D, int G) { return select_kernel<int8_t, kCross>(D, G); }
}  // namespace ftd
