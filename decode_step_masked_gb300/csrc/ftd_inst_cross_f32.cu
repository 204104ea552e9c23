// ftd_inst_cross_f32.cu -- CUDA-core cross-attention kernels, f32 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f32_cross(int D, int G) { return select_kernel<float, kCross>(D, G); }
}  // namespace ftd
