// ftd_inst_beside_f32.cu -- CUDA-core decode kernels beside a shared prefix, f32 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f32_beside(int D, int G) { return select_kernel<float, kBeside>(D, G); }
}  // namespace ftd
