// ftd_inst_beside_f16.cu -- CUDA-core decode kernels beside a shared prefix, f16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f16_beside(int D, int G) { return select_kernel<__half, kBeside>(D, G); }
}  // namespace ftd
