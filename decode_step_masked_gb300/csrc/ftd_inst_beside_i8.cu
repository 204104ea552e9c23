// ftd_inst_beside_i8.cu -- CUDA-core decode kernels beside a shared prefix, i8 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_i8_beside(int D, int G) { return select_kernel<int8_t, kBeside>(D, G); }
}  // namespace ftd
