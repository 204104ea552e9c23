// ftd_inst_beside_bf16.cu -- CUDA-core decode kernels beside a shared prefix, bf16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_bf16_beside(int D, int G) { return select_kernel<__nv_bfloat16, kBeside>(D, G); }
}  // namespace ftd
