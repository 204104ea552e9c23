// ftd_inst_scored_bf16.cu -- CUDA-core decode kernels that keep their scores, bf16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_bf16_scored(int D, int G) { return select_kernel<__nv_bfloat16, kScored>(D, G); }
}  // namespace ftd
