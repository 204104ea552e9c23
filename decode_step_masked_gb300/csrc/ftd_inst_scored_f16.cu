// ftd_inst_scored_f16.cu -- CUDA-core decode kernels that keep their scores, f16 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f16_scored(int D, int G) { return select_kernel<__half, kScored>(D, G); }
}  // namespace ftd
