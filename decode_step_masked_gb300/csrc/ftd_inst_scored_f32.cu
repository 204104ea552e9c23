// ftd_inst_scored_f32.cu -- CUDA-core decode kernels that keep their scores, f32 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_f32_scored(int D, int G) { return select_kernel<float, kScored>(D, G); }
}  // namespace ftd
