// ftd_inst_scored_i8.cu -- CUDA-core decode kernels that keep their scores, i8 caches (one
// translation unit per cache type and mode so the build compiles them in parallel).
#include "ftd_decode_splitk.cuh"

namespace ftd {
KernelInfo select_i8_scored(int D, int G) { return select_kernel<int8_t, kScored>(D, G); }
}  // namespace ftd
