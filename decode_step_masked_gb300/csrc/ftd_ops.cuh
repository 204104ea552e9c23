// ftd_ops.cuh -- parameters and launchers of the operators around the decode step:
// rotary positions (ftd_rope.cu), the accumulated attention weights (ftd_weights.cu)
// and the eviction by them (ftd_evict.cu).
#pragma once

#include "ftd_common.cuh"

namespace ftd {

// Launch on `stream` with programmatic stream serialisation: when the previous operation
// on the stream is a kernel that allows it, this grid's blocks may be placed while it
// drains; they wait in griddepcontrol.wait (grid_dep_wait) for its completion.
inline cudaError_t launch_pdl(const void* fn, dim3 grid, int threads, int smem, void** args, cudaStream_t stream,
                              int cluster = 1) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

struct RopeParams {
    const void* q;     // token t's query heads at q + t * q_stride, dt elements
    const void* k;     // and key / value heads at k, v + t * kv_stride
    const void* v;
    const void* bias;  // [(Hq + 2 Hkv) * D] or nullptr
    void* qo;          // dense [n][Hq][D], [n][Hkv][D]
    void* ko;
    void* vo;
    const int32_t* pos;  // [axes][n]
    long long n, q_stride, kv_stride;
    int Hq, Hkv, heads;  // heads: Hq + Hkv, and Hkv value heads more when they are moved too
    int D, R, dt, axes;
    int adjacent;        // pairs (2i, 2i + 1) instead of (i, i + R / 2)
    uint64_t step[64];   // turns per position of pair i, in units of 2^-64
    unsigned char axis[64];
    // set by the launcher
    int tile, heads_per_block;
    uint32_t div_h[2];
};
// vec: elements per access (up to 16 bytes); every pointer and stride aligned to it, R / 2 a multiple of it.
cudaError_t launch_rope(RopeParams p, int vec, int sms, cudaStream_t stream);

struct WeightsParams {
    const float* scores;  // as DecodeParams::scores / stats
    const float2* stats;
    const int32_t* seq_lens;
    const int32_t* next_pos;     // [B], with positions
    const int32_t* block_table;  // nullptr: planes are [B][Hkv][Lmax], else [num_pages][Hkv][page_size]
    const float* acc;
    float* acc_out;
    int32_t* positions;  // or nullptr
    const uint32_t* err;  // the step's error word: after a timeout the planes stay as they are
    int B, Hkv, Lmax, nq, group, window;
    int pages_per_seq, page_shift, num_pages;
    bool discard;  // set by the launcher: the scores' lines are dropped from L2 once read
};
cudaError_t launch_weights(WeightsParams p, cudaStream_t stream);

struct EvictParams {
    unsigned char* k_cache;
    unsigned char* v_cache;
    float* k_scales;  // nullptr unless INT8
    float* v_scales;
    const int32_t* seq_lens;
    int32_t* new_lens;
    const int32_t* next_pos;
    const int32_t* block_table;
    const float* acc;
    float* acc_out;
    const int32_t* positions;
    int32_t* positions_out;
    uint32_t* keys;   // workspace [B * Hkv][Lmax], for segments whose keys do not fit shared memory
    int2* moves;        // workspace [B * Hkv * (Lmax / 2)]: source and destination cache rows
    int2* local_moves;  // workspace [B * Hkv][kMaxLocalMoves]
    uint32_t* count;    // [2]: moves listed, blocks done; zero between calls
    uint32_t* err;
    int B, Hkv, Lmax;
    int row_bytes;  // D elements
    int budget, recent, sinks;
    int smem_keys;  // set by the launcher: keys of a block that its shared memory holds
    int pages_per_seq, page_shift, num_pages;
};
// Most moves of one kv head that its selection makes itself, in place of the move kernel.
constexpr int kMaxLocalMoves = 256;
cudaError_t launch_evict(EvictParams p, int sms, cudaStream_t stream);
// One-time set-up on the current device (shared-memory limits).
cudaError_t setup_evict();

}  // namespace ftd
