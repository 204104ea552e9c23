// ftd_weights.cu -- accumulated attention weights: the second kernel of
// ftd_decode_mha_scored.
//
// The step's kernel (mode kScored) leaves every visible score s of a query row and the
// row's reference m and 1 / l, l = sum 2^(s - m); here, for each cached position,
//   acc_out[b, h, t] = acc[b, h, t] + sum over the kv head's query rows of 2^(s - m) / l
// (the new tokens' own positions start from 0), and the new positions' ordinals go into
// the positions plane.  One thread owns four consecutive positions, so the sum runs in
// a fixed order, and no atomic takes part.
//
// Why two kernels: a weight needs its row's final maximum and sum, which the split over
// the cache's length knows only at its end.  Keeping the scores costs 4 bytes written
// and read per (query row, position), most of it in L2; reading K a second time
// would cost 2 D bytes per position.  Bound: those scores and 8 bytes of plane.
#include <cuda_runtime.h>

#include "ftd_ops.cuh"

namespace ftd {
namespace {

constexpr int kThreadsW = 128;
constexpr int kPosW = 4 * kThreadsW;  // positions per block

// Cache-plane row of position t (a multiple of 4 and the three after it: pages are multiples of 128)
__device__ __forceinline__ long long plane_row(const WeightsParams& p, int b, int kvh, int t) {
    if (!p.block_table) return (static_cast<long long>(b) * p.Hkv + kvh) * p.Lmax + t;
    const int page = __ldcg(p.block_table + static_cast<size_t>(b) * p.pages_per_seq + (t >> p.page_shift));
    if (page < 0 || page >= p.num_pages) return -1;  // the step's kernel has raised the error
    return ((static_cast<long long>(page) * p.Hkv + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

__global__ void __launch_bounds__(kThreadsW) weights_kernel(const WeightsParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int chunks = (p.Lmax + kPosW - 1) / kPosW;
    const int seg = blockIdx.x / chunks, chunk = blockIdx.x - seg * chunks;
    const int b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    const int L = __ldcg(p.seq_lens + b);
    if (L < 0 || L > p.Lmax - p.nq) return;  // inactive or overflowing: the planes stay as they are
    const int t = chunk * kPosW + 4 * threadIdx.x;
    const int end = L + p.nq;
    if (t >= end) return;
    const int start = window_start(L, p.window);  // the oldest position any row sees
    const bool unseen = t + 3 < start;
    if (unseen && p.acc_out == p.acc) return;
    const long long row = plane_row(p, b, kvh, t);
    if (row < 0) return;
    float a[4];
    *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(p.acc + row);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t + i >= L) a[i] = 0.f;
    if (!unseen) {
        const int rows = p.nq * p.group;
        const size_t r0 = static_cast<size_t>(seg) * rows;
        const float* s = p.scores + r0 * p.Lmax + t;
        const float2* st = p.stats + r0;
        for (int tok = 0; tok < p.nq; ++tok) {
            const int hi = L + tok, lo = p.window > 0 ? hi + 1 - p.window : 0;  // this token sees lo .. hi
            if (t <= hi && t + 3 >= lo) {
                const float* sr = s + static_cast<size_t>(tok) * p.group * p.Lmax;
                const float2* str = st + tok * p.group;
                float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
                for (int g = 0; g < p.group; ++g) {
                    const float4 x = __ldcs(reinterpret_cast<const float4*>(sr + static_cast<size_t>(g) * p.Lmax));
                    const float2 ml = __ldcg(str + g);
                    w[0] = fmaf(exp2f(x.x - ml.x), ml.y, w[0]);
                    w[1] = fmaf(exp2f(x.y - ml.x), ml.y, w[1]);
                    w[2] = fmaf(exp2f(x.z - ml.x), ml.y, w[2]);
                    w[3] = fmaf(exp2f(x.w - ml.x), ml.y, w[3]);
                }
                // (scores outside lo .. hi were never written: whatever they gave is dropped)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t + i >= lo && t + i <= hi) a[i] += w[i];
            }
        }
    }
    if (t + 3 < end) {
        *reinterpret_cast<float4*>(p.acc_out + row) = make_float4(a[0], a[1], a[2], a[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i < end) p.acc_out[row + i] = a[i];
    }
    if (p.positions && t + 3 >= L) {
        const int base = __ldcg(p.next_pos + b) - L;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i >= L && t + i < end) p.positions[row + i] = base + t + i;
    }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, cudaStream_t stream) {
    const int chunks = (p.Lmax + kPosW - 1) / kPosW;
    void* args[] = {const_cast<WeightsParams*>(&p)};
    return launch_pdl(reinterpret_cast<const void*>(&weights_kernel),
                      dim3(static_cast<unsigned>(p.B) * p.Hkv * chunks), kThreadsW, 0, args, stream);
}

}  // namespace ftd
