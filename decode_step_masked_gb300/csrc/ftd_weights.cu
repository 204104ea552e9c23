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
// would cost 2 D bytes per position.  Bound: those scores and 8 bytes of plane.  Measured on top
// of the step's kernel: 4 us for 8 x 32 heads of 2048 rows (launch and latency), 6.4 us for 16 x 8
// heads of 8192 rows with 8 query rows each (42 MB, 6.5 TB/s from L2), 12 us for 64 x 32 heads of 1280 rows
// (32 MB in short rows).
#include <cuda_runtime.h>

#include "ftd_ops.cuh"

namespace ftd {
namespace {

constexpr int kThreadsW = 128;
constexpr int kMaxRowsPerThread = 12;

// What was complete before the step's kernel passed its own wait, read before this grid's: strong loads at
// GPU scope, which an L1 line left over from an earlier launch cannot answer (a plain load may be;
// cache operators are hints).  The old weights read after the wait instead: 7B-shaped 49.3 -> 50.0 us, 70B-shaped
// 95.8 -> 97.3, ragged INT8 135.0 -> 137.5.
__device__ __forceinline__ int ld_early(const int32_t* x) {
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(x));
    return v;
}
__device__ __forceinline__ float4 ld_early(const float4* x) {
    float4 v;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(x));
    return v;
}

// Cache-plane row of position t (a multiple of 4 and the three after it: pages are multiples of 128)
__device__ __forceinline__ long long plane_row(const WeightsParams& p, int b, int kvh, int t) {
    if (!p.block_table) return (static_cast<long long>(b) * p.Hkv + kvh) * p.Lmax + t;
    const int page = ld_early(p.block_table + static_cast<size_t>(b) * p.pages_per_seq + (t >> p.page_shift));
    if (page < 0 || page >= p.num_pages) return -1;  // the step's kernel has raised the error
    return ((static_cast<long long>(page) * p.Hkv + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// Whether a page that slot b's rows see, positions [start, end), is bad (every lane of a warp gets the answer):
// the step's weights are then undefined, and the planes keep the slot's old ones.
__device__ __forceinline__ bool bad_slot(const WeightsParams& p, int b, int start, int end) {
    if (!p.block_table) return false;
    const int32_t* row = p.block_table + static_cast<size_t>(b) * p.pages_per_seq;
    bool bad = false;
    for (int i = (start >> p.page_shift) + (static_cast<int>(threadIdx.x) & 31); i < (end + (1 << p.page_shift) - 1) >> p.page_shift; i += 32) {
        const int page = ld_early(row + i);
        bad |= page < 0 || page >= p.num_pages;
    }
    return __any_sync(0xffffffffu, bad);
}
// Whether the step gave up on a copy (read after the wait: the step's kernel sets it).
__device__ __forceinline__ bool gave_up(const WeightsParams& p) { return *p.err & kErrTimeout; }

// The scores of 128 positions from t0 are read: drop their lines from L2, or they would go to memory
// on their way out, dirty as they are.  Thread i of n drops every n-th line of the segment's rows.
__device__ __forceinline__ void drop_scores(const WeightsParams& p, size_t r0, int t0, int end, int i, int n) {
    for (int k = i; k < 4 * p.nq * p.group; k += n) {
        const int t = t0 + 32 * (k & 3);
        if (t < end)
            asm volatile("discard.global.L2 [%0], 128;" ::"l"(p.scores + (r0 + (k >> 2)) * p.Lmax + t) : "memory");
    }
}

// Each thread owns Q quads of four positions, a block's quads kThreadsW apart: with few
// query rows a quad is one or two 16-byte loads of scores, and several are kept in flight.
template <int Q>
__global__ void __launch_bounds__(kThreadsW) weights_kernel(const WeightsParams p) {
    // Everything but the scores and their statistics is older than the step's kernel, which
    // lets this grid start only after its own wait, and which writes none of it: lengths, pages and old
    // weights are read (ld_early) while that kernel finishes.  Every block waits for it, those without work
    // too: the next launch on the stream counts on this grid's end to come after the step's.
    constexpr int POS = 4 * kThreadsW * Q;  // positions per block
    const int chunks = (p.Lmax + POS - 1) / POS;
    const int seg = blockIdx.x / chunks, chunk = blockIdx.x - seg * chunks;
    const int b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    const int L = ld_early(p.seq_lens + b);
    // inactive or overflowing slots: the planes stay as they are
    const int end = L < 0 || L > p.Lmax - p.nq ? 0 : L + p.nq;
    const int start = window_start(L, p.window);  // the oldest position any row sees
    int t[Q];
    long long row[Q];  // -1: nothing to do
    float a[Q][4], sum[Q][4];  // the old weights, and what this call adds (summed apart: one rounding against a)
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        t[i] = chunk * POS + (i * kThreadsW + static_cast<int>(threadIdx.x)) * 4;
        row[i] = t[i] >= end || (t[i] + 3 < start && p.acc_out == p.acc) ? -1 : plane_row(p, b, kvh, t[i]);
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const float4 x = row[i] >= 0 ? ld_early(reinterpret_cast<const float4*>(p.acc + row[i])) : make_float4(0.f, 0.f, 0.f, 0.f);
        a[i][0] = x.x;
        a[i][1] = x.y;
        a[i][2] = x.z;
        a[i][3] = x.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;
    }
    const size_t r0 = static_cast<size_t>(seg) * (p.nq * p.group);
    const bool bad = bad_slot(p, b, start, end);
    grid_dep_wait();
    grid_dep_launch();
    if (chunk * POS >= end || bad) return;
    const bool keep = gave_up(p);
    float w[Q][4];
    for (int tok = 0; tok < p.nq; ++tok) {
        const int hi = L + tok, lo = p.window > 0 ? hi + 1 - p.window : 0;  // this token sees lo .. hi
        const float* s = p.scores + (r0 + static_cast<size_t>(tok) * p.group) * p.Lmax;
        const float2* st = p.stats + r0 + tok * p.group;
        bool live[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            live[i] = row[i] >= 0 && t[i] <= hi && t[i] + 3 >= lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[i][e] = 0.f;
        }
#pragma unroll (8 / Q)
        for (int g = 0; g < p.group; ++g) {
            const float2 ml = __ldcg(st + g);
            float4 x[Q];
#pragma unroll
            for (int i = 0; i < Q; ++i)
                if (live[i]) x[i] = __ldcs(reinterpret_cast<const float4*>(s + static_cast<size_t>(g) * p.Lmax + t[i]));
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                if (!live[i]) continue;
                w[i][0] = fmaf(exp2f(x[i].x - ml.x), ml.y, w[i][0]);
                w[i][1] = fmaf(exp2f(x[i].y - ml.x), ml.y, w[i][1]);
                w[i][2] = fmaf(exp2f(x[i].z - ml.x), ml.y, w[i][2]);
                w[i][3] = fmaf(exp2f(x[i].w - ml.x), ml.y, w[i][3]);
            }
        }
        // (scores outside lo .. hi were never written: whatever they gave is dropped)
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (live[i] && t[i] + e >= lo && t[i] + e <= hi) sum[i][e] += w[i][e];
    }
    if (keep) return;
    if (p.discard) {
        __syncwarp();  // (orders every lane's reads before the drops)
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < Q; ++i) drop_scores(p, r0, t[i] - 4 * lane, end, lane, 32);
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        if (row[i] < 0) continue;
        // the new tokens' positions start from 0, not from what acc holds there
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = (t[i] + e < L ? a[i][e] : 0.f) + sum[i][e];
        if (t[i] + 3 < end) {
            *reinterpret_cast<float4*>(p.acc_out + row[i]) = make_float4(a[i][0], a[i][1], a[i][2], a[i][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t[i] + e < end) p.acc_out[row[i] + e] = a[i][e];
        }
        if (p.positions && t[i] + 3 >= L) {
            const int base = __ldcg(p.next_pos + b) - L;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t[i] + e >= L && t[i] + e < end) p.positions[row[i] + e] = base + t[i] + e;
        }
    }
}

// Many query rows: a block's warps take every kWarpsW-th row of the same 128 positions and add up
// through shared memory, in warp order.
constexpr int kWarpsW = 8;
__global__ void __launch_bounds__(32 * kWarpsW) weights_rows_kernel(const WeightsParams p) {
    __shared__ float4 part[kWarpsW][32];
    constexpr int POS = 128;
    const int chunks = (p.Lmax + POS - 1) / POS;
    const int seg = blockIdx.x / chunks, chunk = blockIdx.x - seg * chunks;
    const int b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = ld_early(p.seq_lens + b);
    const int start = window_start(L, p.window), t0 = chunk * POS, t = t0 + 4 * lane;
    int end = L < 0 || L > p.Lmax - p.nq ? 0 : L + p.nq;
    if (bad_slot(p, b, start, end)) end = 0;
    grid_dep_wait();  // (as in weights_kernel)
    grid_dep_launch();
    if (t0 >= end || (t0 + POS <= start && p.acc_out == p.acc)) return;
    const bool keep = gave_up(p);
    const int rows = p.nq * p.group;
    const size_t r0 = static_cast<size_t>(seg) * rows;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;
    for (int r = warp; r < rows; r += U * kWarpsW) {
        float4 x[U];
        float2 ml[U];
        int hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = r + u * kWarpsW;
            hi[u] = -1;
            if (i < rows && t < end) {  // (a row may end inside the block's positions)
                hi[u] = L + i / p.group;  // the row's token sees positions up to hi
                ml[u] = __ldcg(p.stats + r0 + i);
                x[u] = __ldcs(reinterpret_cast<const float4*>(p.scores + (r0 + i) * p.Lmax + t));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (hi[u] < 0) continue;
            const int lo = p.window > 0 ? hi[u] + 1 - p.window : 0;
            const float s[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)  // (scores outside lo .. hi were never written)
                if (t + e >= lo && t + e <= hi[u]) w[e] = fmaf(exp2f(s[e] - ml[u].x), ml[u].y, w[e]);
        }
    }
    if (keep) return;
    part[warp][lane] = make_float4(w[0], w[1], w[2], w[3]);
    __syncthreads();
    if (p.discard) drop_scores(p, r0, t0, end, static_cast<int>(threadIdx.x), 32 * kWarpsW);
    if (warp != 0 || t >= end) return;
    const long long row = plane_row(p, b, kvh, t);
    if (row < 0) return;
    const float4 old = *reinterpret_cast<const float4*>(p.acc + row);
    float a[4] = {old.x, old.y, old.z, old.w}, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kWarpsW; ++k) {
        const float4 x = part[k][lane];
        sum[0] += x.x;
        sum[1] += x.y;
        sum[2] += x.z;
        sum[3] += x.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = (t + e < L ? a[e] : 0.f) + sum[e];  // one rounding against the old weight
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (t + e >= end) break;
        p.acc_out[row + e] = a[e];
        if (p.positions && t + e >= L) p.positions[row + e] = __ldcg(p.next_pos + b) + t + e - L;
    }
}

template <int Q>
cudaError_t launch(const WeightsParams& p, cudaStream_t stream) {
    const int chunks = (p.Lmax + 4 * kThreadsW * Q - 1) / (4 * kThreadsW * Q);
    void* args[] = {const_cast<WeightsParams*>(&p)};
    return launch_pdl(reinterpret_cast<const void*>(&weights_kernel<Q>),
                      dim3(static_cast<unsigned>(p.B) * p.Hkv * chunks), kThreadsW, 0, args, stream);
}

}  // namespace

cudaError_t launch_weights(WeightsParams p, cudaStream_t stream) {
    // Quads of positions a thread: four for one or two query rows per kv head, two for three and four, one from five
    // on (their rows keep the loads in flight); above kMaxRowsPerThread rows a block's warps share them.  Whole
    // scored steps of 16 slots, 8 kv heads, 4080 rows, us with four / two / one quad / shared: 1 query row 49.4 / 50.0 /
    // 48.8 / 59.4, 2 62.6 / 61.5 / 61.8 / 71.5, 4 55.6 / 54.5 / 55.0 / 64.4, 8 60.5 / 58.3 / 58.8 / 65.0, 12 72.8 / 69.1 / 69.5 /
    // 74.5, 16 76.7 / 72.3 / 72.4 / 75.8; where a kv head has the blocks to itself, 8 slots, one kv head, 8176 rows: 16
    // query rows 37.4 / 33.0 / 33.4 / 28.7, 24 47.4 / 40.6 / 42.1 / 31.4, 128 167 / 132 / 136 / 55.5.
    const int rows = p.nq * p.group;
    // Workspaces of 16 MB of scores and more, an eighth of L2, are dropped after their reading where rows are
    // whole lines.  Three states in turn, kept -> dropped, us: 16-bit one query row 4.2 / 8.4 / 16.8 MB, half full 49.5 -> 49.6,
    // 89.6 -> 89.0, 172.6 -> 169.6; eight query rows 8.4 / 16.8 / 25.2 / 33.6 MB, full 38.1 -> 39.5, 59.6 -> 58.2, 80.9 -> 77.9, 103.0 ->
    // 97.8; INT8 16.8 MB 132.8 -> 132.9.  The rule goes by the context's size: short contents in a large context (33.6 MB,
    // 512 of 8192 rows) pay for it, 24.3 -> 25.4.
    p.discard = p.Lmax % 32 == 0 && static_cast<size_t>(p.B) * p.Hkv * rows * p.Lmax * sizeof(float) >= (16u << 20);
    if (rows <= 2) return launch<4>(p, stream);
    if (rows <= 4) return launch<2>(p, stream);
    if (rows <= kMaxRowsPerThread) return launch<1>(p, stream);
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(&weights_rows_kernel),
                      dim3(static_cast<unsigned>(p.B) * p.Hkv * ((p.Lmax + 127) / 128)), 32 * kWarpsW, 0, args, stream);
}

}  // namespace ftd
