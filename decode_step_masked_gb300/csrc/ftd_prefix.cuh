// ftd_prefix.cuh -- attention of a batch to a prefix that its slots share, computed once for all
// of them (ftd_decode_mha_prefix): parameters, the cut into work, and the layout of partials.
//
// With B slots of T new tokens and group query heads per kv head, a kv head's query rows over the
// prefix are R = B * T * group, row = (slot * T + token) * group + head in group: a matrix
// product over one K and one V, where the step reads every slot's own rows for T * group rows at
// a time.  The softmax over prefix and own rows together is joined from parts: each part keeps, per query row,
// its reference m, its sum l of 2^(s - m) and its output o (scores s in the log2 domain), and
//   out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),  M = max_i m_i.
// The parts of a row are one of its own rows (the decode step writes its fp32 output, m and
// 1 / l), and one or more of the prefix, from the blocks that shared its length.
//
// Work: a segment is one kv head and one block of query rows, its tiles the rows of the prefix up to
// the longest that a slot of the block sees (a block whose slots see none has no tiles).  All segments'
// tiles form one space, heads first; the blocks of the grid take equal contiguous ranges of it, so a
// segment's pieces lie with neighbouring blocks, in slots (segment + block) of the workspace, which is
// unique because both only grow along the space.
#pragma once

#include "ftd_common.cuh"

namespace ftd {

// Most row blocks of a kv head (the plan keeps their tile prefix in shared memory).
constexpr int kMaxRowBlocks = 1024;

struct PrefixParams {
    const void* q;        // [B][T][Hq][D] qkv dtype
    const void* bias;     // its first Hq * D elements, or nullptr
    const unsigned char* k;  // cache dtype; row of (kv head, position) by prefix_row
    const unsigned char* v;
    const float* k_scales;   // INT8, by the same row
    const float* v_scales;
    const int32_t* table;    // pages of the prefix, or nullptr: rows [Hkv][P]
    const int32_t* prefix_lens;  // [B] rows of the prefix that a slot sees
    const int32_t* seq_lens;     // [B] slots without work see none
    float* ws;            // partials
    int2* seg_info;       // [Hkv * row blocks] first and last block that hold a piece of the segment
    uint32_t* err;
    // The slots' own rows, where the prefix's kernel takes them too (own): a segment is one slot and kv head.
    bool own;
    const void* k_new;    // [B][T][Hkv][D] qkv dtype
    const void* v_new;
    unsigned char* k_cache;  // contiguous [B][Hkv][Lmax][D], or pages through block_table
    unsigned char* v_cache;
    const int32_t* block_table;
    int pages_per_seq;
    float* own_ws;        // their partials
    int2* own_info;       // [B * Hkv] first and last worker of a segment
    // and where the decode step's kernel took them before:
    const float* own_o;   // [B][T][Hq][D]: its fp32 output
    const float2* own_ml; // [B][Hkv][T * group] (m, 1 / l)
    void* out;            // [B][T][Hq][D] out_dtype
    int out_dtype;
    int B, T, Hq, Hkv, group, D, Lmax;
    int P;                // rows of the prefix's buffer
    int R;                // query rows of a kv head: B * T * group
    int row_blocks, block_rows;  // row blocks of a kv head, and rows of a block
    int slot_rows;        // query rows of a partial slot
    bool split;           // the kernel runs two streams of half a slot's rows (prefix_twice)
    int stall;            // test hook: block 0's first copy never comes (see ftd_debug_stall_next)
    int workers;          // blocks of the grid
    int qkv_dtype;
    float qscale;         // softmax scale * log2(e)
    int page_shift, num_pages;
    long long wait_cycles;
};

// A partial slot of the workspace, of slot_rows rows: their m, their l, then D rows of outputs with the query rows
// side by side, as a thread that owns a query row writes them and as the join reads them.  A block of at most half a
// slot's rows (in the tensor-core kernel) is held twice: each half of the slot is one of the block's two streams.
__host__ __device__ inline size_t prefix_slot_floats(int slot_rows, int D) {
    return static_cast<size_t>(slot_rows) * (2 + D);
}
// A partial slot of own rows: m and l of the slot's query rows, then their outputs, D each.
__host__ __device__ inline int own_out_at(int rows) { return (2 * rows + 3) / 4 * 4; }
__host__ __device__ inline size_t own_slot_floats(int rows, int D) { return static_cast<size_t>(own_out_at(rows)) + static_cast<size_t>(rows) * D; }
// Most query rows of a slot's kv head (T * group) that the prefix's kernel takes the own rows of.
constexpr int kMostOwnRows = 32;
// Whether row block rb is held twice.
__device__ __forceinline__ bool prefix_twice(const PrefixParams& p, int rb) {
    return p.split && 2 * min(p.block_rows, p.R - rb * p.block_rows) <= p.slot_rows;
}

// Cache row (of D elements) of position t of kv head h; -1 for a page outside the pool.
__device__ __forceinline__ long long prefix_row(const PrefixParams& p, int h, int t) {
    if (!p.table) return static_cast<long long>(h) * p.P + t;
    const int page = __ldg(p.table + (t >> p.page_shift));
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<long long>(page) * p.Hkv + h) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// Rows of the prefix that a slot sees.
__device__ __forceinline__ int prefix_seen(const PrefixParams& p, int b) {
    const int L = __ldcg(p.seq_lens + b), n = __ldcg(p.prefix_lens + b);
    return L >= 0 && L <= p.Lmax - p.T ? min(max(n, 0), p.P) : 0;
}

// Rows that the row block's longest slot sees, by the lanes of a warp.
__device__ __forceinline__ int prefix_block_seen(const PrefixParams& p, int rb, int lane) {
    const int per = p.T * p.group, lo = rb * p.block_rows, hi = min(p.R, lo + p.block_rows) - 1;
    int most = 0;
    for (int b = lo / per + lane; b <= hi / per; b += 32) most = max(most, prefix_seen(p, b));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, m));
    return most;
}

// The cut of the work: first[rb], tiles (of `tile` rows of the prefix) of the row blocks before rb of one kv
// head, in shared memory.  By all threads of the block; two barriers.
__device__ __forceinline__ void build_prefix_plan(const PrefixParams& p, int* first, int tile) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x) >> 5;
    for (int rb = warp; rb < p.row_blocks; rb += warps) {
        const int most = prefix_block_seen(p, rb, lane);
        if (lane == 0) first[rb + 1] = (most + tile - 1) / tile;
    }
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const int L = __ldcg(p.seq_lens + b);
            if (L >= 0 && L <= p.Lmax - p.T && __ldcg(p.prefix_lens + b) > p.P) atomicOr(p.err, kErrSeqOverflow);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int base = 0; base < p.row_blocks; base += 32) {
            const int rb = base + lane;
            int v = rb < p.row_blocks ? first[rb + 1] : 0;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, m);
                if (lane >= m) v += y;
            }
            if (rb < p.row_blocks) first[rb + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) first[0] = 0;
    }
    __syncthreads();
}

// First of the tiles of worker w, of W that share U equally: floor(w U / W), by divisions of 32 bits where U has no more.
__device__ __forceinline__ long long equal_share(long long U, int W, int w) {
    if (w >= W) return U;
    if (U >= (1LL << 31)) return w * U / W;
    const uint32_t u = static_cast<uint32_t>(U), n = static_cast<uint32_t>(W), q = u / n;
    return static_cast<long long>(w) * q + static_cast<uint32_t>(w) * (u - q * n) / n;  // (w, u mod W < W <= 2^12)
}

// Equal contiguous ranges of U tiles over W blocks.
struct PrefixSplit {
    long long U;
    int W;
    __device__ PrefixSplit(const PrefixParams& p, const int* first)
        : U(static_cast<long long>(p.Hkv) * first[p.row_blocks]), W(static_cast<int>(min(static_cast<long long>(p.workers), max(U, 1LL)))) {}
    __device__ long long begin(int w) const { return equal_share(U, W, w); }
    __device__ int holder(long long u) const { return static_cast<int>(((u + 1) * W - 1) / U); }
};

// Place of tile u: kv head, row block, tile of it, and tiles of the row block.
struct PrefixCursor {
    int h, rb, tile, nt;
};
__device__ __forceinline__ PrefixCursor prefix_locate(long long u, const int* first, int row_blocks) {
    const int per = first[row_blocks];
    PrefixCursor c;
    c.h = u < (1LL << 31) ? static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(per)) : static_cast<int>(u / per);
    const int rem = static_cast<int>(u - static_cast<long long>(c.h) * per);
    int lo = 0, hi = row_blocks - 1;  // largest rb with first[rb] <= rem
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= rem) lo = mid;
        else hi = mid - 1;
    }
    c.rb = lo;
    c.tile = rem - first[lo];
    c.nt = first[lo + 1] - first[lo];
    return c;
}

// Which blocks hold pieces of each segment, for the join; by threads t, t + step, .. of the grid's first block.
__device__ __forceinline__ void write_seg_info(const PrefixParams& p, const int* first, const PrefixSplit& sp, int t, int step = 32) {
    const int per = first[p.row_blocks];
    for (int s = t; s < p.Hkv * p.row_blocks; s += step) {
        const int h = s / p.row_blocks, rb = s - h * p.row_blocks;
        const long long u0 = static_cast<long long>(h) * per + first[rb], u1 = static_cast<long long>(h) * per + first[rb + 1];
        p.seg_info[s] = u0 < u1 ? make_int2(sp.holder(u0), sp.holder(u1 - 1)) : make_int2(0, -1);
    }
}

// Query row -> slot, and row of q and out.
__device__ __forceinline__ int prefix_slot_of(const PrefixParams& p, int row) { return row / (p.T * p.group); }
__device__ __forceinline__ size_t prefix_q_row(const PrefixParams& p, int h, int row) {
    const int bt = row / p.group;
    return static_cast<size_t>(bt) * p.Hq + h * p.group + (row - bt * p.group);
}

struct PrefixKernel {
    const void* fn;
    int smem, threads;
    int block_rows;  // query rows of a block
    int slot_rows;   // and of a partial slot
    bool split;      // two streams of half a slot's rows (prefix_twice)
};
// The CUDA-core kernel: cache type, head dimension, query rows of a kv head.
PrefixKernel select_prefix_cc(int cache_dt, int D, int R);

// Joins every row's parts into out.
cudaError_t launch_prefix_join(PrefixParams p, cudaStream_t stream);

}  // namespace ftd
