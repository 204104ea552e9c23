// ftd_evict.cu -- eviction from the cache by accumulated attention weight
// (ftd_cache_evict): two kernels.
//
// Each (slot, kv head) keeps `budget` of its L rows, in the order of the key
//   protected (position < sinks, or >= next_pos - recent)  >  weight  >  row index (lower first).
// A cache's rows are order free (positions are in K already), so nothing is shifted: the
// j-th kept row at an index >= budget moves into the j-th row below budget that goes.
// Rows move from [budget, L) to [0, budget), so no row is read and written, every move
// can run at the same time, and only rows that must move do.
//
// select_kernel, one block per (slot, kv head): the weights become 32-bit keys whose
// unsigned order is theirs; the budget-th largest key is found two bits at a time, by
// counting, over keys held in shared memory, the four values of the next two bits among
// the keys that match the bits found so far (counts are sums: no atomics, any order gives
// the same result), at most 16 rounds of one block barrier each.  Then two more
// sweeps rank ties and list the moves.  A block reserves its part of the call's one move
// list with an atomic add; the list's order varies, but its moves are independent.
// move_kernel splits the list evenly over all warps and copies rows and their planes.
//
// Bound: 8 bytes per position for the selection, then the moved rows, read and written.
#include <cuda_runtime.h>

#include "ftd_ops.cuh"

namespace ftd {
namespace {

constexpr int kThreadsE = 1024;
constexpr int kWarpsE = kThreadsE / 32;
constexpr int kSmemKeys = 48 * 1024;  // keys that fit shared memory (192 KB)
constexpr int kMoveThreads = 256;

__device__ __forceinline__ long long evict_row(const EvictParams& p, int b, int kvh, int t) {
    if (!p.block_table) return (static_cast<long long>(b) * p.Hkv + kvh) * p.Lmax + t;
    const int page = __ldcg(p.block_table + static_cast<size_t>(b) * p.pages_per_seq + (t >> p.page_shift));
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<long long>(page) * p.Hkv + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// Unsigned key in the order of the weights (NaN below every number), all below ~0u.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreadsE) select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t skeys[];
    __shared__ uint2 cnt[2][kWarpsE];
    __shared__ int wsum[kWarpsE], wsum2[kWarpsE];
    __shared__ uint32_t list_base;
    constexpr unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x, b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    grid_dep_wait();
    grid_dep_launch();
    const int L = __ldcg(p.seq_lens + b);
    if (L <= 0) return;
    if (L > p.Lmax) {
        if (tid == 0) atomicOr(p.err, kErrSeqOverflow);
        return;
    }
    const bool apart = p.acc_out != p.acc, papart = p.positions_out != p.positions;
    if (L <= p.budget) {  // everything stays
        if (apart || papart)
            for (int t = tid; t < L; t += kThreadsE) {
                const long long row = evict_row(p, b, kvh, t);
                if (row < 0) {
                    atomicOr(p.err, kErrBadPage);
                    continue;
                }
                if (apart) p.acc_out[row] = p.acc[row];
                if (papart) p.positions_out[row] = p.positions[row];
            }
        return;
    }
    // ---- keys; a warp owns a contiguous run of positions ----
    uint32_t* keys = L <= kSmemKeys ? skeys : p.keys + static_cast<size_t>(seg) * p.Lmax;
    const int S = ((L + kWarpsE - 1) / kWarpsE + 31) & ~31;
    const int w0 = min(L, warp * S), w1 = min(L, w0 + S);
    const long long fresh = static_cast<long long>(__ldcg(p.next_pos + b)) - p.recent;
    bool bad = false;
    for (int t = w0 + lane; t < w1; t += 32) {
        const long long row = evict_row(p, b, kvh, t);
        uint32_t key = 0u;
        if (row < 0) {
            bad = true;
        } else {
            const int pos = p.positions[row];
            key = ((pos >= 0 && pos < p.sinks) || (p.recent > 0 && pos >= fresh)) ? 0xffffffffu : weight_key(p.acc[row]);
        }
        keys[t] = key;
    }
    if (__syncthreads_or(bad)) {  // a page of this slot is bad: it is left as it is
        if (tid == 0) atomicOr(p.err, kErrBadPage);
        return;
    }
    // ---- the budget-th largest key ----
    uint32_t prefix = 0u;     // bits found so far (from the top)
    int need = p.budget;      // kept rows still to be found among the keys with this prefix
    int shift = 30;
    bool whole = false;       // every key with the prefix is kept
    for (;;) {
        // counts of the next two bits' values, 16 bits each: a warp's run is at most
        // kMaxEvictLen / 32 = 32768 keys
        uint32_t c01 = 0u, c23 = 0u;
        const bool first = shift == 30;
        for (int t = w0 + lane; t < w1; t += 32) {
            const uint32_t k = keys[t];
            if (first || (k >> (shift + 2)) == prefix) {
                const uint32_t d = (k >> shift) & 3u;
                const uint32_t one = (d & 1u) ? 0x10000u : 1u;
                if (d & 2u) c23 += one;
                else c01 += one;
            }
        }
        c01 = __reduce_add_sync(FULL, c01);
        c23 = __reduce_add_sync(FULL, c23);
        const int buf = (shift >> 1) & 1;
        if (lane == 0) cnt[buf][warp] = make_uint2(c01, c23);
        __syncthreads();
        const uint2 x = cnt[buf][lane];
        const int n1 = static_cast<int>(__reduce_add_sync(FULL, x.x >> 16));
        const int n2 = static_cast<int>(__reduce_add_sync(FULL, x.y & 0xffffu));
        const int n3 = static_cast<int>(__reduce_add_sync(FULL, x.y >> 16));
        const int n0 = static_cast<int>(__reduce_add_sync(FULL, x.x & 0xffffu));
        int d, n;
        if (need <= n3) { d = 3; n = n3; }
        else if (need <= n3 + n2) { d = 2; n = n2; need -= n3; }
        else if (need <= n3 + n2 + n1) { d = 1; n = n1; need -= n3 + n2; }
        else { d = 0; n = n0; need -= n3 + n2 + n1; }
        prefix = (prefix << 2) | static_cast<uint32_t>(d);
        whole = need == n;
        if (whole || shift == 0) break;
        shift -= 2;
    }
    const uint32_t lo = prefix << shift;  // the smallest key with the prefix
    // ---- ties: the first `need` keys equal to lo, by row index ----
    int ties_before = 0;  // in earlier warps
    if (!whole) {
        int n = 0;
        for (int t0 = w0; t0 < w1; t0 += 32) {
            const int t = t0 + lane;
            n += __popc(__ballot_sync(FULL, t < w1 && keys[t] == lo));
        }
        if (lane == 0) wsum[warp] = n;
        __syncthreads();
        const int v = wsum[lane];
        ties_before = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < warp ? v : 0)));
        __syncthreads();
    }
    auto kept_at = [&](int t, int& ties) {  // whole warp, consecutive groups in order
        const uint32_t k = t < w1 ? keys[t] : 0u;
        bool kept = t < w1 && (whole ? k >= lo : k > lo);
        if (!whole) {
            const bool tie = t < w1 && k == lo;
            const unsigned m = __ballot_sync(FULL, tie);
            if (tie) kept = ties + __popc(m & ((1u << lane) - 1u)) < need;
            ties += __popc(m);
        }
        return kept;
    };
    // ---- holes below the budget and kept rows from it on: counted, then listed ----
    int holes = 0, movers = 0, ties = ties_before;
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int t = t0 + lane;
        const bool kept = kept_at(t, ties);
        holes += __popc(__ballot_sync(FULL, t < w1 && t < p.budget && !kept));
        movers += __popc(__ballot_sync(FULL, t >= p.budget && kept));
    }
    if (lane == 0) {
        wsum[warp] = holes;
        wsum2[warp] = movers;
    }
    __syncthreads();
    {
        const int h = wsum[lane], m = wsum2[lane];
        holes = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < warp ? h : 0)));
        movers = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < warp ? m : 0)));
        const uint32_t total = __reduce_add_sync(FULL, static_cast<unsigned>(h));
        if (tid == 0) list_base = total ? atomicAdd(p.count, total) : 0u;
    }
    __syncthreads();
    int2* list = p.moves + list_base;
    ties = ties_before;
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int t = t0 + lane;
        const bool kept = kept_at(t, ties);
        const bool hole = t < w1 && t < p.budget && !kept, mover = t >= p.budget && kept;
        const unsigned hm = __ballot_sync(FULL, hole), mm = __ballot_sync(FULL, mover);
        const unsigned below = (1u << lane) - 1u;
        if (hole) list[holes + __popc(hm & below)].y = static_cast<int>(evict_row(p, b, kvh, t));
        if (mover) list[movers + __popc(mm & below)].x = static_cast<int>(evict_row(p, b, kvh, t));
        holes += __popc(hm);
        movers += __popc(mm);
        if ((apart || papart) && kept && t < p.budget) {
            const long long row = evict_row(p, b, kvh, t);
            if (apart) p.acc_out[row] = p.acc[row];
            if (papart) p.positions_out[row] = p.positions[row];
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
    constexpr int U = 4;
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const long long W = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    const long long w = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
    const long long M = __ldcg(p.count);
    const int m0 = static_cast<int>(M * w / W), m1 = static_cast<int>(M * (w + 1) / W);
    // a row's K and V as 16-byte words, consecutive lanes along one row
    const int words = p.row_bytes >> 4;             // a power of two
    const int shift = 31 - __clz(2 * words);
    const long long i1 = static_cast<long long>(m1) << shift;
    for (long long i = (static_cast<long long>(m0) << shift) + lane; i < i1; i += 32 * U) {
        uint4 x[U];
        unsigned char* dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long j = i + 32 * u;
            dst[u] = nullptr;
            if (j < i1) {
                const int2 mv = __ldcg(p.moves + (j >> shift));
                const int c = static_cast<int>(j) & (2 * words - 1);
                unsigned char* base = c < words ? p.k_cache : p.v_cache;
                const int off = (c & (words - 1)) * 16;
                x[u] = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<long long>(mv.x) * p.row_bytes + off));
                dst[u] = base + static_cast<long long>(mv.y) * p.row_bytes + off;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
    }
    for (int m = m0 + lane; m < m1; m += 32) {
        const int2 mv = __ldcg(p.moves + m);
        p.acc_out[mv.y] = p.acc[mv.x];
        p.positions_out[mv.y] = p.positions[mv.x];
        if (p.k_scales) {
            p.k_scales[mv.y] = p.k_scales[mv.x];
            p.v_scales[mv.y] = p.v_scales[mv.x];
        }
    }
    // new lengths after every selection has read the old ones (new_lens may be seq_lens)
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += kMoveThreads) {
            const int L = p.seq_lens[b];
            p.new_lens[b] = (L > p.budget && L <= p.Lmax) ? p.budget : L;
        }
    // the last block to finish leaves the counters at zero for the next call
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t done = arrive_acq_rel(p.count + 1, 1u);
        if (done == gridDim.x - 1) {
            p.count[0] = 0u;
            p.count[1] = 0u;
        }
    }
}

}  // namespace

cudaError_t setup_evict() {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(&select_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemKeys * 4);
}

cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    void* args[] = {const_cast<EvictParams*>(&p)};
    const int nk = p.Lmax < kSmemKeys ? p.Lmax : kSmemKeys;
    const cudaError_t e = launch_pdl(reinterpret_cast<const void*>(&select_kernel),
                                     dim3(static_cast<unsigned>(p.B) * p.Hkv), kThreadsE, nk * 4, args, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(reinterpret_cast<const void*>(&move_kernel), dim3(static_cast<unsigned>(sms) * 4), kMoveThreads, 0,
                      args, stream);
}

}  // namespace ftd
