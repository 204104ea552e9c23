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
// select_kernel, one cluster of 1 to 8 blocks per (slot, kv head), each block with a
// contiguous part of the rows: the weights become 32-bit keys whose unsigned order is
// theirs, held in shared memory; the budget-th largest is found eight bits at a time
// (histograms of the next byte among the keys that match so far, added up over the
// cluster through distributed shared memory: sums, so any order of the atomics gives the
// same result), in at most four rounds.  Then the moves are listed in row order
// (ranks by ballots, warp and block prefixes).  The cluster reserves its part of the
// call's one move list with an atomic add; the list's order varies, its moves are independent.
// move_kernel deals the list out to all warps in chunks of rows and copies rows and planes.
//
// Bound: 8 bytes per position for the selection, then the moved rows, read and written.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "ftd_ops.cuh"

namespace cg = cooperative_groups;

namespace ftd {
namespace {

constexpr int kThreadsE = 512;
constexpr int kWarpsE = kThreadsE / 32;
constexpr int kMaxCluster = 8;
constexpr int kSmemKeys = 48 * 1024;  // keys of a block that fit shared memory (192 KB)
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;  // rows a warp copies at a time

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

// What the blocks of a cluster read of each other.
struct alignas(16) Shared {
    uint32_t hist[2][256];
    int ties, holes, movers;  // of this block
    uint32_t list_base;       // of the cluster (block 0's)
    int bad;
};

__global__ void __launch_bounds__(kThreadsE) select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t skeys[];
    __shared__ Shared sh;
    __shared__ int wsum[kWarpsE], wsum2[kWarpsE];
    __shared__ int found[3];  // digit, rows needed of it, keys with it
    constexpr unsigned FULL = 0xffffffffu;
    const cg::cluster_group cluster = cg::this_cluster();
    const int cl = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x / cl, b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    // every thread of the cluster (or, alone, of the block) has written what it shares
    auto meet = [&]() {
        if (cl > 1) cluster.sync();
        else __syncthreads();
    };
    if (tid < 256) sh.hist[0][tid] = 0u;
    if (tid == 0) sh.bad = 0;
    grid_dep_wait();
    grid_dep_launch();
    const int L = __ldcg(p.seq_lens + b);
    if (L <= 0) return;
    if (L > p.Lmax) {
        if (tid == 0 && rank == 0) atomicOr(p.err, kErrSeqOverflow);
        return;
    }
    const bool apart = p.acc_out != p.acc, papart = p.positions_out != p.positions;
    if (L <= p.budget) {  // everything stays
        if (apart || papart)
            for (int t = rank * kThreadsE + tid; t < L; t += cl * kThreadsE) {
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
    // ---- keys; a warp owns a contiguous run of S rows, a block the runs of its warps ----
    const int S = ((L + cl * kWarpsE - 1) / (cl * kWarpsE) + 31) & ~31;
    const int c0 = rank * kWarpsE * S;  // the block's first row (may lie past L)
    const int w0 = min(L, c0 + warp * S), w1 = min(L, w0 + S);
    // keys[t] for row t of this block
    uint32_t* keys = (S * kWarpsE <= p.smem_keys ? skeys : p.keys + static_cast<size_t>(seg) * p.Lmax + min(c0, L)) - min(c0, L);
    const long long fresh = static_cast<long long>(__ldcg(p.next_pos + b)) - p.recent;
    bool bad = false;
    constexpr int U = 4;  // rows a lane has in flight
    for (int t0 = w0 + lane; t0 < w1; t0 += 32 * U) {
        float a[U];
        int ps[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + 32 * u;
            a[u] = 0.f;
            ps[u] = 0;
            if (t < w1) {
                const long long row = evict_row(p, b, kvh, t);
                if (row < 0) {
                    bad = true;
                } else {
                    a[u] = p.acc[row];
                    ps[u] = p.positions[row];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + 32 * u;
            if (t < w1)
                keys[t] = ((ps[u] >= 0 && ps[u] < p.sinks) || (p.recent > 0 && ps[u] >= fresh)) ? 0xffffffffu : weight_key(a[u]);
        }
    }
    if (bad) sh.bad = 1;
    __syncthreads();
    // ---- the budget-th largest key, a byte at a time from the top ----
    uint32_t prefix = 0u;  // bytes found so far
    int need = p.budget;   // kept rows still to be found among the keys with this prefix
    int shift = 24;
    bool whole = false;    // every key with the prefix is kept
    for (int round = 0;; ++round) {
        uint32_t* hist = sh.hist[round & 1];
        for (int t = w0 + lane; t < w1; t += 32) {
            const uint32_t k = keys[t];
            if (round == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        meet();
        if (round == 0) {
            int any = 0;
            for (int r = 0; r < cl; ++r) any |= cl > 1 ? *cluster.map_shared_rank(&sh.bad, r) : sh.bad;
            if (any) {  // a page of this slot is bad: it is left as it is
                if (tid == 0 && rank == 0) atomicOr(p.err, kErrBadPage);
                meet();  // no block leaves while another reads its flag
                return;
            }
        }
        if (tid < 256) sh.hist[(round + 1) & 1][tid] = 0u;  // (read last before this meeting)
        if (warp == 0) {
            // lane owns bytes 8 lane .. 8 lane + 7; keys above them: those of the later lanes
            uint32_t h[8] = {};
            for (int r = 0; r < cl; ++r) {
                const uint32_t* rh = cl > 1 ? cluster.map_shared_rank(hist, r) : hist;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4*>(rh + 8 * lane + 4 * i);
                    h[4 * i] += x.x;
                    h[4 * i + 1] += x.y;
                    h[4 * i + 2] += x.z;
                    h[4 * i + 3] += x.w;
                }
            }
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += static_cast<int>(h[i]);
            int incl = sum;  // of this lane and the later ones
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_down_sync(FULL, incl, m);
                if (lane + m < 32) incl += y;
            }
            int left = need - (incl - sum);  // still needed when this lane's bytes are reached
            if (left > 0 && left <= sum) {
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    const int n = static_cast<int>(h[i]);
                    if (left > 0 && left <= n) {
                        found[0] = 8 * lane + i;
                        found[1] = left;
                        found[2] = n;
                    }
                    left -= n;
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(found[0]);
        need = found[1];
        whole = need == found[2];
        if (whole || shift == 0) break;
        shift -= 8;
    }
    const uint32_t lo = prefix << shift;  // the smallest key with the prefix
    // exclusive prefix of v over the block's warps, and the block's sum (after a barrier)
    auto over_warps = [&](const int* w, int& before, int& sum) {
        const int v = lane < kWarpsE ? w[lane] : 0;
        before = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < warp ? v : 0)));
        sum = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(v)));
    };
    // ---- ties: the first `need` keys equal to lo, by row ----
    int ties_before = 0, sum;
    if (!whole) {
        int n = 0;
        for (int t0 = w0; t0 < w1; t0 += 32) {
            const int t = t0 + lane;
            n += __popc(__ballot_sync(FULL, t < w1 && keys[t] == lo));
        }
        if (lane == 0) wsum[warp] = n;
        __syncthreads();
        over_warps(wsum, ties_before, sum);
        if (cl > 1) {
            if (tid == 0) sh.ties = sum;
            meet();
            for (int r = 0; r < rank; ++r) ties_before += *cluster.map_shared_rank(&sh.ties, r);
        } else {
            __syncthreads();  // wsum is written again below
        }
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
        int total, sum2;
        over_warps(wsum, holes, sum);
        over_warps(wsum2, movers, sum2);
        total = sum;
        if (cl > 1) {
            if (tid == 0) {
                sh.holes = sum;
                sh.movers = sum2;
            }
            meet();
            total = 0;
            for (int r = 0; r < cl; ++r) {
                const int h = *cluster.map_shared_rank(&sh.holes, r), m = *cluster.map_shared_rank(&sh.movers, r);
                total += h;
                if (r < rank) {
                    holes += h;
                    movers += m;
                }
            }
        }
        if (rank == 0 && tid == 0) sh.list_base = total ? atomicAdd(p.count, static_cast<uint32_t>(total)) : 0u;
        meet();
    }
    int2* list = p.moves + (cl > 1 ? *cluster.map_shared_rank(&sh.list_base, 0) : sh.list_base);
    if (cl > 1) cluster.barrier_arrive();  // (no block's shared memory is read past this point)
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
    if (cl > 1) cluster.barrier_wait();
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
    constexpr int U = 4;
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int W = gridDim.x * (kMoveThreads / 32), w = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    const int M = static_cast<int>(__ldcg(p.count));
    // a row's K and V as 16-byte words, consecutive lanes along one row
    const int words = p.row_bytes >> 4;  // a power of two
    const int shift = 31 - __clz(2 * words);
    // chunks of neighbouring rows in turn, so that all warps work in the same part of the cache;
    // a call with few moves deals out single rows
    const int rows = M >= W * kMoveRows ? kMoveRows : 1;
    for (long long m0 = static_cast<long long>(w) * rows; m0 < M; m0 += static_cast<long long>(W) * rows) {
        const int n = static_cast<int>(min(static_cast<long long>(rows), M - m0));
        const int2* list = p.moves + m0;
        for (int i = lane; i < n << shift; i += 32 * U) {
            uint4 x[U];
            unsigned char* dst[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = i + 32 * u;
                dst[u] = nullptr;
                if (j < n << shift) {
                    const int2 mv = __ldcg(list + (j >> shift));
                    const int c = j & (2 * words - 1);
                    unsigned char* base = c < words ? p.k_cache : p.v_cache;
                    const int off = (c & (words - 1)) * 16;
                    x[u] = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<long long>(mv.x) * p.row_bytes + off));
                    dst[u] = base + static_cast<long long>(mv.y) * p.row_bytes + off;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (dst[u]) __stcs(reinterpret_cast<uint4*>(dst[u]), x[u]);
        }
        if (lane < n) {
            const int2 mv = __ldcg(list + lane);
            p.acc_out[mv.y] = p.acc[mv.x];
            p.positions_out[mv.y] = p.positions[mv.x];
            if (p.k_scales) {
                p.k_scales[mv.y] = p.k_scales[mv.x];
                p.v_scales[mv.y] = p.v_scales[mv.x];
            }
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

cudaError_t launch_evict(EvictParams p, int sms, cudaStream_t stream) {
    // Blocks per selection: more while the blocks stay within two per SM and each keeps 2048 rows.
    const long long segs = static_cast<long long>(p.B) * p.Hkv;
    int cl = 1;
    while (cl < kMaxCluster && segs * cl * 2 <= 2LL * sms && p.Lmax / (cl * 2) >= 2048) cl *= 2;
    const int per = (p.Lmax + cl - 1) / cl + 32 * kWarpsE;  // a block's rows, its warps' runs rounded up
    p.smem_keys = per < kSmemKeys ? per : kSmemKeys;
    void* args[] = {&p};
    const cudaError_t e = launch_pdl(reinterpret_cast<const void*>(&select_kernel), dim3(static_cast<unsigned>(segs * cl)),
                                     kThreadsE, p.smem_keys * 4, args, stream, cl);
    if (e != cudaSuccess) return e;
    return launch_pdl(reinterpret_cast<const void*>(&move_kernel), dim3(static_cast<unsigned>(sms) * 4), kMoveThreads, 0,
                      args, stream);
}

}  // namespace ftd
