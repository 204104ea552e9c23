// ftd_evict.cu -- eviction from the cache by accumulated attention weight
// (ftd_cache_evict): a selection and a move kernel.
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
// (ranks by ballots, warp, block and cluster prefixes).  A cluster with few moves, as when
// a cache is kept at its budget from step to step, makes them itself; else it appends them
// to the call's list (one atomic add reserves its part; the list's order varies, its
// moves are independent).
// move_kernel deals the list out to all warps in chunks of 2 KB, so that ragged slots
// do not leave SMs idle, and writes the new lengths, which may overwrite the old ones: every
// cluster has read them by then.
//
// Bound: 8 bytes per position for the selection, then the moved rows, read and written.
// Measured (a graph on one cache; a stream over three caches in turn): one row over in each of 8 x 32 heads of
// 2049 rows 9.2 us, 9.5 (launches, the selection's chain of barriers and two dependent reads of memory); 32
// ragged slots of 40 heads cut to 2048 rows 129 us, 133, of which the moves take about 110 at 5.6 TB/s; 4 x 8
// heads of 65536 INT8 rows cut to 8192 49 us, 56, half of it the selection, half 128-byte rows gathered
// and scattered.
// With 4 KB a warp in flight the moves took 15 % longer, with 512 threads three times an SM 12 %:
// more reads and writes in flight at once than that slow one another down.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ftd_ops.cuh"

namespace cg = cooperative_groups;

namespace ftd {
namespace {

constexpr int kThreadsE = 512;
constexpr int kWarpsE = kThreadsE / 32;
constexpr int kMaxCluster = 8;
constexpr int kSmemKeys = 48 * 1024;  // keys of a block that fit shared memory (192 KB)
constexpr int kLocalMoves = kMaxLocalMoves / kMaxCluster;  // moves per block that a cluster makes itself
constexpr int kMoveThreads = 256;
constexpr int kMoveU = 4;                 // 16-byte words a lane has in flight: 2 KB a warp

// Cache row of position index t, -1 behind a bad page (rows are below 2^31).
__device__ __forceinline__ int evict_row(const EvictParams& p, int b, int kvh, int t) {
    if (!p.block_table) return (b * p.Hkv + kvh) * p.Lmax + t;
    const int page = p.block_table[static_cast<size_t>(b) * p.pages_per_seq + (t >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) return -1;
    return ((page * p.Hkv + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// Unsigned key in the order of the weights (NaN below every number), all below ~0u.  The two zeros are
// equal weights, which go by their rows, so they share a key: -0 + 0 is +0, other sums are w.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Copies n rows (n * the words of a row at most 32 * kMoveU) of K and V and their plane entries, by
// one warp; lane m < n holds the m-th move.
__device__ __forceinline__ void copy_rows(const EvictParams& p, int2 mv, int n, int lane) {
    const int words = p.row_bytes >> 4;  // 16-byte words of a row, a power of two
    const int shift = 31 - __clz(2 * words);
    uint4 x[kMoveU];
    float a = 0.f, ks = 0.f, vs = 0.f;
    int ps = 0;
    if (lane < n) {
        a = p.acc[mv.x];
        ps = p.positions[mv.x];
        if (p.k_scales) {
            ks = p.k_scales[mv.x];
            vs = p.v_scales[mv.x];
        }
    }
    // word j of the chunk: K then V of row j >> shift, consecutive lanes along one row
    auto place = [&](int j, int row) {
        const int c = j & (2 * words - 1);
        return (c < words ? p.k_cache : p.v_cache) + static_cast<long long>(row) * p.row_bytes + (c & (words - 1)) * 16;
    };
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
        const int j = lane + 32 * u;
        const int src = __shfl_sync(0xffffffffu, mv.x, min(j >> shift, 31));
        if (j >> shift < n) x[u] = __ldcs(reinterpret_cast<const uint4*>(place(j, src)));
    }
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
        const int j = lane + 32 * u;
        const int dst = __shfl_sync(0xffffffffu, mv.y, min(j >> shift, 31));
        if (j >> shift < n) __stcs(reinterpret_cast<uint4*>(place(j, dst)), x[u]);
    }
    if (lane < n) {
        p.acc_out[mv.y] = a;
        p.positions_out[mv.y] = ps;
        if (p.k_scales) {
            p.k_scales[mv.y] = ks;
            p.v_scales[mv.y] = vs;
        }
    }
}

// What the blocks of a cluster read of each other.
struct alignas(16) Shared {
    uint32_t hist[2][256];
    int ties, holes, movers;  // of this block
    int bad;
    uint32_t list_base;       // of the cluster (block 0's)
};

// MULTI: clusters of several blocks.
template <bool MULTI>
__device__ __forceinline__ void evict_segment(const EvictParams& p, uint32_t* skeys, int seg, int rank, int cl) {
    __shared__ Shared sh;
    __shared__ __align__(16) uint32_t tot[256];
    __shared__ int2 few[kLocalMoves];
    __shared__ int wsum[kWarpsE], wsum2[kWarpsE];
    __shared__ int found[3];  // digit, rows needed of it, keys with it
    constexpr unsigned FULL = 0xffffffffu;
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    // every thread of the cluster (or, alone, of the block) has written what it shares
    auto meet = [&]() {
        if constexpr (MULTI) cluster.sync();
        else __syncthreads();
    };
    auto peer = [&](auto* x, int r) {
        if constexpr (MULTI) return cluster.map_shared_rank(x, r);
        return x;
    };
    // lane r < cl: block r's x (every lane loads at once; the others get 0)
    auto of_peers = [&](int* x) { return lane < cl ? *peer(x, lane) : 0; };
    if (tid < 256) sh.hist[0][tid] = 0u;
    if (tid == 0) sh.bad = 0;
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
                const int row = evict_row(p, b, kvh, t);
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
    const int c0 = min(L, rank * kWarpsE * S);  // the block's first row
    const int w0 = min(L, c0 + warp * S), w1 = min(L, w0 + S);
    // keys[t - c0] for row t
    uint32_t* keys = S * kWarpsE <= p.smem_keys ? skeys : p.keys + static_cast<size_t>(seg) * p.Lmax + c0;
    const long long fresh = static_cast<long long>(__ldcg(p.next_pos + b)) - p.recent;
    bool bad = false;
    constexpr int U = MULTI ? 8 : 4;  // rows a lane has in flight
    for (int t0 = w0 + lane; t0 < w1; t0 += 32 * U) {
        float a[U];
        int ps[U], row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) row[u] = t0 + 32 * u < w1 ? evict_row(p, b, kvh, t0 + 32 * u) : -2;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bad |= row[u] == -1;
            a[u] = row[u] >= 0 ? p.acc[row[u]] : 0.f;
            ps[u] = row[u] >= 0 ? p.positions[row[u]] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + 32 * u;
            if (row[u] == -2) continue;
            keys[t - c0] = ps[u] < p.sinks || ps[u] >= fresh ? 0xffffffffu : weight_key(a[u]);
            // planes apart: entries below the budget go over as they are, and the moves then
            // overwrite those of the rows that go
            if (row[u] >= 0 && t < p.budget) {
                if (apart) p.acc_out[row[u]] = a[u];
                if (papart) p.positions_out[row[u]] = ps[u];
            }
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
#pragma unroll 4
        for (int t = w0 + lane; t < w1; t += 32) {
            const uint32_t k = keys[t - c0];
            if (round == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        meet();
        if (round == 0) {
            if (__any_sync(FULL, of_peers(&sh.bad) != 0)) {  // a page of this slot is bad: its rows are left where they are
                if (tid == 0 && rank == 0) atomicOr(p.err, kErrBadPage);
                meet();  // no block leaves while another reads its flag
                return;
            }
        }
        if (tid < 256) {
            sh.hist[(round + 1) & 1][tid] = 0u;  // (read last before this meeting)
            if constexpr (MULTI) {
                uint32_t n = 0u;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) n += r < cl ? *peer(hist + tid, r) : 0u;
                tot[tid] = n;
            }
        }
        if constexpr (MULTI) __syncthreads();
        if (warp == 0) {
            // lane owns bytes 8 lane .. 8 lane + 7; keys above them: those of the later lanes
            const uint4* ht = reinterpret_cast<const uint4*>((MULTI ? tot : hist) + 8 * lane);
            const uint4 h0 = ht[0], h1 = ht[1];
            const uint32_t h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
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
    // exclusive prefix of w over the block's warps, and the block's sum (after a barrier)
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
            n += __popc(__ballot_sync(FULL, t < w1 && keys[t - c0] == lo));
        }
        if (lane == 0) wsum[warp] = n;
        __syncthreads();
        over_warps(wsum, ties_before, sum);
        if (MULTI && tid == 0) sh.ties = sum;
        meet();  // (and wsum may be written again)
        if constexpr (MULTI) {
            const int v = of_peers(&sh.ties);
            ties_before += static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < rank ? v : 0)));
        }
    }
    // Calls f(t, ev, nb) for the warp's rows, 32 at a time in order: nb of the 32 lie below the budget,
    // and ev says whether row t is a hole (below, not kept) or has to move (kept, not below).
    auto for_rows = [&](auto all, auto&& f) {
        int ties = ties_before;
#pragma unroll 4
        for (int t0 = w0; t0 < w1; t0 += 32) {
            const int t = t0 + lane;
            const bool in = t < w1;
            const uint32_t k = in ? keys[t - c0] : 0u;
            bool kept = k >= lo;
            if constexpr (!decltype(all)::value) {
                const bool tie = in && k == lo;
                const unsigned m = __ballot_sync(FULL, tie);
                if (tie) kept = ties + __popc(m & ((1u << lane) - 1u)) < need;
                ties += __popc(m);
            }
            const int nb = p.budget - t0;
            f(t, in && kept == (lane >= nb), nb);
        }
    };
    // ---- holes below the budget and kept rows from it on: counted, then listed ----
    int holes = 0, movers = 0;
    auto count = [&](int, bool ev, int nb) {
        holes += ev && lane < nb;
        movers += ev && lane >= nb;
    };
    if (whole) for_rows(std::true_type{}, count);
    else for_rows(std::false_type{}, count);
    holes = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(holes)));
    movers = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(movers)));
    if (lane == 0) {
        wsum[warp] = holes;
        wsum2[warp] = movers;
    }
    __syncthreads();
    int total, sum2;
    over_warps(wsum, holes, total);
    over_warps(wsum2, movers, sum2);
    if constexpr (MULTI) {
        if (tid == 0) {
            sh.holes = total;
            sh.movers = sum2;
        }
        cluster.sync();
        const int h = of_peers(&sh.holes), m = of_peers(&sh.movers);
        total = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(h)));
        holes += static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < rank ? h : 0)));
        movers += static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(lane < rank ? m : 0)));
    }
    // the moves' place: shared by the whole call, or, for few, this cluster's own
    const bool local = total <= kLocalMoves * cl;
    int2* list = MULTI ? p.local_moves + static_cast<size_t>(seg) * kMaxLocalMoves : few;
    if (!local) {
        if (rank == 0 && tid == 0) sh.list_base = atomicAdd(p.count, static_cast<uint32_t>(total));
        meet();
        list = p.moves + *peer(&sh.list_base, 0);
    }
    auto enter = [&](int t, bool ev, int nb) {
        const unsigned m = __ballot_sync(FULL, ev);
        if (!m) return;
        const unsigned low = nb >= 32 ? FULL : nb <= 0 ? 0u : (1u << nb) - 1u;  // the rows below the budget
        const unsigned before = (1u << lane) - 1u;
        if (ev) {
            const int row = evict_row(p, b, kvh, t);
            if (lane < nb) list[holes + __popc(m & low & before)].y = row;
            else list[movers + __popc(m & ~low & before)].x = row;
        }
        holes += __popc(m & low);
        movers += __popc(m & ~low);
    };
    if (whole) for_rows(std::true_type{}, enter);
    else for_rows(std::false_type{}, enter);
    meet();  // the list is complete (and no block's shared memory is read past this point)
    if (local)
        for (int m = rank * kWarpsE + warp; m < total; m += cl * kWarpsE) copy_rows(p, MULTI ? __ldcg(list + m) : list[m], 1, lane);
}

template <bool MULTI>
__global__ void __launch_bounds__(kThreadsE, 2) select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t skeys[];
    int cl = 1, rank = 0;
    if constexpr (MULTI) {
        const cg::cluster_group cluster = cg::this_cluster();
        cl = static_cast<int>(cluster.num_blocks());
        rank = static_cast<int>(cluster.block_rank());
    }
    grid_dep_wait();
    grid_dep_launch();
    evict_segment<MULTI>(p, skeys, static_cast<int>(blockIdx.x) / cl, rank, cl);
}

__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int W = gridDim.x * (kMoveThreads / 32), w = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    const int M = static_cast<int>(__ldcg(p.count));
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += kMoveThreads) {
            const int L = __ldcg(p.seq_lens + b);
            p.new_lens[b] = (L > p.budget && L <= p.Lmax) ? p.budget : L;
        }
    if (M == 0) return;
    // Chunks of neighbouring rows in turn, so that all warps work in the same part of the cache; the
    // next chunk's moves are loaded while this one's rows are copied.
    const int rows = 32 * kMoveU * 8 / p.row_bytes;  // 2 KB of K and V (2 to 16 rows)
    const long long step = static_cast<long long>(W) * rows;
    long long m0 = static_cast<long long>(w) * rows;
    int2 mv = make_int2(0, 0);
    if (m0 + lane < M && lane < rows) mv = __ldcg(p.moves + m0 + lane);
    for (; m0 < M; m0 += step) {
        int2 next = make_int2(0, 0);
        if (m0 + step + lane < M && lane < rows) next = __ldcg(p.moves + m0 + step + lane);
        copy_rows(p, mv, static_cast<int>(min(static_cast<long long>(rows), M - m0)), lane);
        mv = next;
    }
    // the last block to finish leaves the counters at zero for the next call
    __syncthreads();
    if (threadIdx.x == 0 && arrive_acq_rel(p.count + 1, 1u) == gridDim.x - 1) {
        p.count[0] = 0u;
        p.count[1] = 0u;
    }
}

}  // namespace

cudaError_t setup_evict() {
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&select_kernel<false>),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKeys * 4);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&select_kernel<true>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKeys * 4);
    return e;
}

cudaError_t launch_evict(EvictParams p, int sms, cudaStream_t stream) {
    // Blocks per selection: more while the blocks stay within two per SM and each keeps 2048 rows.
    const long long segs = static_cast<long long>(p.B) * p.Hkv;
    int cl = 1;
    while (cl < kMaxCluster && segs * cl * 2 <= 2LL * sms && p.Lmax / (cl * 2) >= 2048) cl *= 2;
    const int per = (p.Lmax + cl - 1) / cl + 32 * kWarpsE;  // a block's rows, its warps' runs rounded up
    p.smem_keys = per < kSmemKeys ? per : kSmemKeys;
    const void* fn = cl > 1 ? reinterpret_cast<const void*>(&select_kernel<true>)
                            : reinterpret_cast<const void*>(&select_kernel<false>);
    void* args[] = {&p};
    const cudaError_t e = launch_pdl(fn, dim3(static_cast<unsigned>(segs * cl)), kThreadsE, p.smem_keys * 4, args, stream, cl);
    if (e != cudaSuccess) return e;
    return launch_pdl(reinterpret_cast<const void*>(&move_kernel), dim3(static_cast<unsigned>(sms) * 4), kMoveThreads, 0,
                      args, stream);
}

}  // namespace ftd
