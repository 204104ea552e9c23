// ftd_tables.cu -- block tables and slot maps from request lengths (ftd_build_tables).
//
// Every slot goes from old_b to new_b cached rows.  With ps rows a page it holds
// ceil(old_b / ps) table entries and wants ceil(new_b / ps):
//   the entries that slots give back, F of them in (slot, entry) order, go on top of the free
//   list, and the A entries that slots ask for are taken from its top in slot order.
// So entry a of the asked ones (the pages asked for by the slots before it are a prefix sum)
// is the given-back entry F - 1 - a, or, behind those, free_pages[n_free - 1 - (a - F)], and the
// given-back entries 0 .. F - A - 1 stay on the list, at n_free and on.  A slot is served when all
// pages asked for by it and the slots before it are there (A_b <= n_free + F): slots that ask
// for nothing always are, and no slot overtakes an earlier one.
// Nothing is read that another block writes: table entries in use stay, entries given back keep
// their old value, the part of the list that is read and the part that is written never meet,
// and a new token's page comes from the formula above rather than from the new table entry.
// So the call needs no order among its blocks and the same result comes out every time; only
// the values that may be updated in place (n_free, the lengths) are written by the block that
// arrives last, after every block has read them.
//
// Bound: 8 bytes written per token and per page, so a step's call is launch latency (every block
// scans the lengths, one thread a slot) and a prompt's call is its stores: a thread finds the slot
// of four neighbouring tokens by one search of the offsets in shared memory and stores 16 bytes
// to each map.  Measured on the device: one token for each of 64 slots 5.6 us; 256 prompts, 1 M tokens, 9.3; 1023 slots that begin,
// grow, shrink and end, 2.1 M tokens, 17.9 (17 MB written: the searches' instructions bound it, 58 % of issue).
#include <cuda_runtime.h>

#include "ftd_internal.cuh"
#include "ftd_ops.cuh"

namespace ftd {
namespace {

constexpr int kTabThreads = kMaxBatch;  // one thread a slot in the scans
constexpr int kTabTokens = 4;           // tokens of a thread at a time

// Inclusive sum over the block's threads; total over all of them.  One barrier; warp_sums is this scan's own.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m) v += y;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    long long w = lane < static_cast<int>(blockDim.x) / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, m);
        if (lane >= m) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);  // the warps before this one's
    return v + (warp ? before : 0);
}

// Largest i of [0, n) with first[i] <= x, for first[0] <= x.
template <typename V>
__device__ __forceinline__ int last_at_most(const V* first, int n, V x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The map's elements, N neighbours to a thread.  A warp has a run of its own, so the slot and the page of the last round
// mostly are this one's too.  page_of(s, e) is the page of entry e of slot s.
template <int N, typename PageOf>
__device__ __forceinline__ void write_map(const TablesParams& p, long long warp, long long warps, long long tokens, const int* start,
                                          const long long* first, PageOf page_of) {
    constexpr int kRound = 32 * N;
    const int mask = (1 << p.page_shift) - 1;
    const long long rounds = (p.cap + kRound - 1) / kRound, each = (rounds + warps - 1) / warps;
    const long long end = min(p.cap, (warp + 1) * each * kRound);
    int s = -1, entry = -1, page = 0;
#pragma unroll 1
    for (long long t0 = warp * each * kRound + (threadIdx.x & 31) * N; t0 < end; t0 += kRound) {
        int at[N], ps[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const long long t = t0 + i;
            at[i] = -1;
            ps[i] = 0;
            if (t >= tokens) continue;
            if (s < 0 || first[s + 1] <= t) {
                const int from = s + 1;  // (first[from] <= t)
                s = from + last_at_most(first + from, p.B + 1 - from, t);
                entry = -1;
            }
            const int pos = start[s] + static_cast<int>(t - first[s]);
            ps[i] = pos;
            if (!p.block_table) {
                at[i] = s * p.Lmax + pos;
            } else {
                const int e = pos >> p.page_shift;
                if (e != entry) {
                    entry = e;
                    page = page_of(s, e);
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(p.err, kErrBadPage);
                        page = -1;
                    }
                }
                if (page >= 0) at[i] = (page << p.page_shift) + (pos & mask);
            }
        }
        if (N == 4 && t0 + N <= p.cap) {
            if (p.slots) *reinterpret_cast<int4*>(p.slots + t0) = make_int4(at[0], at[1 % N], at[2 % N], at[3 % N]);
            if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(ps[0], ps[1 % N], ps[2 % N], ps[3 % N]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (t0 + i >= p.cap) break;
                if (p.slots) p.slots[t0 + i] = at[i];
                if (p.positions) p.positions[t0 + i] = ps[i];
            }
        }
    }
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
    __shared__ int asked[kMaxBatch];      // pages asked for by the slots before
    __shared__ int back[kMaxBatch];       // pages given back by the slots before
    __shared__ int held[kMaxBatch];       // entries a slot holds before the call
    __shared__ int want[kMaxBatch];       // and after it
    __shared__ int start[kMaxBatch];      // rows before the call
    __shared__ long long first[kMaxBatch + 1];  // new tokens of the slots before
    __shared__ long long page_sums[32], token_sums[32];
    __shared__ int s_grow, s_last;
    const int b = threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    if (b == 0) s_grow = 0;

    // ---- one thread a slot: pages asked for and given back ----
    const bool slot = b < p.B;
    const int old_raw = slot ? __ldcg(p.old_lens + b) : 0, new_raw = slot ? __ldcg(p.new_lens + b) : 0;
    const int free_raw = p.block_table ? __ldcg(p.n_free) : 0;
    const bool fits = old_raw <= p.Lmax && new_raw <= p.Lmax;
    const int L0 = fits ? max(old_raw, 0) : 0, L1 = fits ? max(new_raw, 0) : 0;
    const int ps1 = (1 << p.page_shift) - 1;
    const int h = p.block_table ? static_cast<int>((static_cast<long long>(L0) + ps1) >> p.page_shift) : 0;
    int w = p.block_table ? static_cast<int>((static_cast<long long>(L1) + ps1) >> p.page_shift) : 0;
    const int grow = max(0, w - h), give = max(0, h - w);
    // (both sums in one scan: a slot's pages and a call's fit 31 bits)
    long long both;
    const long long ends = block_scan(static_cast<long long>(grow) << 32 | give, page_sums, both);
    const int a_end = static_cast<int>(ends >> 32), f_end = static_cast<int>(ends), F = static_cast<int>(both);
    const int n_free = min(max(free_raw, 0), p.num_pages);
    const bool bad = free_raw != n_free;
    const bool served = fits && (grow == 0 || a_end <= static_cast<long long>(n_free) + F);
    if (grow > 0 && served) atomicMax(&s_grow, a_end);
    if (!served) w = h;
    long long tokens;
    const long long t_end = block_scan(served ? max(0, L1 - L0) : 0, token_sums, tokens);
    if (slot) {
        asked[b] = a_end - grow;
        back[b] = f_end - give;
        held[b] = h;
        want[b] = w;
        start[b] = L0;
        first[b + 1] = t_end;
    }
    if (b == 0) first[0] = 0;
    __syncthreads();
    const int A = s_grow;

    // ---- what may be updated in place: by the last block to have read it ----
    if (b == 0) {
        s_last = arrive_acq_rel(p.count, 1u) == gridDim.x - 1;
        if (s_last) *p.count = 0u;
    }
    __syncthreads();
    if (s_last) {
        if (slot) {
            p.served[b] = served ? new_raw : old_raw;
            if (p.offsets) p.offsets[b + 1] = static_cast<int>(min(t_end, static_cast<long long>(INT32_MAX)));
            if (!fits) atomicOr(p.err, kErrSeqOverflow);
        }
        if (b == 0) {
            if (p.offsets) p.offsets[0] = 0;
            if (tokens > (p.slots || p.positions ? p.cap : static_cast<long long>(INT32_MAX))) atomicOr(p.err, kErrSeqOverflow);
            if (p.block_table) {
                const long long left = static_cast<long long>(n_free) + F - A;
                if (bad || left > p.num_pages) atomicOr(p.err, kErrBadPage);
                *p.n_free_out = static_cast<int>(min(left, static_cast<long long>(p.num_pages)));
            }
        }
    }

    // entry f of those given back, and the page that asked entry a gets
    auto given = [&](int f) -> int {
        const int s = last_at_most(back, p.B, f);
        return __ldcg(p.block_table + static_cast<size_t>(s) * p.per + want[s] + (f - back[s]));
    };
    auto page_for = [&](int a) -> int { return a < F ? given(F - 1 - a) : __ldcg(p.free_pages + n_free - 1 - (a - F)); };
    auto page_of = [&](int s, int e) -> int {
        return e < held[s] ? __ldcg(p.block_table + static_cast<size_t>(s) * p.per + e) : page_for(asked[s] + (e - held[s]));
    };
    const long long tid = static_cast<long long>(blockIdx.x) * blockDim.x + b;
    const long long threads = static_cast<long long>(gridDim.x) * blockDim.x;

    // ---- pages that change hands ----
    if (p.block_table) {
        // (the last threads first: the first ones have the map's first tokens)
        for (long long a = threads - 1 - tid; a < A; a += threads) {
            const int page = page_for(static_cast<int>(a));
            const int s = last_at_most(asked, p.B, static_cast<int>(a));
            if (page < 0 || page >= p.num_pages) atomicOr(p.err, kErrBadPage);
            p.block_table[static_cast<size_t>(s) * p.per + held[s] + (static_cast<int>(a) - asked[s])] = page;
        }
        const int left = F - A;
        for (long long f = tid; f < left && n_free + f < p.num_pages; f += threads) {
            const int page = given(static_cast<int>(f));
            if (page < 0 || page >= p.num_pages) atomicOr(p.err, kErrBadPage);
            p.free_pages[n_free + f] = page;
        }
    }

    // ---- the slot map: new tokens packed in slot order, -1 behind them ----
    if (!p.slots && !p.positions) return;
    if (p.vec && p.cap > threads) write_map<kTabTokens>(p, tid >> 5, threads >> 5, tokens, start, first, page_of);
    else write_map<1>(p, tid >> 5, threads >> 5, tokens, start, first, page_of);
}

}  // namespace

cudaError_t launch_tables(TablesParams p, int sms, cudaStream_t stream) {
    // A thread a slot, 256 at the least; as many blocks as give each thread four tokens (a call without maps: four
    // entries), 1024 threads an SM at the most.
    const int threads = p.B <= 256 ? 256 : p.B <= 512 ? 512 : kTabThreads;
    const long long per_block = static_cast<long long>(threads) * kTabTokens, most = static_cast<long long>(sms) * (kTabThreads / threads);
    const long long items = p.slots || p.positions ? p.cap : static_cast<long long>(p.B) * p.per;
    const long long blocks = (items + per_block - 1) / per_block;
    const dim3 grid(static_cast<unsigned>(blocks < 1 ? 1 : blocks < most ? blocks : most));
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(&tables_kernel), grid, threads, 0, args, stream);
}

}  // namespace ftd
