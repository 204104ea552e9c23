// ftd_prefix_tc.cu -- attention to a shared prefix on the tensor cores (fp16 and bf16 caches;
// ftd_prefix.cuh has the mathematics, the cut into work and the layout of the partials).
//
// With every slot's rows together the products are dense: per tile of 128 prefix rows and 128 query rows
//   S [128 x 128] = Q [128 x D] . K^T          (both K-major in shared memory, S in TMEM)
//   O [128 x D]  += P [128 x 128] . V          (P from TMEM, V MN-major in shared memory, O in TMEM)
// A block runs two such streams at a time, so that one's softmax runs under the other's products:
// the two halves of 256 query rows over the same tiles, or, for a row block of at most 128 rows, the even and
// the odd tiles of the same rows.  The tensor cores' order is S0 S1 | PV0 S0' PV1 S1' | ...: P of a stream lies over its S
// (a thread has read a score before it writes the weight there), and S' is issued behind the PV that reads P.
// TMEM is full: two S of 128 columns and two O of D.
//
// A softmax thread owns one query row: no exchange between threads.  It takes the weights against
// its running reference m while it reads the scores, packs them, and only when a score passes m by
// more than 2^8 (the first tile always) moves m, takes the weights again and rescales its row of O; the
// product of the tile before has ended by then, since the score product behind it has.
//
// PAIR: q and the weights as pairs of 16-bit numbers, hi and lo, two products each (about 16 mantissa bits with
// bf16, 22 with fp16): for fp32 out, and where q is no 16-bit number of the cache's type (a bias, another
// type).  Both streams then share one row block of 128.
//
// Roles (384 threads, one block an SM): warp 0 copies K and V tiles (TMA, a ring of whole tiles K0 V0 K1
// V1 ..); warp 1 allocates TMEM, zeroes the V rows behind the prefix's seen end and issues the products;
// warps 4-7 and 8-11 are the two streams' softmax, q load and partials (warps 2 and 3 idle: a warp reaches
// the TMEM lanes of its number mod 4).
#include <cuda_runtime.h>

#include "ftd_internal.cuh"
#include "ftd_prefix_tc.cuh"

namespace ftd {
namespace ptc {

constexpr int TK = 128;   // prefix rows of a tile, and query rows of a stream
constexpr int KB = tc::KB;
constexpr int kThreads = 384;
constexpr int kMostBlocks = 256;  // row blocks of a kv head (room of the plan)
constexpr float kNone = -1e30f;   // reference of a row that has seen nothing

template <int D>
struct Layout {
    static constexpr int TILE = D / 64 * KB;
    static constexpr int NSLOT = D == 128 ? 5 : 8;
    static constexpr int OFF_Q = NSLOT * TILE;  // two streams' q, or hi and lo of one
    static constexpr int OFF_MISC = OFF_Q + 2 * TILE;
    static constexpr int NBARS = 2 * NSLOT + 8;
    static constexpr int OFF_FIRST = OFF_MISC + NBARS * 8 + 16;
    static constexpr int SMEM = OFF_FIRST + (kMostBlocks + 1) * 4 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
};

// pairs of fp32 in one register pair
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <typename CT>
__device__ __forceinline__ uint32_t pack_ct(float a, float b) {
    uint32_t r;
    if constexpr (std::is_same_v<CT, __nv_bfloat16>) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&r, &h, 4);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        memcpy(&r, &h, 4);
    }
    return r;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Eight elements of a q or bias row from element i on, as floats (16-byte loads where the base allows).
__device__ __forceinline__ void load8(const void* base, int dt, size_t i, bool vec, float (&x)[8]) {
    if (!vec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ld_qkv(base, dt, i + e);
    } else if (dt == kF32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
        const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i + 4));
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(base) + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = raw_to_f((e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu, dt);
    }
}

template <typename CT, int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const PrefixParams p) {
    using LY = Layout<D>;
    constexpr int NSLOT = LY::NSLOT, TILE = LY::TILE;
    constexpr bool BF = std::is_same_v<CT, __nv_bfloat16>;
    constexpr unsigned FULL = 0xffffffffu;
    enum : int { kFull = 0, kEmpty = NSLOT, kSFull = 2 * NSLOT, kPFull = kSFull + 2, kOFull = kSFull + 4, kStart = kSFull + 6, kDrain = kSFull + 7 };
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::OFF_MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + LY::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* first = reinterpret_cast<int*>(smem + LY::OFF_FIRST);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    if (tid == 0) {
        for (int i = 0; i < LY::NBARS; ++i) mbar_init(bar(i), i >= kPFull && i < kPFull + 2 ? 4 : i == kStart ? 8 : 1);
        *abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_mbar_init();
    tc::tc_fence_before();
    // Runs beside the step's last blocks (see the CUDA-core kernel).
    build_prefix_plan(p, first, TK);
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const PrefixSplit sp(p, first);
    if (blockIdx.x == 0) write_seg_info(p, first, sp);
    const int w = blockIdx.x;
    const long long u_begin = sp.begin(w), u_end = sp.begin(w + 1);
    // pieces: (kv head, row block, tiles); the roles walk them in step
    struct Piece {
        PrefixCursor c;
        int nt;
        bool twice;
    };
    auto piece_at = [&](long long u) {
        Piece x;
        x.c = prefix_locate(u, first, p.row_blocks);
        x.nt = static_cast<int>(min(static_cast<long long>(x.c.nt - x.c.tile), u_end - u));
        x.twice = prefix_twice(p, x.c.rb);
        return x;
    };
    // tiles of stream s in a piece, and the piece's tile that is its j-th
    auto tiles_of = [](const Piece& x, int s) { return x.twice ? (x.nt - s + 1) / 2 : x.nt; };
    auto tile_of = [](const Piece& x, int s, int j) { return x.twice ? 2 * j + s : j; };

    int issued = 0;  // producer: tiles K and V copied (or withheld)
    const bool withhold = p.stall && blockIdx.x == 0;  // test hook: block 0's first copy never comes
    if (u_begin < u_end) {
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            if (lane == 0) {
                bool ok = true;
                for (long long u = u_begin; u < u_end && ok;) {
                    const Piece x = piece_at(u);
                    for (int i = 0; i < 2 * x.nt && ok; ++i) {
                        const int slot = issued % NSLOT;
                        if (issued >= NSLOT)
                            ok = tc::wait_or_abort(bar(kEmpty + slot), ((issued / NSLOT) - 1) & 1, p.err, abort_flag, p.wait_cycles);
                        if (!ok) break;
                        if (!(withhold && issued == 0)) {
                            long long row = prefix_row(p, x.c.h, (x.c.tile + (i >> 1)) * TK);
                            if (row < 0) {
                                atomicOr(p.err, kErrBadPage);
                                row = 0;
                            }
                            const uint32_t dst = smem_addr(smem + slot * TILE);
                            mbar_arrive_expect_tx(bar(kFull + slot), TILE);
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load(dst + b * KB, (i & 1) ? &tmv : &tmk, 64 * b, static_cast<int>(row), bar(kFull + slot));
                        }
                        ++issued;
                    }
                    u += x.nt;
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ products
            const uint32_t id_s = tc::instr_desc(BF, TK, TK, false), id_o = tc::instr_desc(BF, TK, D, false, true);
            const uint64_t dq0 = tc::smem_desc_sw128(smem_addr(smem + LY::OFF_Q), 16, 1024);
            const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(smem), 16, 1024);
            const uint64_t dv0 = tc::smem_desc_sw128(smem_addr(smem), KB, 1024);
            int base = 0, pieces = 0;  // tiles copied for the pieces before; pieces begun
            int np[2] = {0, 0};        // products P.V issued per stream
            bool ok = true;
            auto wait = [&](int b, int parity) {
                return __all_sync(FULL, tc::wait_or_abort(bar(b), parity, p.err, abort_flag, p.wait_cycles));
            };
            // the scores of stream s's j-th tile
            auto scores = [&](const Piece& x, int s, int j) -> bool {
                const int item = 2 * (base + tile_of(x, s, j)), slot = item % NSLOT;
                if (!wait(kFull + slot, (item / NSLOT) & 1)) return false;
                if (lane == 0) {
                    tc::tc_fence_after();
                    const uint64_t ka = dk0 + static_cast<uint32_t>(slot * (TILE >> 4));
                    const uint64_t qa = dq0 + static_cast<uint32_t>((PAIR ? 0 : s) * (TILE >> 4));
#pragma unroll
                    for (int kq = 0; kq < D / 16; ++kq) {
                        const uint32_t o = ((kq >> 2) * KB + (kq & 3) * 32) >> 4;
                        tc::mma_f16(tmem + s * TK, qa + o, ka + o, id_s, kq > 0);
                        if constexpr (PAIR) tc::mma_f16(tmem + s * TK, qa + (TILE >> 4) + o, ka + o, id_s, true);
                    }
                    tc::mma_commit(bar(kSFull + s));
                    if (x.twice || s == 1) tc::mma_commit(bar(kEmpty + slot));
                }
                __syncwarp();
                return true;
            };
            for (long long u = u_begin; u < u_end && ok;) {
                const Piece x = piece_at(u);
                const int seen = prefix_block_seen(p, x.c.rb, lane);
                ok = wait(kStart, pieces & 1);  // q is there, O and S of the piece before are read
                ++pieces;
                for (int s = 0; s < 2 && ok; ++s)
                    if (tiles_of(x, s) > 0) ok = scores(x, s, 0);
                const int most = tiles_of(x, 0);
                for (int j = 0; j < most && ok; ++j) {
                    for (int s = 0; s < 2 && ok; ++s) {
                        const int n = tiles_of(x, s);
                        if (j >= n) continue;
                        const int t = tile_of(x, s, j), item = 2 * (base + t) + 1, slot = item % NSLOT;
                        ok = wait(kFull + slot, (item / NSLOT) & 1);
                        if (!ok) break;
                        const int valid = seen - (x.c.tile + t) * TK;
                        if (valid < TK && (x.twice || s == 0)) {
                            // rows that no slot of the block sees: zero, so that a weight of zero meets a number
                            unsigned char* v = smem + slot * TILE;
                            const int nz = (TK - valid) * 8;
                            for (int i = lane; i < nz * (D / 64); i += 32)
                                *reinterpret_cast<uint4*>(v + (i / nz) * KB + valid * 128 + (i % nz) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        ok = wait(kPFull + s, np[s] & 1);
                        if (!ok) break;
                        ++np[s];
                        if (lane == 0) {
                            tc::tc_fence_after();
                            const uint64_t vb = dv0 + static_cast<uint32_t>(slot * (TILE >> 4));
#pragma unroll
                            for (int kq = 0; kq < TK / 16; ++kq) {
                                tc::mma_f16_ta(tmem + 2 * TK + s * TK, tmem + s * TK + kq * 8, vb + (kq * 2048 >> 4), id_o, j > 0 || kq > 0);
                                if constexpr (PAIR)
                                    tc::mma_f16_ta(tmem + 2 * TK + s * TK, tmem + s * TK + 64 + kq * 8, vb + (kq * 2048 >> 4), id_o, true);
                            }
                            if (x.twice || s == 1) tc::mma_commit(bar(kEmpty + slot));
                            if (j + 1 == n) tc::mma_commit(bar(kOFull + s));
                        }
                        __syncwarp();
                        if (j + 1 < n) ok = scores(x, s, j + 1);
                    }
                }
                base += x.nt;
                u += x.nt;
            }
            // one last commit: it completes once every product issued above has
            if (lane == 0) tc::mma_commit(bar(kDrain));
            __syncwarp();
        } else if (warp >= 4) {
            // ------------------------------------------------ softmax of one stream
            const int s = (warp >> 2) - 1, r = (warp & 3) * 32 + lane;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t ts = tmem + lanes + s * TK, to = tmem + lanes + 2 * TK + s * TK;
            const bool vec = ((reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.bias)) & 15u) == 0;
            int ns = 0, no[2] = {0, 0};  // score tiles taken; outputs waited for, of both streams
            bool ok = true;
            auto wait = [&](int b, int parity) {
                return __all_sync(FULL, tc::wait_or_abort(bar(b), parity, p.err, abort_flag, p.wait_cycles));
            };
            const float qscale = p.qscale;
            for (long long u = u_begin; u < u_end && ok;) {
                const Piece x = piece_at(u);
                const int n = tiles_of(x, s);
                const int row = x.c.rb * p.block_rows + (x.twice ? r : s * TK + r);
                const bool live = row < p.R;
                // ---- q ----
                {
                    const size_t qi = live ? prefix_q_row(p, x.c.h, row) * D : 0;
                    const size_t bi = live ? static_cast<size_t>(x.c.h * p.group + row % p.group) * D : 0;
                    unsigned char* qs = smem + LY::OFF_Q + (PAIR ? 0 : s * TILE);
                    // (a pair's q is made by both streams, half of the dimensions each)
                    constexpr int DN = PAIR ? D / 2 : D;
#pragma unroll 4
                    for (int c = 0; c < DN / 8; ++c) {
                        const int d = c * 8 + (PAIR ? s * DN : 0);
                        float q[8];
                        load8(p.q, p.qkv_dtype, qi + d, vec, q);
                        if constexpr (PAIR) {
                            if (p.bias) {
                                float b[8];
                                load8(p.bias, p.qkv_dtype, bi + d, vec, b);
#pragma unroll
                                for (int e = 0; e < 8; ++e) q[e] += b[e];
                            }
                        }
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = live ? q[2 * e] : 0.f, b = live ? q[2 * e + 1] : 0.f;
                            if constexpr (PAIR) wide::split_pair<CT>(a, b, hi[e], lo[e]);
                            else hi[e] = pack_ct<CT>(a, b);
                        }
                        *reinterpret_cast<uint4*>(qs + tc::sw128_offset(r, d, TK)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (PAIR)
                            *reinterpret_cast<uint4*>(qs + TILE + tc::sw128_offset(r, d, TK)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kStart));
                }
                const int seen = live ? prefix_seen(p, prefix_slot_of(p, row)) : 0;
                float m = kNone, l = 0.f;
                for (int j = 0; j < n; ++j) {
                    const int lim = seen - (x.c.tile + tile_of(x, s, j)) * TK;  // columns that the row sees
                    ok = wait(kSFull + s, ns & 1);
                    if (!ok) break;
                    ++ns;
                    tc::tc_fence_after();
                    uint32_t hi[TK / 2], lo[PAIR ? TK / 2 : 1];
                    float top, sum;
                    // weights against reference m, their sum and the largest score
                    auto weigh = [&](auto masked, float ref) {
                        const uint64_t sc2 = pack2(qscale, qscale), m2 = pack2(-ref, -ref);
                        uint64_t acc = pack2(0.f, 0.f);
                        top = -INFINITY;
#pragma unroll
                        for (int c = 0; c < TK / 32; ++c) {
                            float v[32];
                            wide::tmem_ld_rows<32>(ts + 32 * c, v);
                            if constexpr (decltype(masked)::value) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (32 * c + e >= lim) v[e] = -INFINITY;
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                top = fmaxf(top, fmaxf(v[e], v[e + 1]));
                                float a, b;
                                unpack2(fma2(pack2(v[e], v[e + 1]), sc2, m2), a, b);
                                a = wide::ex2(a);
                                b = wide::ex2(b);
                                acc = add2(acc, pack2(a, b));
                                if constexpr (PAIR) wide::split_pair<CT>(a, b, hi[16 * c + e / 2], lo[16 * c + e / 2]);
                                else hi[16 * c + e / 2] = pack_ct<CT>(a, b);
                            }
                        }
                        float a, b;
                        unpack2(acc, a, b);
                        sum = a + b;
                    };
                    const bool full = __all_sync(FULL, lim >= TK);
                    if (full) weigh(std::false_type{}, m);
                    else weigh(std::true_type{}, m);
                    if (__any_sync(FULL, top * qscale > m + tc::kRescaleLog2)) {
                        // references move (rows whose score does not pass theirs keep it)
                        const float mn = fmaxf(m, top * qscale), alpha = wide::ex2(m - mn);
                        if (full) weigh(std::false_type{}, mn);
                        else weigh(std::true_type{}, mn);
                        m = mn;
                        l *= alpha;
                        if (j > 0) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                wide::tmem_ld_rows<32>(to + 32 * c, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                                wide::tmem_st16(to + 32 * c, o);
                                wide::tmem_st16(to + 32 * c + 16, o + 16);
                            }
                        }
                    }
                    l += sum;
#pragma unroll
                    for (int c = 0; c < TK / 32; ++c) {
                        tc::tmem_st16(ts + 16 * c, hi + 16 * c);
                        if constexpr (PAIR) tc::tmem_st16(ts + 64 + 16 * c, lo + 16 * c);
                    }
                    wide::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kPFull + s));
                }
                if (!ok) break;
                // ---- the piece's partial ----
                float* slot = p.ws + static_cast<size_t>(x.c.h * p.row_blocks + x.c.rb + w) * prefix_slot_floats(p.slot_rows, D) + s * TK + r;
                __stcg(slot, m);
                __stcg(slot + p.slot_rows, l);
                if (n > 0) {
                    ok = wait(kOFull + s, no[s] & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        wide::tmem_ld_rows<32>(to + 32 * c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) __stcg(slot + static_cast<size_t>(2 + 32 * c + e) * p.slot_rows, o[e]);
                    }
                    tc::tc_fence_before();
                    ++no[s];
                }
                if (tiles_of(x, s ^ 1) > 0) {
                    // the q of a pair, which both streams share, is free when the other's products are done too; and a stream
                    // without a tile must not come to the next piece's start ahead of the other
                    if (PAIR || n == 0) ok = wait(kOFull + (s ^ 1), no[s ^ 1] & 1);
                    ++no[s ^ 1];
                }
                u += x.nt;
            }
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (*abort_flag && warp == 0 && lane == 0) {
        // a bounded wait ran out: wait (long drain limit) for the copies in flight
        for (int i = max(0, issued - NSLOT); i < issued; ++i)
            if (!(withhold && i == 0)) mbar_wait_bounded(bar(kFull + i % NSLOT), (i / NSLOT) & 1, p.err, kDrainLimitCycles);
    }
    if (warp == 1) {
        if (lane == 0 && u_begin < u_end) mbar_wait_bounded(bar(kDrain), 0u, p.err, kDrainLimitCycles);
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
    grid_dep_launch();
    grid_dep_wait();  // the step before has ended when this grid has: the join reads both
}

template <typename CT, int D>
PrefixKernel pick(bool pair) {
    using LY = Layout<D>;
    if (pair) return {reinterpret_cast<const void*>(&prefix_tc_kernel<CT, D, true>), LY::SMEM, kThreads, TK, 2 * TK, true};
    return {reinterpret_cast<const void*>(&prefix_tc_kernel<CT, D, false>), LY::SMEM, kThreads, 2 * TK, 2 * TK, true};
}

}  // namespace ptc

PrefixKernel select_prefix_tc(bool bf16, int D, bool pair) {
    if (bf16) return D == 64 ? ptc::pick<__nv_bfloat16, 64>(pair) : ptc::pick<__nv_bfloat16, 128>(pair);
    return D == 64 ? ptc::pick<__half, 64>(pair) : ptc::pick<__half, 128>(pair);
}

}  // namespace ftd
