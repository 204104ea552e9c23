// ftd_prefix_tc_kernel.cuh -- attention to a shared prefix, and to the slots' own rows beside it, on the
// tensor cores (ftd_prefix.cuh has the mathematics, the cut into work and the layout of the partials).
//
// With every slot's rows together the products over the prefix are dense: per tile of 128 prefix rows and 128 query rows
//   S [128 x 128] = Q [128 x D] . K^T          (both K-major in shared memory, S in TMEM)
//   O [128 x D]  += P [128 x 128] . V          (P from TMEM, V MN-major in shared memory, O in TMEM)
// A block runs two such streams at a time, so that one's softmax runs under the other's products:
// the two halves of 256 query rows over the same tiles, or, for a row block of at most 128 rows, the even and
// the odd tiles of the same rows.  The order of a stream is S | P V, S' | ..: P lies over S
// (a thread has read a score before it writes the weight there), and S' is issued behind the PV that reads P.
// TMEM is full: two S of 128 columns and two O of D.
//
// The slots' own rows run through the same streams, each block taking its share of the prefix's tiles
// and its share of the own ones (odd blocks the own ones first, so that the memory works while other blocks
// compute).  An own segment, a slot's kv head, has a few query rows only (T * group, at most 32); the products over
// them are mostly empty, but even so cost less than a tile's way from memory.  Here each stream walks its own range of tiles, and no stream waits at a segment's end: the next q
// is already in its other buffer, O is read while the next scores are made.  Which own rows come here, and which go by the decode
// step's kernel before, is a rule with both sides measured at ftd_enable_prefix.
//
// A softmax thread owns one query row: no exchange between threads.  It reads its scores once for the largest and once for
// the weights, and only when a score passes its running reference m by more than 2^8 (the first tile always) moves
// m and rescales its row of O; the product of the tile before has ended by then, since the score product
// behind it has.
//
// The weights are pairs of 16-bit numbers, hi and lo, two products each (about 16 mantissa bits with bf16, 22 with fp16),
// whatever the type of out, as in the decode step: single ones made a 16-bit out, whose own rounding is 1.65e-3
// (bf16) or 2.07e-4 (fp16) in the 2-norm, 2.2e-3 to 2.4e-3 and 2.65e-4.  PQ: q too, where it is no 16-bit number of the cache's
// type (a bias, another type).  With PQ both streams share one row block of 128.
//
// I8: codes become 16-bit numbers on the chip, exactly: K's of the type of q (or bf16 where q is a pair), V's bf16. K's scales
// multiply the scores and V's the weights, in the softmax threads (take_tile_i8).  Four warps more read tiles of codes
// straight from memory, one ahead of the ones they convert, in place of the copying warp and of warp 2.  The slots' own
// rows go by the decode step's kernel.
//
// Measured, all launches of a call: 64 70B-shaped slots of two tokens (1024 query rows a kv head) behind 32768 rows, bf16,
// 193 us, 714 TFLOP/s of useful products (with single weights 147); a tile of both streams takes some 6900 cycles (the time over a
// block's tiles), of which its products 1536, the softmax threads the rest (128 ex2 a thread and tile are 2048 cycles of the SM's
// units for two streams).  INT8 for the same shapes: 312 us (with single weights 259, 5800 cycles a tile).
//
// Roles (384 threads, one block an SM): warp 0 copies K and V tiles (TMA, a ring of whole tiles), then writes for the
// join which blocks hold what; warps 1 and 3 issue the products, each of one stream (one warp for both was busy all the
// time with a third of the products that the tensor cores can take: a wait and its loop are about 200 cycles); warp 2 sees to
// tiles that are not whole: it writes the step's new rows into them and into the cache, and zeroes V rows
// that nobody sees, so that a weight of zero meets a number; warps 4-7 and 8-11 are the two streams' softmax,
// partials and q (a warp reaches the TMEM lanes of its number mod 4; on own rows the first warp of a stream has all
// of them, the others fetch the next q).
#pragma once

#include <cuda_runtime.h>

#include "ftd_internal.cuh"
#include "ftd_prefix_tc.cuh"

namespace ftd {
namespace ptc {

constexpr int TK = 128;   // prefix rows of a tile, and query rows of a stream
constexpr int KB = tc::KB;
constexpr int kThreads = 384;
constexpr int kThreadsI8 = 512;  // and four warps that make codes into 16-bit numbers
constexpr int kMostBlocks = 256;  // row blocks of a kv head (room of the plan)
constexpr float kNone = -1e30f;   // reference of a row that has seen nothing

// A block's share of the work: tiles of the prefix; own tiles of its two streams, as which workers, and how many each.
struct Share {
    long long u_begin, u_end, own_at[2];
    int own_v[2], own_n[2];
};

template <int D, bool I8>
struct Layout {
    static constexpr int TILE = D / 64 * KB;
    // K slots, then V slots: a K tile is free when its scores are made, a V tile, which waits for the softmax, later
    // (one ring of five, in which a K tile's place can be that of an earlier V tile, kept the next scores waiting)
    static constexpr int NK = D == 128 ? 2 : 4, NV = D == 64 ? 4 : I8 ? 2 : 3, NSLOT = NK + NV;
    // INT8: the scales of a tile's rows (K, V), free when the tile's V slot is; a K tile is made behind the V tile before it, so
    // one buffer more than V slots never waits.  Behind them 128 ones.
    static constexpr int NSC = I8 ? NV + 1 : 0;
    // Two streams' q, or hi and lo of one; on own rows two buffers a stream.  It lies before the ring: a product over
    // a few own rows reads 128 all the same, what lies behind them (its rows of S are never looked at).
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OWN_BOX = kMostOwnRows * 128;  // 64 columns of an own q
    static constexpr int OWN_LO = TILE / 4;             // its lo half
    static constexpr int OWN_BUF = TILE / 2;            // the other buffer
    static constexpr int OFF_MISC = OFF_RING + NSLOT * TILE;
    static constexpr int NBARS = 3 * NSLOT + 11;
    static constexpr int OFF_FIRST = OFF_MISC + NBARS * 8 + 16;
    static constexpr int OFF_COARSE = OFF_FIRST + (kMostBlocks + 1) * 4;
    static constexpr int OFF_SHARE = (OFF_COARSE + (kMaxBatch / 32 + 1) * 4 + 7) / 8 * 8;
    static constexpr int OFF_SCALES = (OFF_SHARE + static_cast<int>(sizeof(Share)) + 15) / 16 * 16;
    static constexpr int SMEM = OFF_SCALES + (I8 ? (2 * NSC + 1) * TK * 4 : 0) + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(D / 64 * OWN_BOX <= OWN_LO, "an own q's hi half");
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// Eight elements of a row of q, k, v or the bias from element i on, as loaded (16-byte loads where the base allows), and their values.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) == 4 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, size_t i, bool vec) {
        const T* s = static_cast<const T*>(base) + i;
        if (vec) {
            w[0] = __ldg(reinterpret_cast<const uint4*>(s));
            if constexpr (sizeof(T) == 4) w[1] = __ldg(reinterpret_cast<const uint4*>(s) + 1);
        } else {
            load_each(s);
        }
    }
    __device__ __noinline__ void load_each(const T* s) {
        T e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = s[k];
        memcpy(w, e, sizeof w);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        T e[8];
        memcpy(e, w, sizeof w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (sizeof(T) == 4) x[k] = e[k];
            else if constexpr (std::is_same_v<T, __half>) x[k] = __half2float(e[k]);
            else x[k] = __bfloat162float(e[k]);
        }
    }
};

// A wait whose barrier's phase is not complete yet, by a converged warp (tc::wait_or_abort).
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint32_t* err, volatile int* abort_flag, long long limit) {
    return __all_sync(0xffffffffu, tc::wait_or_abort(bar, parity, err, abort_flag, limit)) != 0;
}

// The roles' inner steps are loops or calls, each there once: unrolled and inlined at every place, the code of
// a tile (about 40 KB with pairs) ran from beyond the instruction cache, ten cycles an instruction (a pair's softmax
// took 20000 cycles a tile).

// q (and the bias) of query rows b0 + r, r_begin <= r < r_begin + rows (at most 32), of kv head h into rows r of a K-major operand of
// box_rows rows a box: hi at dst and lo lo_at behind; zeros for rows past the last.  By the 32 lanes of a warp
// together: pieces of 16 bytes lane + 32 w, lane + 32 (w + ws), ..; a lane finds the place of one row (a division) and the others ask it.
struct QRows {
    int at, head;  // row of q, or -1, and its head
    __device__ __forceinline__ QRows(const PrefixParams& p, int h, int row, bool on) : at(-1), head(0) {
        if (on && row < p.R) {
            const int bt = row / p.group;
            head = h * p.group + (row - bt * p.group);
            at = bt * p.Hq + head;
        }
    }
};
template <typename CT, typename T, int D>
static __device__ __noinline__ void put_q_as(const PrefixParams& p, unsigned char* dst, int box_rows, int lo_at, int h, int b0, int r_begin,
                                             int rows, int w, int ws) {
    constexpr int C = D / 8, U = sizeof(T) == 4 ? 2 : 4;
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, n = rows * C;
    const bool vec = ((reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.bias)) & 15u) == 0;
    const bool has_bias = p.bias != nullptr;
    const QRows mine(p, h, b0 + r_begin + lane, lane < rows);
#pragma unroll 1
    for (int i = 32 * w; i < n; i += U * 32 * ws) {
        Raw8<T> q[U], b[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int at = i + k * 32 * ws + lane, d = (at % C) * 8;
            const int row = __shfl_sync(FULL, mine.at, (at / C) & 31), head = __shfl_sync(FULL, mine.head, (at / C) & 31);
            q[k] = b[k] = Raw8<T>{};
            if (at >= n || row < 0) continue;
            q[k].load(p.q, static_cast<size_t>(row) * D + d, vec);
            if (has_bias) b[k].load(p.bias, static_cast<size_t>(head) * D + d, vec);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int at = i + k * 32 * ws + lane, r = r_begin + at / C, d = (at % C) * 8;
            float x[8], y[8];
            q[k].values(x);
            b[k].values(y);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) wide::split_pair<CT>(x[2 * e] + y[2 * e], x[2 * e + 1] + y[2 * e + 1], hi[e], lo[e]);
            if (at >= n) continue;
            unsigned char* to = dst + tc::sw128_offset(r, d, box_rows);
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// The same for a q of the cache's type: copied as it is, all pieces in flight at once where q is 16-byte aligned.
template <int D>
static __device__ __noinline__ void copy_q(const PrefixParams& p, unsigned char* dst, int box_rows, int h, int b0, int r_begin, int rows, int w,
                                           int ws) {
    constexpr int C = D / 8;
    const int lane = threadIdx.x & 31, n = rows * C;
    const bool vec = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0;
    const QRows mine(p, h, b0 + r_begin + lane, lane < rows);
#pragma unroll 2
    for (int i = 32 * w; i < n; i += 32 * ws) {
        const int at = i + lane, r = r_begin + at / C, d = (at % C) * 8;
        const int row = __shfl_sync(0xffffffffu, mine.at, (at / C) & 31);
        if (at >= n) continue;
        unsigned char* to = dst + tc::sw128_offset(r, d, box_rows);
        const unsigned short* src = static_cast<const unsigned short*>(p.q) + (row < 0 ? 0 : static_cast<size_t>(row) * D + d);
        if (vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(src), "r"(row < 0 ? 0 : 16) : "memory");
        } else {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) reinterpret_cast<unsigned short*>(to)[e] = row < 0 ? static_cast<unsigned short>(0) : src[e];
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}
template <typename CT, int D, bool PQ>
__device__ __forceinline__ void put_q(const PrefixParams& p, unsigned char* dst, int box_rows, int lo_at, int h, int b0, int r_begin, int rows,
                                      int w, int ws) {
    if constexpr (!PQ) copy_q<D>(p, dst, box_rows, h, b0, r_begin, rows, w, ws);
    else wide::with_qkv_type(p.qkv_dtype, [&](auto tag) { put_q_as<CT, decltype(tag), D>(p, dst, box_rows, lo_at, h, b0, r_begin, rows, w, ws); });
}

// One piece of 16 bytes of a new row of K and of V (elements si of both, bias at bk and bv): the bias is added in fp32 and the sum
// rounded once.
template <typename CT, typename T>
static __device__ __noinline__ void new_row8(const PrefixParams& p, size_t si, size_t bk, size_t bv, uint4 (&kv)[2]) {
    const bool vec = ((reinterpret_cast<uintptr_t>(p.k_new) | reinterpret_cast<uintptr_t>(p.v_new) | reinterpret_cast<uintptr_t>(p.bias)) & 15u) == 0;
    Raw8<T> a[2], b[2];
    a[0].load(p.k_new, si, vec);
    a[1].load(p.v_new, si, vec);
    b[0] = b[1] = Raw8<T>{};
    if (p.bias) {
        b[0].load(p.bias, bk, vec);
        b[1].load(p.bias, bv, vec);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float x[8], y[8];
        a[v].values(x);
        b[v].values(y);
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
        kv[v] = make_uint4(pack_ct<CT>(x[0], x[1]), pack_ct<CT>(x[2], x[3]), pack_ct<CT>(x[4], x[5]), pack_ct<CT>(x[6], x[7]));
    }
}

// All 128 scores of this thread's row.
__device__ __forceinline__ void load_scores(uint32_t ts, float (&v)[128]) {
    uint32_t u[128];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]),
          "=r"(u[32]), "=r"(u[33]), "=r"(u[34]), "=r"(u[35]), "=r"(u[36]), "=r"(u[37]), "=r"(u[38]), "=r"(u[39]),
          "=r"(u[40]), "=r"(u[41]), "=r"(u[42]), "=r"(u[43]), "=r"(u[44]), "=r"(u[45]), "=r"(u[46]), "=r"(u[47]),
          "=r"(u[48]), "=r"(u[49]), "=r"(u[50]), "=r"(u[51]), "=r"(u[52]), "=r"(u[53]), "=r"(u[54]), "=r"(u[55]),
          "=r"(u[56]), "=r"(u[57]), "=r"(u[58]), "=r"(u[59]), "=r"(u[60]), "=r"(u[61]), "=r"(u[62]), "=r"(u[63]),
          "=r"(u[64]), "=r"(u[65]), "=r"(u[66]), "=r"(u[67]), "=r"(u[68]), "=r"(u[69]), "=r"(u[70]), "=r"(u[71]),
          "=r"(u[72]), "=r"(u[73]), "=r"(u[74]), "=r"(u[75]), "=r"(u[76]), "=r"(u[77]), "=r"(u[78]), "=r"(u[79]),
          "=r"(u[80]), "=r"(u[81]), "=r"(u[82]), "=r"(u[83]), "=r"(u[84]), "=r"(u[85]), "=r"(u[86]), "=r"(u[87]),
          "=r"(u[88]), "=r"(u[89]), "=r"(u[90]), "=r"(u[91]), "=r"(u[92]), "=r"(u[93]), "=r"(u[94]), "=r"(u[95]),
          "=r"(u[96]), "=r"(u[97]), "=r"(u[98]), "=r"(u[99]), "=r"(u[100]), "=r"(u[101]), "=r"(u[102]), "=r"(u[103]),
          "=r"(u[104]), "=r"(u[105]), "=r"(u[106]), "=r"(u[107]), "=r"(u[108]), "=r"(u[109]), "=r"(u[110]), "=r"(u[111]),
          "=r"(u[112]), "=r"(u[113]), "=r"(u[114]), "=r"(u[115]), "=r"(u[116]), "=r"(u[117]), "=r"(u[118]), "=r"(u[119]),
          "=r"(u[120]), "=r"(u[121]), "=r"(u[122]), "=r"(u[123]), "=r"(u[124]), "=r"(u[125]), "=r"(u[126]), "=r"(u[127])
        : "r"(ts)
        : "memory");
#pragma unroll
    for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(u[i]);
}

// 32 scores on their way (nothing may touch v before land_scores), and their arrival.
__device__ __forceinline__ void fetch_scores(uint32_t ts, uint32_t (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(ts)
                 : "memory");
}
__device__ __forceinline__ void land_scores(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

// The scores of a tile that ends inside a row's view: those from column lim on become -inf, in TMEM.
static __device__ __noinline__ void mask_scores(uint32_t ts, int lim) {
#pragma unroll 1
    for (int c = 0; c < TK / 8; ++c) {
        float v[8];
        wide::tmem_ld_rows<8>(ts + 8 * c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * c + e >= lim) v[e] = -INFINITY;
        wide::tmem_st8(ts + 8 * c, v);
    }
    wide::tmem_st_wait();
}

// The weights of a tile in two passes over its scores: the largest, then the weights against the reference that it leaves.
template <typename CT, int D>
static __device__ __noinline__ float2 weigh_tile(uint32_t ts, uint32_t to, bool sees, bool chained, float2 ml, float qscale) {
    constexpr unsigned FULL = 0xffffffffu;
    float m = ml.x, l = ml.y;
    // the largest score, and what it does to the reference
    float t[4];
    {
        float v[TK];
        load_scores(ts, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = fmaxf(v[2 * k], v[2 * k + 1]);
#pragma unroll
        for (int e = 8; e < TK; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = fmaxf(t[k], fmaxf(v[e + 2 * k], v[e + 2 * k + 1]));
    }
    uint32_t v[32];
    fetch_scores(ts, v);
    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * qscale;
    if (__any_sync(FULL, sees && top > m + tc::kRescaleLog2)) {
        // (rows that see nothing of the tile, or whose scores do not pass their reference, keep it)
        const float mn = sees ? fmaxf(m, top) : m, alpha = wide::ex2(m - mn);
        m = mn;
        l *= alpha;
        if (chained) {
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
                float o[8];
                wide::tmem_ld_rows<8>(to + 8 * c, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= alpha;
                wide::tmem_st8(to + 8 * c, o);
            }
        }
    }
    // (a row that sees nothing of the tile: weights of 2^-inf)
    const float ref = sees ? -m : -INFINITY;
    const uint64_t sc2 = pack2(qscale, qscale), m2 = pack2(ref, ref);
    uint64_t acc0 = pack2(0.f, 0.f), acc1 = acc0;
    // a loop of 32 keys, the next ones' scores under way: the code of all 128 (18 KB) would not stay in the
    // instruction cache beside the other roles'
#pragma unroll 1
    for (int c = 0; c < TK / 32; ++c) {
        land_scores(v);
        uint32_t hi[16], lo[16];
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]);
        if (c + 1 < TK / 32) fetch_scores(ts + 32 * (c + 1), v);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float a, b;
            unpack2(fma2(pack2(x[e], x[e + 1]), sc2, m2), a, b);
            a = wide::ex2(a);
            b = wide::ex2(b);
            if (e & 2) acc1 = add2(acc1, pack2(a, b));
            else acc0 = add2(acc0, pack2(a, b));
            wide::split_pair<CT>(a, b, hi[e / 2], lo[e / 2]);
        }
        // 32 keys' weights: 16 columns of hi and 16 of lo, over scores that have been read
        tc::tmem_st16(ts + 32 * c, hi);
        tc::tmem_st16(ts + 32 * c + 16, lo);
    }
    float a, b;
    unpack2(add2(acc0, acc1), a, b);
    wide::tmem_st_wait();
    tc::tc_fence_before();
    return make_float2(m, l + (a + b));
}

// A tile whose scores are in TMEM at ts: the weights of this thread's row, which sees the first `lim` of its columns (none:
// <= 0), over them.  Columns from `edge` on belong to nobody and may hold anything.  live: the row is one; chained: its row of O, at to, holds earlier tiles.  ml: running reference and sum.
template <typename CT, int D>
static __device__ __noinline__ float2 take_tile(uint32_t ts, uint32_t to, int lim, int edge, bool live, bool chained, float2 ml, float qscale) {
    constexpr unsigned FULL = 0xffffffffu;
    const bool sees = live && lim > 0;
    const bool masked = live && lim < TK && (lim > 0 || edge < TK);
    if (__any_sync(FULL, masked)) mask_scores(ts, masked ? lim : TK);
    return weigh_tile<CT, D>(ts, to, sees, chained, ml, qscale);
}

// INT8: a tile's scores, times its rows' scales; those from column lim on become -inf.  In TMEM.
static __device__ __noinline__ void scale_scores(uint32_t ts, int lim, const float* ks) {
#pragma unroll 1
    for (int c = 0; c < TK / 8; ++c) {
        float v[8];
        wide::tmem_ld_rows<8>(ts + 8 * c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 8 * c + e < lim ? v[e] * ks[8 * c + e] : -INFINITY;
        wide::tmem_st8(ts + 8 * c, v);
    }
    wide::tmem_st_wait();
}

// A new reference for the rows of a warp that need one (moves) in the middle of a tile of codes, whose chunks of 32 columns before
// c0 hold weights already: the largest of the row's scores from there on, rounded up to a whole number.  What the old
// one has made (weights, O, the sum) is rescaled, by a power of two: exactly, so that the pairs keep their bits, which may
// count as much as the new weights (they may be 2^kReach of the old reference).  The other rows keep theirs, and nothing of
// them changes.
template <int D>
static __device__ __noinline__ float2 move_reference(uint32_t ts, uint32_t to, int c0, bool moves, bool chained, float2 ml, const float* ks) {
    float top = -INFINITY;
    wide::tmem_st_wait();  // the chunks before c0 are read below: a load is not ordered behind the stores of their weights
#pragma unroll 1
    for (int c = 4 * c0; c < TK / 8; ++c) {
        float x[8];
        wide::tmem_ld_rows<8>(ts + 8 * c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, x[e] * ks[8 * c + e]);
    }
    const float mn = moves ? ceilf(top) : ml.x, down = mn - ml.x;  // (whole numbers, or the first reference)
    const float alpha = down > 126.f ? 0.f : __int_as_float((127 - static_cast<int>(down)) << 23);
#pragma unroll 1
    for (int c = 0; c < 4 * c0; ++c) {
        float x[8];
        wide::tmem_ld_rows<8>(ts + 8 * c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t w = __float_as_uint(x[e]);
            x[e] = __uint_as_float(pack_ct<__nv_bfloat16>(__uint_as_float(w << 16) * alpha, __uint_as_float(w & 0xFFFF0000u) * alpha));
        }
        wide::tmem_st8(ts + 8 * c, x);
    }
    if (chained) {
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
            float o[8];
            wide::tmem_ld_rows<8>(to + 8 * c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= alpha;
            wide::tmem_st8(to + 8 * c, o);
        }
    }
    wide::tmem_st_wait();
    return make_float2(mn, alpha);
}

// take_tile for codes: S and the weights are of codes, whose rows' scales are in shared memory.  K's (times the softmax scale)
// multiply the scores, V's the weights behind their sum: bf16 numbers, whose range takes any scale, and any weight up to 2^kReach
// besides, so the reference stays where it is until a score is that far above it, and one pass over the scores is enough (a pass for
// the largest score first took 304 us instead of 259, with single weights, for 64 70B-shaped slots of two tokens behind
// 32768 rows, their own rows included).  ones: 128 of them, for scores
// that are scaled already.  In chunks of 32 columns: 128 registers a thread.
constexpr float kReach = 40.f;
template <int D>
static __device__ __noinline__ float2 take_tile_i8(uint32_t ts, uint32_t to, int lim, bool chained, float2 ml, const float* ks, const float* vs,
                                                   const float* ones) {
    constexpr unsigned FULL = 0xffffffffu;
    const bool sees = lim > 0, masked = sees && lim < TK;
    if (__any_sync(FULL, masked)) {
        scale_scores(ts, masked ? lim : TK, ks);
        ks = ones;
    }
    uint32_t v[32];
    fetch_scores(ts, v);
    float ref = sees ? -ml.x : -INFINITY;  // (a row that sees nothing of the tile: weights of 2^-inf)
    uint64_t acc0 = pack2(0.f, 0.f), acc1 = acc0;
#pragma unroll 1
    for (int c = 0; c < TK / 32; ++c) {
        land_scores(v);
        float x[32], t0 = -INFINITY, t1 = -INFINITY;
        auto relative = [&] {
            const uint64_t m2 = pack2(ref, ref);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + e);
                unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), pack2(k.x, k.y), m2), x[e], x[e + 1]);
                unpack2(fma2(pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), pack2(k.z, k.w), m2), x[e + 2], x[e + 3]);
            }
        };
        relative();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            t0 = fmaxf(t0, fmaxf(x[e], x[e + 1]));
            t1 = fmaxf(t1, fmaxf(x[e + 2], x[e + 3]));
        }
        const bool moves = sees && fmaxf(t0, t1) > kReach;
        if (__any_sync(FULL, moves)) {
            const float2 moved = move_reference<D>(ts, to, c, moves, chained, ml, ks);
            const uint64_t a2 = pack2(moved.y, moved.y);
            ml = make_float2(moved.x, ml.y * moved.y);
            acc0 = mul2(acc0, a2);
            acc1 = mul2(acc1, a2);
            ref = sees ? -ml.x : -INFINITY;
            fetch_scores(ts + 32 * c, v);
            land_scores(v);
            relative();
        }
        if (c + 1 < TK / 32) fetch_scores(ts + 32 * (c + 1), v);
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(vs + 32 * c + e);
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                float a = wide::ex2(x[e + g]), b = wide::ex2(x[e + g + 1]);
                const uint64_t ab = pack2(a, b);
                if (g) acc1 = add2(acc1, ab);
                else acc0 = add2(acc0, ab);
                unpack2(mul2(ab, g ? pack2(w.z, w.w) : pack2(w.x, w.y)), a, b);
                wide::split_pair<__nv_bfloat16>(a, b, hi[(e + g) / 2], lo[(e + g) / 2]);
            }
        }
        tc::tmem_st16(ts + 32 * c, hi);
        tc::tmem_st16(ts + 32 * c + 16, lo);
    }
    float a, b;
    unpack2(add2(acc0, acc1), a, b);
    wide::tmem_st_wait();
    tc::tc_fence_before();
    return make_float2(ml.x, ml.y + (a + b));
}

// Two codes (bytes of x by sel, 0x4140 or 0x4342) as a pair of bf16 numbers: under the exponent of 128 the low seven bits are
// 128 + them, and the sign bit alone is 128 or 256, which is subtracted exactly.
__device__ __forceinline__ uint32_t codes_to_bf2(uint32_t x, uint32_t sel) {
    const uint32_t h = __byte_perm(x, 0x43434343u, sel), a = h & 0xFF7FFF7Fu, b = h & 0xFF80FF80u;
    __nv_bfloat162 va, vb;
    memcpy(&va, &a, 4);
    memcpy(&vb, &b, 4);
    va = __hsub2(va, vb);
    uint32_t r;
    memcpy(&r, &va, 4);
    return r;
}
// Eight codes as eight 16-bit numbers
template <typename CT>
__device__ __forceinline__ uint4 eight_codes(uint32_t x, uint32_t y) {
    if constexpr (std::is_same_v<CT, __half>) {
        x ^= 0x80808080u;
        y ^= 0x80808080u;
        return make_uint4(tc::codes_to_h2(x, 0x4140), tc::codes_to_h2(x, 0x4342), tc::codes_to_h2(y, 0x4140), tc::codes_to_h2(y, 0x4342));
    } else {
        return make_uint4(codes_to_bf2(x, 0x4140), codes_to_bf2(x, 0x4342), codes_to_bf2(y, 0x4140), codes_to_bf2(y, 0x4342));
    }
}

// One thread's part (t of 128) of a tile of codes: pieces of 16 codes t + 128 k, from global memory (zeros from row `rows` on), and
// to a K-major (V: MN-major, the same places) operand of 16-bit numbers.
template <int D>
struct Codes {
    static constexpr int N = D / 16;  // pieces of a thread, and of a row
    uint4 w[N];
    __device__ __forceinline__ void load(const unsigned char* base, long long row, int rows, int t) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = t + 128 * k, r = i / N;
            w[k] = r < rows ? __ldcg(reinterpret_cast<const uint4*>(base + (row + r) * D) + i % N) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    template <typename CT>
    __device__ __forceinline__ void store(unsigned char* tile, int t) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = t + 128 * k, r = i / N, d = (i % N) * 16, swap = (i % N) >> 2;  // (lanes four pieces apart: the same banks)
            const uint4 a = eight_codes<CT>(w[k].x, w[k].y), b = eight_codes<CT>(w[k].z, w[k].w);
            *reinterpret_cast<uint4*>(tile + tc::sw128_offset(r, d + 8 * swap, TK)) = swap ? b : a;
            *reinterpret_cast<uint4*>(tile + tc::sw128_offset(r, d + 8 * (swap ^ 1), TK)) = swap ? a : b;
        }
    }
};

// The products take their operands as uniform registers.  What is the same for the whole warp is handed round once, so that
// the compiler knows it to be, and descriptors are built from their low halves (the high ones are all alike: rows 1 KB apart
// in groups of eight, 128-byte swizzle).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }

// D (TMEM) (+)= A (shared memory) . B (shared memory)
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(add), "n"(kDescHigh)
        : "memory");
}
// D (TMEM) (+)= A (TMEM) . B (shared memory)
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(add), "n"(kDescHigh)
        : "memory");
}

// The scores' products: q at qa (lo half lo_at behind, boxes box_at apart, in 16-byte units), K at ka.  One thread.
template <int D, bool PQ>
__device__ __forceinline__ void issue_scores(uint32_t ts, uint32_t qa, uint32_t ka, uint32_t lo_at, uint32_t box_at, uint32_t id) {
    tc::tc_fence_after();
#pragma unroll
    for (int kq = 0; kq < D / 16; ++kq) {
        const uint32_t k = ka + (((kq >> 2) * KB + (kq & 3) * 32) >> 4), q = qa + (kq >> 2) * box_at + (kq & 3) * 2;
        product_ss(ts, q, k, id, kq > 0);
        if constexpr (PQ) product_ss(ts, q + lo_at, k, id, 1u);
    }
}

// The weights (TMEM at tp) times V at vb into O at to, which begins (more 0) or goes on.  One thread.
template <int D>
__device__ __forceinline__ void issue_values(uint32_t to, uint32_t tp, uint32_t vb, uint32_t more, uint32_t id) {
    tc::tc_fence_after();
#pragma unroll
    for (int kq = 0; kq < TK / 16; ++kq) {
        // (chunks of 32 keys: 16 columns of hi, 16 of lo)
        const uint32_t v = vb + (kq * 2048 >> 4), c = tp + (kq >> 1) * 32 + (kq & 1) * 8;
        product_ts(to, c, v, id, kq > 0 ? 1u : more);
        product_ts(to, c + 16, v, id, 1u);
    }
}

// One thread of a converged warp, known to the compiler as one (operands of the tensor-core instructions are then uniform).
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Rows of a slot's own segment: its cached ones and the new ones; 0 without work.
__device__ __forceinline__ int own_rows(const PrefixParams& p, int L) { return L >= 0 && L <= p.Lmax - p.T ? L + p.T : 0; }

static __device__ __noinline__ PrefixCursor locate_piece(const int* first, long long u, int row_blocks) { return prefix_locate(u, first, row_blocks); }

// A walk over the tiles of the slots' own rows: slots in order, their kv heads, the tiles of a segment.  By the
// 32 lanes of a warp together, which keep the lengths of 32 slots.
struct OwnWalk {
    int b, h, tile, nt, L;
    int base, lens;  // first slot of the 32, and this lane's length

    __device__ __forceinline__ void fetch(const PrefixParams& p, int group, int lane) {
        base = group * 32;
        lens = base + lane < p.B ? __ldcg(p.seq_lens + base + lane) : -1;
    }
    // tile u of the space; coarse[k]: tiles of one kv head of the slots before 32 k
    __device__ __noinline__ void locate(const PrefixParams& p, const int* coarse, long long u, int lane) {
        int lo = 0, hi = (p.B + 31) / 32 - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (static_cast<long long>(coarse[mid]) * p.Hkv <= u) lo = mid;
            else hi = mid - 1;
        }
        fetch(p, lo, lane);
        const int n = (own_rows(p, lens) + TK - 1) / TK;
        int before = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, m);
            if (lane >= m) before += y;
        }
        before += coarse[lo] - n;
        const unsigned at = __ballot_sync(0xffffffffu, n > 0 && static_cast<long long>(before) * p.Hkv <= u);
        const int i = 31 - __clz(at);
        b = base + i;
        nt = __shfl_sync(0xffffffffu, n, i);
        L = __shfl_sync(0xffffffffu, lens, i);
        const int rem = static_cast<int>(u - static_cast<long long>(__shfl_sync(0xffffffffu, before, i)) * p.Hkv);
        h = rem / nt;
        tile = rem - h * nt;
    }
    // to the first tile of the next segment (there is one)
    __device__ __noinline__ void next_segment(const PrefixParams& p, int lane) {
        tile = 0;
        if (++h < p.Hkv) return;
        h = 0;
        do {
            ++b;
            if (b >= base + 32) fetch(p, b >> 5, lane);
            L = __shfl_sync(0xffffffffu, lens, b - base);
        } while (own_rows(p, L) == 0 && b + 1 < p.B);
        nt = (own_rows(p, L) + TK - 1) / TK;
    }
    __device__ __forceinline__ void next(const PrefixParams& p, int lane) {
        if (++tile == nt) next_segment(p, lane);
    }
};

// Cache row of position t of (slot, kv head); -1 for a page outside the pool.
__device__ __forceinline__ long long own_row(const PrefixParams& p, int b, int h, int t) {
    if (!p.block_table) return (static_cast<long long>(b) * p.Hkv + h) * p.Lmax + t;
    const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.pages_per_seq + (t >> p.page_shift));
    if (page < 0 || page >= p.num_pages) return -1;
    return ((static_cast<long long>(page) * p.Hkv + h) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// Equal contiguous ranges of the own tiles over the streams of all blocks (two a block); none is empty, so every worker
// between a segment's first and last holds a piece of it.
struct OwnSplit {
    long long U;
    int V;
    __device__ OwnSplit(const PrefixParams& p, const int* coarse)
        : U(p.own ? static_cast<long long>(p.Hkv) * coarse[(p.B + 31) / 32] : 0),
          V(static_cast<int>(min(2LL * p.workers, max(U, 1LL)))) {}
    __device__ long long begin(int v) const { return equal_share(U, V, v); }
    __device__ int tiles(int v) const { return static_cast<int>(begin(v + 1) - begin(v)); }
    __device__ int holder(long long u) const { return static_cast<int>(((u + 1) * V - 1) / U); }
};

// CT: the type of q and K as operands, and without I8 of V and the weights too (with it those are bf16)
template <typename CT, int D, bool PQ, bool I8>
__global__ void __launch_bounds__(I8 ? kThreadsI8 : kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ CUtensorMap tmk_own, const __grid_constant__ CUtensorMap tmv_own,
                     const __grid_constant__ PrefixParams p) {
    using LY = Layout<D, I8>;
    using WT = std::conditional_t<I8, __nv_bfloat16, CT>;
    constexpr int NK = LY::NK, NV = LY::NV, NSLOT = LY::NSLOT, TILE = LY::TILE, BOXES = D / 64;
    constexpr bool BF = std::is_same_v<CT, __nv_bfloat16>;
    constexpr unsigned FULL = 0xffffffffu;
    enum : int {
        kFull = 0, kReady = NSLOT, kEmpty = 2 * NSLOT,  // a slot's tile has landed, is whole, is read
        kSFull = 3 * NSLOT, kPFull = kSFull + 2, kOFull = kSFull + 4,  // of each stream
        kStart = kSFull + 6, kMeet = kSFull + 7, kDrain = kSFull + 8, kTurn = kSFull + 9
    };
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* ring = smem + LY::OFF_RING;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LY::OFF_MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + LY::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* first = reinterpret_cast<int*>(smem + LY::OFF_FIRST);
    int* coarse = reinterpret_cast<int*>(smem + LY::OFF_COARSE);  // [k]: own tiles of one kv head of the slots before 32 k
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < LY::NBARS; ++i) mbar_init(bar(i), (i >= kPFull && i < kPFull + 2) || (I8 && i >= kReady && i < kReady + NSLOT) ? 4 : i == kStart || i == kMeet ? 8 : i == kDrain || (i >= kEmpty && i < kEmpty + NSLOT) ? 2 : 1);
        *abort_flag = 0;
    }
    float* const scales = reinterpret_cast<float*>(smem + LY::OFF_SCALES);  // INT8: [NSC][K, V][TK], and the ones
    if (I8 && tid < TK) scales[2 * LY::NSC * TK + tid] = 1.f;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_mbar_init();
    tc::tc_fence_before();
    // With own rows this is the call's first kernel; behind the step's it runs beside its last blocks (see the CUDA-core kernel).
    if (p.own) {
        grid_dep_wait();
        const int groups = (p.B + 31) / 32;
#pragma unroll 1
        for (int g = warp; g < groups; g += kThreads / 32) {
            const int b = g * 32 + lane, L = b < p.B ? __ldcg(p.seq_lens + b) : -1;
            int n = (own_rows(p, L) + TK - 1) / TK;
            if (blockIdx.x == 0 && L > p.Lmax - p.T) atomicOr(p.err, kErrSeqOverflow);
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) n += __shfl_xor_sync(FULL, n, m);
            if (lane == 0) coarse[g + 1] = n;
        }
    }
    build_prefix_plan(p, first, TK);
    const int w = blockIdx.x;
    Share& share = *reinterpret_cast<Share*>(smem + LY::OFF_SHARE);
    if (tid == 0) {
        if (p.own) {
            coarse[0] = 0;
#pragma unroll 1
            for (int g = 0; g < (p.B + 31) / 32; ++g) coarse[g + 1] += coarse[g];
        }
        const PrefixSplit sp(p, first);
        const OwnSplit so(p, coarse);
        share.u_begin = sp.begin(w);
        share.u_end = sp.begin(w + 1);
        // workers w and w + workers, the one with more tiles as stream 0
        const int n0 = so.tiles(w), n1 = so.tiles(w + p.workers), swap = n1 > n0;
        share.own_v[0] = swap ? w + p.workers : w;
        share.own_v[1] = swap ? w : w + p.workers;
        share.own_n[0] = max(n0, n1);
        share.own_n[1] = min(n0, n1);
        share.own_at[0] = so.begin(share.own_v[0]);
        share.own_at[1] = so.begin(share.own_v[1]);
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long u_begin = share.u_begin, u_end = share.u_end;
    const int* own_n = share.own_n;
    const int* own_v = share.own_v;
    const bool owns = own_n[0] > 0;
    const bool own_first = w & 1;
    const bool works = u_begin < u_end || owns;
    // pieces of the prefix: (kv head, row block, tiles); the roles walk them in step
    struct Piece {
        PrefixCursor c;
        int nt;
        bool twice;
    };
    auto piece_at = [&](long long u) {
        Piece x;
        x.c = locate_piece(first, u, p.row_blocks);
        x.nt = static_cast<int>(min(static_cast<long long>(x.c.nt - x.c.tile), u_end - u));
        x.twice = prefix_twice(p, x.c.rb);
        return x;
    };
    // tiles of stream s in a piece, and the piece's tile that is its j-th
    auto tiles_of = [](const Piece& x, int s) { return x.twice ? (x.nt - s + 1) / 2 : x.nt; };
    auto tile_of = [](const Piece& x, int s, int j) { return x.twice ? 2 * j + s : j; };
    // Tiles are counted in the order of the copies: a piece's tiles in turn; on own rows stream 0's i-th tile, then stream 1's.
    // K and V slot of tile t, and the parity of its round
    auto k_slot = [](int t) { return t % NK; };
    auto k_par = [](int t) { return (t / NK) & 1; };
    auto v_slot = [](int t) { return NK + t % NV; };
    auto v_par = [](int t) { return (t / NV) & 1; };
    auto wait = [&](int b, int parity) {
        if (__all_sync(FULL, mbar_try_wait(bar(b), parity))) return true;
        return wait_on(bar(b), parity, p.err, abort_flag, p.wait_cycles);
    };

    int issued = 0;  // producer: K and V tiles copied (or withheld)
    const bool withhold = p.stall && blockIdx.x == 0;  // test hook: block 0's first copy never comes
    if (!I8 && works && warp == 0) {
        // ------------------------------------------------ TMA producer
        bool ok = true;
        auto copy = [&](const CUtensorMap* mk, const CUtensorMap* mv, long long row) -> bool {
            if (row < 0) {
                if (lane == 0) atomicOr(p.err, kErrBadPage);
                row = 0;
            }
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                const int t = issued >> 1, slot = v ? v_slot(t) : k_slot(t);
                if (t >= (v ? NV : NK) && !wait(kEmpty + slot, (v ? v_par(t) : k_par(t)) ^ 1)) return false;
                if (!(withhold && issued == 0) && elect_one()) {
                    const uint32_t dst = smem_addr(ring + slot * TILE);
                    mbar_arrive_expect_tx(bar(kFull + slot), TILE);
#pragma unroll
                    for (int b = 0; b < BOXES; ++b) tma_load(dst + b * KB, v ? mv : mk, 64 * b, static_cast<int>(row), bar(kFull + slot));
                }
                __syncwarp();
                ++issued;
            }
            return true;
        };
        for (int ph = 0; ph < 2 && ok; ++ph) {
            if ((ph == 0) != own_first) {
#pragma unroll 1
                for (long long u = u_begin; u < u_end && ok;) {
                    const Piece x = piece_at(u);
#pragma unroll 1
                    for (int i = 0; i < x.nt && ok; ++i) {
                        const long long row = prefix_row(p, x.c.h, (x.c.tile + i) * TK);
                        ok = copy(&tmk, &tmv, row);
                    }
                    u += x.nt;
                }
            } else if (owns) {
                OwnWalk k[2];
                k[0].locate(p, coarse, share.own_at[0], lane);
                if (own_n[1]) k[1].locate(p, coarse, share.own_at[1], lane);
#pragma unroll 1
                for (int i = 0; i < own_n[0] && ok; ++i) {
#pragma unroll 1
                    for (int s = 0; s < 2; ++s) {
                        if (i >= own_n[s] || !ok) continue;
                        const long long row = own_row(p, k[s].b, k[s].h, k[s].tile * TK);
                        ok = copy(&tmk_own, &tmv_own, row);
                        if (i + 1 < own_n[s]) k[s].next(p, lane);
                    }
                }
            }
        }
    } else if (works && (warp == 1 || warp == 3)) {
        // ------------------------------------------------ products of one stream
        const int s = warp >> 1;
        const uint32_t id_s = tc::instr_desc(BF, TK, TK, false), id_o = tc::instr_desc(std::is_same_v<WT, __nv_bfloat16>, TK, D, false, true);
        const uint32_t dq0 = desc_low(smem_addr(smem), 16), dk0 = desc_low(smem_addr(ring), 16), dv0 = desc_low(smem_addr(ring), KB);
        const uint32_t ts = uniform(tmem + s * TK), to = ts + 2 * TK;
        int tiles = 0, starts = 0;  // tiles of the pieces before; starts waited for
        int np = 0, turns = 0;      // products P.V issued; steps taken
        bool ok = true;
        auto tile_ready = [&](int slot, int parity) { return wait(kReady + slot, parity) && (I8 || wait(kFull + slot, parity)); };
        // a slot is free when both streams are through with it; a tile of one stream counts twice
        auto release = [&](uint32_t slot, bool both) {
            tc::mma_commit(bar(kEmpty + slot));
            if (!both) tc::mma_commit(bar(kEmpty + slot));
        };
        // One step: the weights times V of tile v (none: < 0) once they are there, then the scores with K of tile k
        // (none: < 0).  The tiles are waited for before the weights, so nothing comes between the two products.
        // fresh, end: O begins and is complete with this product; both: the other stream takes the tiles too.
        // The streams take turns, so that one's softmax falls under the other's products: without, both come at once, and both
        // wait for twice the products (4250 against 3000 cycles a step).
        auto step = [&](int v, bool fresh, bool end, int k, uint32_t q_at, uint32_t lo_at, uint32_t box_at, bool both) -> bool {
            if (v >= 0 && !tile_ready(v_slot(v), v_par(v))) return false;
            if (k >= 0 && !tile_ready(k_slot(k), k_par(k))) return false;
            if (v >= 0 && !wait(kPFull + s, np++ & 1)) return false;
            if (s + turns > 0 && !wait(kTurn + s, (turns + s - 1) & 1)) return false;
            ++turns;
            const uint32_t vs = uniform(v >= 0 ? v_slot(v) : 0), ks = uniform(k >= 0 ? k_slot(k) : 0), qa = uniform(dq0 + (q_at >> 4));
            const uint32_t does = uniform((v >= 0) | (k >= 0) << 1 | end << 2 | both << 3 | !fresh << 4);
            if (elect_one()) {
                if (does & 1) {
                    issue_values<D>(to, ts, dv0 + vs * (TILE >> 4), does >> 4, id_o);
                    release(vs, does & 8);
                    if (does & 4) tc::mma_commit(bar(kOFull + s));
                }
                if (does & 2) {
                    issue_scores<D, PQ>(ts, qa, dk0 + ks * (TILE >> 4), lo_at >> 4, box_at >> 4, id_s);
                    tc::mma_commit(bar(kSFull + s));
                    release(ks, does & 8);
                }
                mbar_arrive(bar(kTurn + (s ^ 1)));
            }
            __syncwarp();
            return true;
        };
#pragma unroll 1
        for (int ph = 0; ph < 2 && ok; ++ph) {
            if ((ph == 0) != own_first) {
#pragma unroll 1
                for (long long u = u_begin; u < u_end && ok;) {
                    const Piece x = piece_at(u);
                    ok = wait(kStart, starts & 1);  // q is there, O of the piece before is read
                    ++starts;
                    const int n = tiles_of(x, s);
                    if (n == 0 && lane == 0) mbar_arrive(bar(kOFull + s));  // (so that no role passes a piece ahead of another)
                    const int most = tiles_of(x, 0);
#pragma unroll 1
                    for (int j = -1; j < most && ok; ++j)
                        ok = step(j < 0 || j >= n ? -1 : tiles + tile_of(x, s, j), j == 0, j + 1 == n, j + 1 < n ? tiles + tile_of(x, s, j + 1) : -1,
                                  PQ ? 0 : s * TILE, TILE, KB, !x.twice);
                    tiles += x.nt;
                    u += x.nt;
                }
            } else if (owns) {
                const int n = own_n[s];
                OwnWalk k;  // of the scores
                if (n > 0) k.locate(p, coarse, share.own_at[s], lane);
                int buf = 0;
                bool fresh = true;
                ok = wait(kStart, starts & 1);
                ++starts;
                if (n == 0 && lane == 0) mbar_arrive(bar(kOFull + s));
#pragma unroll 1
                for (int i = -1; i < own_n[0] && ok; ++i) {
                    const bool has = i >= 0 && i < n, end = has && (k.tile + 1 == k.nt || i + 1 == n);  // of the piece of tile i
                    if (has && i + 1 < n) k.next(p, lane);
                    if (end) buf ^= 1;
                    ok = step(has ? tiles + 2 * i + s : -1, fresh, end, i + 1 < n ? tiles + 2 * (i + 1) + s : -1,
                              s * TILE + buf * LY::OWN_BUF, LY::OWN_LO, LY::OWN_BOX, false);
                    if (has) fresh = end;
                }
                tiles += own_n[0] + own_n[1];
            }
        }
        // one last commit: it completes once every product issued above has
        if (elect_one()) tc::mma_commit(bar(kDrain));
        __syncwarp();
    } else if (!I8 && works && warp == 2) {
        // ------------------------------------------------ tiles that are not whole
        int items = 0;
        bool ok = true;
        auto slot_of = [&]() { return items & 1 ? v_slot(items >> 1) : k_slot(items >> 1); };
        auto landed = [&]() { return wait(kFull + slot_of(), items & 1 ? v_par(items >> 1) : k_par(items >> 1)); };
        auto pass = [&](bool written) {
            if (written) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kReady + slot_of()));
            ++items;
        };
        // rows from `from` on of the V tile that is there become zeros
        auto zero_rows = [&](int from) {
            unsigned char* tile = ring + slot_of() * TILE + from * 128;
            const int nz = (TK - from) * 8;
#pragma unroll 4
            for (int i = lane; i < nz; i += 32) {
#pragma unroll
                for (int b = 0; b < BOXES; ++b) *reinterpret_cast<uint4*>(tile + b * KB + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
        };
        for (int ph = 0; ph < 2 && ok; ++ph) {
            if ((ph == 0) != own_first) {
#pragma unroll 1
                for (long long u = u_begin; u < u_end && ok;) {
                    const Piece x = piece_at(u);
                    const int seen = prefix_block_seen(p, x.c.rb, lane);
#pragma unroll 1
                    for (int i = 0; i < 2 * x.nt && ok; ++i) {
                        ok = landed();
                        const int left = seen - (x.c.tile + (i >> 1)) * TK;  // (at least 1)
                        const bool cut = (i & 1) && left < TK && ok;
                        if (cut) zero_rows(left);
                        pass(cut);
                    }
                    u += x.nt;
                }
            } else if (owns) {
                OwnWalk k[2];
                k[0].locate(p, coarse, share.own_at[0], lane);
                if (own_n[1]) k[1].locate(p, coarse, share.own_at[1], lane);
#pragma unroll 1
                for (int i = 0; i < own_n[0] && ok; ++i) {
#pragma unroll 1
                    for (int s = 0; s < 2 && ok; ++s) {
                        if (i >= own_n[s]) continue;
                        const int L = k[s].L, t0 = k[s].tile * TK, b = k[s].b, h = k[s].h;
                        const int from = max(L, t0), upto = min(L + p.T, t0 + TK);
                        // eight elements of a new row of K and of V per lane and turn; the first turn's, and their places in the
                        // cache, are there before the tiles are
                        const int n = max(0, upto - from) * (D / 8);
                        uint4 kv[2];
                        long long row = -1;
                        auto fetch = [&](int j) {
                            const int d0 = (j % (D / 8)) * 8, pos = from + j / (D / 8);
                            const size_t si = ((static_cast<size_t>(b) * p.T + (pos - L)) * p.Hkv + h) * D + d0;
                            const size_t bi = static_cast<size_t>(p.Hq + h) * D + d0, vi = static_cast<size_t>(p.Hkv) * D;
                            row = own_row(p, b, h, pos);
                            wide::with_qkv_type(p.qkv_dtype, [&](auto tag) { new_row8<CT, decltype(tag)>(p, si, bi, bi + vi, kv); });
                        };
                        if (lane < n) fetch(lane);
#pragma unroll 1
                        for (int v = 0; v < 2 && ok; ++v) {
                            ok = landed();
                            if (!ok) break;
                            unsigned char* tile = ring + slot_of() * TILE;
                            unsigned char* cache = v ? p.v_cache : p.k_cache;
#pragma unroll 1
                            for (int j = lane; j < n; j += 32) {
                                if (n > 32) fetch(j);  // (both turns' do not fit the registers)
                                const int d0 = (j % (D / 8)) * 8, pos = from + j / (D / 8);
                                *reinterpret_cast<uint4*>(tile + tc::sw128_offset(pos - t0, d0, TK)) = kv[v];
                                if (row >= 0) *reinterpret_cast<uint4*>(cache + (row * D + d0) * 2) = kv[v];
                            }
                            const int end = L + p.T - t0;
                            if (v && end < TK) zero_rows(end);
                            pass(n > 0 || (v && end < TK));
                        }
                        if (i + 1 < own_n[s]) k[s].next(p, lane);
                    }
                }
            }
        }
    } else if (I8 && works && warp >= 12) {
        // ------------------------------------------------ codes into 16-bit numbers
        const int t = tid - kThreads;
        int tile = 0;  // tiles made
        bool ok = true;
        Piece x = piece_at(u_begin);
        int i = 0, most = prefix_block_seen(p, x.c.rb, lane);
        long long u = u_begin;
        long long row = 0;
        int rows = 0;
        auto place = [&] {  // of tile i of the piece
            const int t0 = (x.c.tile + i) * TK;
            row = prefix_row(p, x.c.h, t0);
            rows = min(TK, most - t0);
            if (row < 0) {
                if (t == 0) atomicOr(p.err, kErrBadPage);
                row = 0;
            }
        };
        auto publish = [&](int slot, bool held) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !held) mbar_arrive(bar(kReady + slot));
        };
        // a row's two scales go with its K: the softmax takes both as soon as there are scores
        Codes<D> k, v;
        float k_scale, v_scale;
        auto load_k = [&] {
            place();
            k.load(p.k, row, rows, t);
            k_scale = t < rows ? __ldcg(p.k_scales + row + t) : 0.f;
            v_scale = t < rows ? __ldcg(p.v_scales + row + t) : 0.f;
        };
        load_k();
#pragma unroll 1
        while (ok) {
            float* sc = scales + tile % (I8 ? LY::NSC : 1) * (2 * TK);
            v.load(p.v, row, rows, t);
            if (tile >= NK) ok = wait(kEmpty + k_slot(tile), k_par(tile) ^ 1);
            if (!ok) break;
            k.template store<CT>(ring + k_slot(tile) * TILE, t);
            sc[t] = k_scale * p.qscale;
            sc[TK + t] = v_scale;
            publish(k_slot(tile), withhold && tile == 0);
            if (++i == x.nt) {
                u += x.nt;
                i = 0;
                if (u < u_end) {
                    x = piece_at(u);
                    most = prefix_block_seen(p, x.c.rb, lane);
                }
            }
            const bool more = u < u_end;
            if (more) load_k();
            if (tile >= NV) ok = wait(kEmpty + v_slot(tile), v_par(tile) ^ 1);
            if (!ok) break;
            v.template store<WT>(ring + v_slot(tile) * TILE, t);
            publish(v_slot(tile), false);
            ++tile;
            if (!more) break;
        }
    } else if (works && warp >= 4 && warp < 12) {
        // ------------------------------------------------ softmax of one stream
        const int s = (warp >> 2) - 1, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + s * TK, to = tmem + lanes + 2 * TK + s * TK;
        int tiles = 0;  // of the pieces before
        int ns = 0, no[2] = {0, 0};  // score tiles taken; outputs completed, of both streams
        bool ok = true;
        float2 ml = make_float2(kNone, 0.f);  // running reference and sum of the row
#pragma unroll 1
        for (int ph = 0; ph < 2 && ok; ++ph) {
            if (ph == 1 && u_begin < u_end && owns) {
                // both streams are through with the phase before: their q's share memory with the next one's
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kMeet));
                ok = wait(kMeet, 0);
                if (!ok) break;
            }
            if ((ph == 0) != own_first) {
#pragma unroll 1
                for (long long u = u_begin; u < u_end && ok;) {
                    const Piece x = piece_at(u);
                    const int n = tiles_of(x, s);
                    const int row = x.c.rb * p.block_rows + (x.twice ? r : s * TK + r);
                    const bool live = row < p.R, any_live = __any_sync(FULL, live);  // (a warp past the last row: its O is nobody's)
                    {
                        // q: neighbouring lanes take neighbouring 16 bytes of a row (a pair's q is made by both streams, half
                        // of the rows each)
                        const int r0 = quarter * 32 + (PQ ? 16 * s : 0);
                        put_q<CT, D, PQ>(p, smem + (PQ ? 0 : s * TILE), TK, TILE, x.c.h, x.c.rb * p.block_rows + (x.twice ? 0 : s * TK), r0,
                                           PQ ? 16 : 32, 0, 1);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kStart));
                    }
                    const int seen = live ? prefix_seen(p, prefix_slot_of(p, row)) : 0, most = prefix_block_seen(p, x.c.rb, lane);
                    ml = make_float2(kNone, 0.f);
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        ok = wait(kSFull + s, ns & 1);
                        if (!ok) break;
                        ++ns;
                        tc::tc_fence_after();
                        const int at = tile_of(x, s, j), lim = seen - (x.c.tile + at) * TK;
                        if (!any_live) {
                        } else if constexpr (I8) {
                            const float* sc = scales + (tiles + at) % LY::NSC * (2 * TK);
                            ml = take_tile_i8<D>(ts, to, lim, j > 0, ml, sc, sc + TK, scales + 2 * LY::NSC * TK);
                        } else {
                            ml = take_tile<CT, D>(ts, to, lim, most - (x.c.tile + at) * TK, true, j > 0, ml, p.qscale);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kPFull + s));
                    }
                    if (!ok) break;
                    // ---- the piece's partial ----
                    float* slot = p.ws + static_cast<size_t>(x.c.h * p.row_blocks + x.c.rb + w) * prefix_slot_floats(p.slot_rows, D) + s * TK + r;
                    constexpr int SR = 2 * TK;  // p.slot_rows
                    __stcg(slot, ml.x);
                    __stcg(slot + SR, ml.y);
                    ok = wait(kOFull + s, no[s] & 1);
                    if (!ok) break;
                    ++no[s];
                    tc::tc_fence_after();
                    if (n > 0 && any_live) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            wide::tmem_ld_rows<32>(to + 32 * c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) __stcg(slot + (2 + 32 * c + e) * SR, o[e]);
                        }
                        tc::tc_fence_before();
                    }
                    if (PQ) ok = wait(kOFull + (s ^ 1), no[s ^ 1] & 1);  // the q that both streams share is free
                    ++no[s ^ 1];
                    tiles += x.nt;
                    u += x.nt;
                }
            } else if (owns) {
                const int n = own_n[s], rows = p.T * p.group;
                const bool live = r < rows;
                const int tok = live ? r / p.group : 0;
                OwnWalk k;
                if (n > 0) k.locate(p, coarse, share.own_at[s], lane);
                // the q of a segment into buffer `buf`, by the warps from q0 on
                auto fetch_q = [&](const OwnWalk& at, int buf, int q0) {
                    put_q<CT, D, PQ>(p, smem + s * TILE + buf * LY::OWN_BUF, kMostOwnRows, LY::OWN_LO, at.h, at.b * rows, 0, rows,
                                       quarter - q0, 4 - q0);
                    fence_proxy_async_smem();
                };
                auto fetch_next = [&](const OwnWalk& from, int to_buf) {
                    OwnWalk nx = from;
                    nx.next_segment(p, lane);
                    fetch_q(nx, to_buf, 1);
                };
                if (n > 0) fetch_q(k, 0, 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kStart));
                int buf = 0;
                bool fresh = true;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const bool end = k.tile + 1 == k.nt || i + 1 == n;
                    if (quarter > 0) {
                        // no row of its own: the next segment's q, at the piece's first tile (the buffer's last reader was the piece
                        // before, whose scores are done when this piece's are), behind its weights where another tile follows
                        const bool next_q = fresh && n - i > k.nt - k.tile;
                        ok = wait(kSFull + s, ns & 1);
                        if (!ok) break;
                        ++ns;
                        if (next_q && end) fetch_next(k, buf ^ 1);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kPFull + s));
                        if (next_q && !end) fetch_next(k, buf ^ 1);
                    } else {
                        if (fresh) ml = make_float2(kNone, 0.f);
                        ok = wait(kSFull + s, ns & 1);
                        if (!ok) break;
                        ++ns;
                        tc::tc_fence_after();
                        if constexpr (!I8) ml = take_tile<CT, D>(ts, to, k.L + tok + 1 - k.tile * TK, k.L + p.T - k.tile * TK, live, !fresh, ml, p.qscale);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kPFull + s));
                    }
                    fresh = end;
                    if (end) {
                        buf ^= 1;
                        if (quarter == 0) {
                            ok = wait(kOFull + s, no[s] & 1);
                            if (!ok) break;
                            tc::tc_fence_after();
                            float* slot = p.own_ws + (static_cast<size_t>(k.b) * p.Hkv + k.h + own_v[s]) * own_slot_floats(rows, D);
                            if (live) {
                                __stcg(slot + r, ml.x);
                                __stcg(slot + rows + r, ml.y);
                            }
                            float4* dst = reinterpret_cast<float4*>(slot + own_out_at(rows) + r * D);
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                wide::tmem_ld_rows<32>(to + 32 * c, o);
                                if (live) {
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        __stcg(dst + 8 * c + e, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                                }
                            }
                            tc::tc_fence_before();
                        }
                        ++no[s];
                    }
                    if (i + 1 < n) k.next(p, lane);
                }
                if (!ok) break;
                if (n == 0) {
                    ok = wait(kOFull + s, no[s] & 1);
                    ++no[s];
                }
                // (pieces that the other stream ended in this phase)
                if (own_n[s ^ 1] == 0) ++no[s ^ 1];
                if (own_n[s ^ 1] > 0) {
                    OwnWalk x;
                    x.locate(p, coarse, share.own_at[s ^ 1], lane);
#pragma unroll 1
                    for (int left = own_n[s ^ 1]; left > 0;) {
                        left -= x.nt - x.tile;
                        ++no[s ^ 1];
                        if (left > 0) x.next_segment(p, lane);
                    }
                }
            }
        }
    }
    if (warp == 0) {
        // ------------------------------------------------ for the join
        const PrefixSplit sp(p, first);
        const OwnSplit so(p, coarse);
        if (blockIdx.x == 0) write_seg_info(p, first, sp, lane);
        if (p.own) {
#pragma unroll 1
            for (int g = blockIdx.x; g < (p.B + 31) / 32; g += gridDim.x) {
                const int b = g * 32 + lane;
                const int n = b < p.B ? (own_rows(p, __ldcg(p.seq_lens + b)) + TK - 1) / TK : 0;
                int before = n;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int y = __shfl_up_sync(FULL, before, m);
                    if (lane >= m) before += y;
                }
                before += coarse[g] - n;
#pragma unroll 1
                for (int h = 0; h < p.Hkv && b < p.B; ++h) {
                    const long long u = static_cast<long long>(before) * p.Hkv + static_cast<long long>(h) * n;
                    p.own_info[static_cast<size_t>(b) * p.Hkv + h] = n > 0 ? make_int2(so.holder(u), so.holder(u + n - 1)) : make_int2(0, -1);
                }
            }
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (*abort_flag && warp == 0 && lane == 0) {
        // a bounded wait ran out: wait (long drain limit) for the copies in flight
#pragma unroll 1
        for (int i = max(0, issued - 2 * NV); i < issued; ++i) {
            const int t = i >> 1;
            if (!(i & 1) && t + NK < (issued + 1) / 2) continue;  // (a K slot that was filled again since)
            if (!(withhold && i == 0))
                mbar_wait_bounded(bar(kFull + ((i & 1) ? v_slot(t) : k_slot(t))), (i & 1) ? v_par(t) : k_par(t), p.err, kDrainLimitCycles);
        }
    }
    if (warp == 1) {
        if (lane == 0 && works) mbar_wait_bounded(bar(kDrain), 0u, p.err, kDrainLimitCycles);
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
    grid_dep_launch();
    if (!p.own) grid_dep_wait();  // the step before has ended when this grid has: the join reads both
}

template <typename CT, int D, bool PQ, bool I8>
PrefixKernel kernel_of() {
    return {reinterpret_cast<const void*>(&prefix_tc_kernel<CT, D, PQ, I8>), Layout<D, I8>::SMEM, I8 ? kThreadsI8 : kThreads,
            PQ ? TK : 2 * TK, 2 * TK, true};
}

}  // namespace ptc
}  // namespace ftd
