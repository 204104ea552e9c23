// ftd_prefix.cu -- attention to a shared prefix on CUDA cores, and the join of a row's parts
// (see ftd_prefix.cuh for the mathematics and the cut into work).
//
// The CUDA-core kernel serves fp32 caches, whose products the tensor cores would round, and
// every cache where the context asks for CUDA cores.  It is bound by fp32 FMAs: 4 D of them per
// query row and prefix row.  A block takes 64 query rows and walks tiles of 64 prefix rows: K, V and q lie in
// shared memory as fp32 rows of D + 4 floats (eight neighbouring rows' 16-byte words fall into different
// banks); a thread of the 16 x 16 keeps 4 rows x 4 keys of scores and 4 rows x D / 16 outputs in registers, so
// 16 products of a 16-byte step cost two loads.  Blocks of 16 rows, a warp for every two rows, serve up
// to 32 query rows, where 64-row blocks would compute mostly zeros; they are bound by shared-memory reads (each warp reads
// all of K and V).  fp32 tiles are copied asynchronously a tile ahead.
#include <cuda_runtime.h>

#include "ftd_internal.cuh"
#include "ftd_ops.cuh"
#include "ftd_prefix.cuh"

namespace ftd {
namespace {

constexpr int kCcThreads = 256;
constexpr int kCcTile = 64;  // prefix rows of a tile
constexpr float kNone = -1e30f;  // reference of a row that has seen nothing: finite, so 2^(s - m) needs no test

template <typename CT, int D, int RT>
struct CcLayout {
    static constexpr int ROW = D + 4;  // floats
    static constexpr int QS = RT * ROW, KV = kCcTile * ROW, PS = RT * (kCcTile + 4);
    static constexpr int FLOATS = QS + 4 * KV + PS;
    static constexpr int PLAN = (kMaxRowBlocks + 1) * 4 / 16 * 16 + 16;
    static constexpr int SMEM = PLAN + FLOATS * 4;
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void fma4(float& a, const float4& x, const float4& y) {
    a = fmaf(x.x, y.x, a);
    a = fmaf(x.y, y.y, a);
    a = fmaf(x.z, y.z, a);
    a = fmaf(x.w, y.w, a);
}

// Four elements of a cache row as fp32 (INT8: codes times the row's scale).
template <typename CT>
__device__ __forceinline__ float4 cache4(const unsigned char* row, int d, float scale) {
    if constexpr (std::is_same_v<CT, float>) {
        return __ldg(reinterpret_cast<const float4*>(row) + d / 4);
    } else if constexpr (std::is_same_v<CT, int8_t>) {
        const char4 c = __ldg(reinterpret_cast<const char4*>(row) + d / 4);
        return make_float4(c.x * scale, c.y * scale, c.z * scale, c.w * scale);
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(row) + d / 4);
        CT e[4];
        memcpy(e, &u, 8);
        return make_float4(static_cast<float>(e[0]), static_cast<float>(e[1]), static_cast<float>(e[2]), static_cast<float>(e[3]));
    }
}

// One tile's K and V rows into shared memory; rows past the prefix's seen end become zeros, so that what lies there
// (not a number, even) never meets a weight of zero.
template <typename CT, int D>
__device__ __forceinline__ void load_tile(const PrefixParams& p, int h, int t0, int n, float* Ks, float* Vs) {
    constexpr int ROW = D + 4, C4 = D / 4;
    for (int i = threadIdx.x; i < kCcTile * C4; i += kCcThreads) {
        const int r = i / C4, d = (i - r * C4) * 4;
        long long row = -1;
        if (r < n) {
            row = prefix_row(p, h, t0 + r);
            if (row < 0) atomicOr(p.err, kErrBadPage);
        }
        if constexpr (std::is_same_v<CT, float>) {
            const size_t o = row < 0 ? 0 : (static_cast<size_t>(row) * D + d) * 4;
            cp_async16(smem_addr(Ks + r * ROW + d), p.k + o, row < 0 ? 0 : 16);
            cp_async16(smem_addr(Vs + r * ROW + d), p.v + o, row < 0 ? 0 : 16);
        } else {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (row >= 0) {
                constexpr int EB = sizeof(CT);
                const bool i8 = std::is_same_v<CT, int8_t>;
                const size_t o = static_cast<size_t>(row) * D * EB;
                a = cache4<CT>(p.k + o, d, i8 ? __ldg(p.k_scales + row) : 1.f);
                b = cache4<CT>(p.v + o, d, i8 ? __ldg(p.v_scales + row) : 1.f);
            }
            *reinterpret_cast<float4*>(Ks + r * ROW + d) = a;
            *reinterpret_cast<float4*>(Vs + r * ROW + d) = b;
        }
    }
    cp_async_commit();
}

template <typename CT, int D, int RT>
__global__ void __launch_bounds__(kCcThreads, 1) prefix_cc_kernel(const PrefixParams p) {
    using LY = CcLayout<CT, D, RT>;
    constexpr int ROW = LY::ROW, PROW = kCcTile + 4;
    constexpr bool WIDE = RT == 64;           // else a warp for every two rows
    constexpr int NR = WIDE ? 4 : 2;          // rows of a thread
    constexpr int ND = WIDE ? D / 16 : D / 32;  // output dimensions of a thread
    static_assert(RT == 64 || RT == 16, "row blocks");
    extern __shared__ __align__(16) unsigned char smem[];
    int* first = reinterpret_cast<int*>(smem);
    float* Qs = reinterpret_cast<float*>(smem + LY::PLAN);
    float* KV = Qs + LY::QS;                  // two stages of K and V
    float* Ps = KV + 4 * LY::KV;
    const int tid = threadIdx.x, lane = tid & 31;
    // Runs beside the step's last blocks: the step was launched before and reads and writes nothing that this kernel writes,
    // and everything before the step has ended (its blocks wait for that before they let this grid start).
    build_prefix_plan(p, first, kCcTile);
    const PrefixSplit sp(p, first);
    if (blockIdx.x == 0) write_seg_info(p, first, sp, threadIdx.x, kCcThreads);
    const int w = blockIdx.x;
    long long u = sp.begin(w);
    const long long end = sp.begin(w + 1);
    // this thread's rows of the block, and its first key and dimension
    const int r0 = WIDE ? (tid >> 4) * 4 : (tid >> 5) * 2;
    const int kx = lane & 15;
    const int dhalf = WIDE ? 0 : (lane >> 4);
    while (u < end) {
        const PrefixCursor c = prefix_locate(u, first, p.row_blocks);
        const int nt = static_cast<int>(min(static_cast<long long>(c.nt - c.tile), end - u));
        __syncthreads();  // the buffers of the piece before are read
        // seen end of the block's longest row (the segment's tiles end with it)
        const int seen = prefix_block_seen(p, c.rb, lane);
        auto fetch = [&](int i) {
            const int t0 = (c.tile + i) * kCcTile;
            load_tile<CT, D>(p, c.h, t0, min(kCcTile, seen - t0), KV + (i & 1) * 2 * LY::KV, KV + (i & 1) * 2 * LY::KV + LY::KV);
        };
        fetch(0);
        for (int i = tid; i < RT * D; i += kCcThreads) {
            const int r = i / D, d = i - r * D, row = c.rb * RT + r;
            float x = 0.f;
            if (row < p.R) {
                x = ld_qkv(p.q, p.qkv_dtype, prefix_q_row(p, c.h, row) * D + d);
                if (p.bias) x += ld_qkv(p.bias, p.qkv_dtype, static_cast<size_t>(c.h * p.group + row % p.group) * D + d);
            }
            Qs[r * ROW + d] = x * p.qscale;
        }
        int lim[NR];
        float m[NR], l[NR], o[NR][ND];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int row = c.rb * RT + r0 + j;
            lim[j] = row < p.R ? prefix_seen(p, prefix_slot_of(p, row)) : 0;
            m[j] = kNone;
            l[j] = 0.f;
#pragma unroll
            for (int e = 0; e < ND; ++e) o[j][e] = 0.f;
        }
        for (int i = 0; i < nt; ++i) {
            if (i + 1 < nt) {
                fetch(i + 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncthreads();
            const float* Ks = KV + (i & 1) * 2 * LY::KV;
            const float* Vs = Ks + LY::KV;
            const int t0 = (c.tile + i) * kCcTile;
            // ---- scores of NR rows and keys kx + 16 j ----
            float s[NR][4];
#pragma unroll
            for (int a = 0; a < NR; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) s[a][b] = 0.f;
            constexpr int DN = WIDE ? D : D / 2;
#pragma unroll 4
            for (int d = 0; d < DN; d += 4) {
                const int dd = d + dhalf * DN;
                float4 qv[NR], kv[4];
#pragma unroll
                for (int a = 0; a < NR; ++a) qv[a] = load4(Qs + (r0 + a) * ROW + dd);
#pragma unroll
                for (int b = 0; b < 4; ++b) kv[b] = load4(Ks + (kx + 16 * b) * ROW + dd);
#pragma unroll
                for (int a = 0; a < NR; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) fma4(s[a][b], qv[a], kv[b]);
            }
            float alpha[NR];
#pragma unroll
            for (int a = 0; a < NR; ++a) {
                float top = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (!WIDE) s[a][b] += __shfl_xor_sync(0xffffffffu, s[a][b], 16);
                    if (t0 + kx + 16 * b >= lim[a]) s[a][b] = -INFINITY;
                    top = fmaxf(top, s[a][b]);
                }
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float mn = fmaxf(m[a], top);
                alpha[a] = exp2f(m[a] - mn);
                m[a] = mn;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float e = exp2f(s[a][b] - mn);
                    sum += e;
                    if (WIDE || dhalf == 0) Ps[(r0 + a) * PROW + kx + 16 * b] = e;
                }
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[a] = l[a] * alpha[a] + sum;
#pragma unroll
                for (int e = 0; e < ND; ++e) o[a][e] *= alpha[a];
            }
            __syncwarp();  // a row's weights are written and read by one warp
            // ---- o += p V ----
#pragma unroll 4
            for (int k = 0; k < kCcTile; k += 4) {
                float4 pv[NR];
#pragma unroll
                for (int a = 0; a < NR; ++a) pv[a] = load4(Ps + (r0 + a) * PROW + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float* vr = Vs + (k + kk) * ROW;
                    float vv[ND];
                    if constexpr (WIDE) {
#pragma unroll
                        for (int e = 0; e < ND; e += 4) *reinterpret_cast<float4*>(vv + e) = load4(vr + kx * 4 + 16 * e);
                    } else if constexpr (ND == 4) {
                        *reinterpret_cast<float4*>(vv) = load4(vr + lane * 4);
                    } else {
                        *reinterpret_cast<float2*>(vv) = *reinterpret_cast<const float2*>(vr + lane * 2);
                    }
#pragma unroll
                    for (int a = 0; a < NR; ++a) {
                        const float pk = kk == 0 ? pv[a].x : kk == 1 ? pv[a].y : kk == 2 ? pv[a].z : pv[a].w;
#pragma unroll
                        for (int e = 0; e < ND; ++e) o[a][e] = fmaf(pk, vv[e], o[a][e]);
                    }
                }
            }
            __syncthreads();  // the stage may be filled again
        }
        // ---- the piece's partial ----
        float* slot = p.ws + static_cast<size_t>(c.h * p.row_blocks + c.rb + w) * prefix_slot_floats(RT, D);
#pragma unroll
        for (int a = 0; a < NR; ++a) {
            if (kx == 0 && dhalf == 0) {
                slot[r0 + a] = m[a];
                slot[RT + r0 + a] = l[a];
            }
        }
#pragma unroll
        for (int e = 0; e < ND; ++e) {
            const int d = WIDE ? kx * 4 + 16 * (e & ~3) + (e & 3) : lane * ND + e;
            float* dst = slot + (2 + d) * RT + r0;
            if constexpr (WIDE) *reinterpret_cast<float4*>(dst) = make_float4(o[0][e], o[1][e], o[2][e], o[3][e]);
            else *reinterpret_cast<float2*>(dst) = make_float2(o[0][e], o[1][e]);
        }
        u += nt;
    }
    grid_dep_launch();
    grid_dep_wait();  // the step before has ended when this grid has: the join reads both
}

// A block joins 32 query rows of a kv head (all of one row block, so 16 where those have no more) and 32 outputs of each: a
// lane per row, so a partial's loads are whole lines of neighbouring rows, and a warp for 16 outputs of every fourth partial;
// the sums then go through shared memory to meet each other and the row's own output and leave as rows. It is bound by the
// chain of dependent loads: with all outputs and every partial in one warp's turn (a quarter of the blocks), 20 partials of 256
// rows took 22 us.
constexpr int kJoinRows = 32, kJoinThreads = 256, kJoinOut = 32, kJoinParts = 4;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixParams p) {
    constexpr int N = kJoinOut * kJoinParts / (kJoinThreads / 32);  // outputs of a thread
    static_assert(N == 16, "two warps for the outputs");
    __shared__ float acc_s[kJoinParts][kJoinRows][kJoinOut + 1];
    __shared__ float M_s[kJoinParts][kJoinRows], S_s[kJoinParts][kJoinRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp >> 1, d_at = (warp & 1) * N;
    const int d_block = static_cast<int>(blockIdx.x) % (D / kJoinOut) * kJoinOut, hr = static_cast<int>(blockIdx.x) / (D / kJoinOut);
    const int h = hr % p.Hkv, row0 = hr / p.Hkv * min(kJoinRows, p.block_rows), d0 = d_block + d_at;
    grid_dep_wait();
    grid_dep_launch();
    const int rb = row0 / p.block_rows;
    const bool twice = prefix_twice(p, rb);
    const int half = p.slot_rows / 2, r = row0 - rb * p.block_rows + lane;
    const int2 range = __ldcg(p.seg_info + h * p.row_blocks + rb);
    const size_t stride = prefix_slot_floats(p.slot_rows, D);
    const float* slot = p.ws + static_cast<size_t>(h * p.row_blocks + rb + range.x) * stride;
    const int n = r < p.block_rows ? (range.y - range.x + 1) * (twice ? 2 : 1) : 0;
    float M = kNone, S = 0.f, acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
#pragma unroll 2
    for (int k = part; k < n; k += kJoinParts) {
        const float* s = slot + (twice ? k >> 1 : k) * stride + (twice ? r + (k & 1) * half : r);
        const float mk = __ldcg(s), lk = __ldcg(s + p.slot_rows);
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = __ldcg(s + (2 + d0 + e) * p.slot_rows);
        if (lk == 0.f && mk <= kNone) continue;  // a piece that the row saw nothing of
        const float mn = fmaxf(M, mk), a = exp2f(M - mn), f = exp2f(mk - mn);
        S = S * a + lk * f;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = acc[e] * a + o[e] * f;
        M = mn;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) acc_s[part][lane][d_at + e] = acc[e];
    if (!(warp & 1)) {
        M_s[part][lane] = M;
        S_s[part][lane] = S;
    }
    __syncthreads();
    // ---- with the rows' own parts ----
    for (int i = threadIdx.x; i < kJoinRows * (kJoinOut / 4); i += kJoinThreads) {
        const int rr = i / (kJoinOut / 4), c = (i - rr * (kJoinOut / 4)) * 4, d = d_block + c, row = row0 + rr;
        if (row >= p.R || row0 - rb * p.block_rows + rr >= p.block_rows) continue;
        const int b = prefix_slot_of(p, row), L = __ldcg(p.seq_lens + b);
        const size_t at = prefix_q_row(p, h, row) * D + d;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (L >= 0 && L <= p.Lmax - p.T) {
            const int per = p.T * p.group, r_own = row - b * per;
            float M = kNone, S = 0.f;
            // a part without weight leaves the sums as they are
            auto add = [&](float m, float l, float o_l, const float4& o) {
                const float mn = fmaxf(M, m), f = exp2f(m - mn) * o_l, a = S == 0.f ? 0.f : exp2f(M - mn);
                S = S * a + exp2f(m - mn) * l;
                x = make_float4(x.x * a + o.x * f, x.y * a + o.y * f, x.z * a + o.z * f, x.w * a + o.w * f);
                M = mn;
            };
#pragma unroll
            for (int k = 0; k < kJoinParts; ++k) {
                const float* o = &acc_s[k][rr][c];
                if (S_s[k][rr] != 0.f || M_s[k][rr] > kNone) add(M_s[k][rr], S_s[k][rr], 1.f, make_float4(o[0], o[1], o[2], o[3]));
            }
            if (p.own) {
                const int2 v = __ldcg(p.own_info + static_cast<size_t>(b) * p.Hkv + h);
                const size_t step = own_slot_floats(per, D);
                const float* s = p.own_ws + (static_cast<size_t>(b) * p.Hkv + h + v.x) * step;
#pragma unroll 2
                for (int k = v.x; k <= v.y; ++k, s += step) {
                    const float m = __ldcg(s + r_own), l = __ldcg(s + per + r_own);
                    const float4 o = __ldcg(reinterpret_cast<const float4*>(s + own_out_at(per) + r_own * D + d));
                    if (l == 0.f && m <= kNone) continue;  // tokens that came later than the row
                    add(m, l, 1.f, o);
                }
            } else {
                const float2 own = __ldcg(p.own_ml + (static_cast<size_t>(b) * p.Hkv + h) * per + r_own);
                const float l = 1.f / own.y;
                add(own.x, l, l, __ldcg(reinterpret_cast<const float4*>(p.own_o + at)));
            }
            const float inv = 1.f / S;
            x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        }
        st_out4(p.out, at, x.x, x.y, x.z, x.w, p.out_dtype);
    }
}

template <typename CT, int D>
PrefixKernel pick_cc(int R) {
    if (R <= 32)
        return {reinterpret_cast<const void*>(&prefix_cc_kernel<CT, D, 16>), CcLayout<CT, D, 16>::SMEM, kCcThreads, 16, 16, false};
    return {reinterpret_cast<const void*>(&prefix_cc_kernel<CT, D, 64>), CcLayout<CT, D, 64>::SMEM, kCcThreads, 64, 64, false};
}

}  // namespace

PrefixKernel select_prefix_cc(int cache_dt, int D, int R) {
    switch (cache_dt) {
        case kF32: return D == 64 ? pick_cc<float, 64>(R) : pick_cc<float, 128>(R);
        case kF16: return D == 64 ? pick_cc<__half, 64>(R) : pick_cc<__half, 128>(R);
        case kBF16: return D == 64 ? pick_cc<__nv_bfloat16, 64>(R) : pick_cc<__nv_bfloat16, 128>(R);
        default: return D == 64 ? pick_cc<int8_t, 64>(R) : pick_cc<int8_t, 128>(R);
    }
}

cudaError_t launch_prefix_join(PrefixParams p, cudaStream_t stream) {
    const int per = p.block_rows < kJoinRows ? p.block_rows : kJoinRows;  // rows of a block
    const dim3 grid(static_cast<unsigned>((p.R + per - 1) / per) * static_cast<unsigned>(p.Hkv) * static_cast<unsigned>(p.D / kJoinOut));
    void* args[] = {&p};
    const void* fn = p.D == 64 ? reinterpret_cast<const void*>(&prefix_join_kernel<64>)
                               : reinterpret_cast<const void*>(&prefix_join_kernel<128>);
    return launch_pdl(fn, grid, kJoinThreads, 0, args, stream);
}

}  // namespace ftd
