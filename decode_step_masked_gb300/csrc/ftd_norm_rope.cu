// ftd_norm_rope.cu -- norms of the query and key heads and rotary positions in one pass, with the
// fused QKV bias, into dense rows or into the cache by a slot map (ftd_norm_rope_qkv).
//
// For every token and query or key head, x = in + bias:
//   y_e = x_e / sqrt(mean(x^2) + eps) * (w_e + offset)      (when the head has a weight)
//   (a, b) -> (a cos w - b sin w, b cos w + a sin w)        for the pairs of the rotary part,
// in fp32, then one rounding: to the qkv type, or for keys and values that go to the cache, to its
// type; an INT8 cache takes codes rint(y / scale), scale = absmax / 127 of the head's row, as the
// step's own append does.  Angles are ftd_rope.cu's: exact fractions of a turn.
//
// Bound: each head is read and written once; the norm's sum needs the whole head before the first
// product, so a head stays in registers: D / 16 neighbouring lanes hold 16 elements each (eight
// pairs) and exchange their sums in two or three shuffles.  A lane keeps its head and walks the tokens,
// its bias and weights in registers as fp32 (read anew for every token they cost many instructions, and
// the kernel was bound by those); the next token's loads go out before the present one is
// worked on.  A block takes a tile of tokens and forms their cosines, sines and cache rows once in shared memory.
// Measured: 16381 tokens of 64 + 2 * 8 heads, bf16, into pages, 147 us (67 % of the copy peak; with bias and weights read for each
// token 169, in registers 162, with packed arithmetic and blocks without idle lanes 147): loads in flight bound it, 15 warps
// an SM with one token ahead.  4001 tokens of 32 + 2 * 32 heads into an INT8 cache 54 us (with a quotient for every code 70).
#include <cuda_runtime.h>

#include <algorithm>

#include "ftd_internal.cuh"
#include "ftd_ops.cuh"
#include "ftd_rope.cuh"

namespace ftd {
namespace {

constexpr int kNormThreads = 256;   // most threads of a block
constexpr int kNormTile = 16;         // most tokens of a tile

// Two fp32 values that the packed forms take at once (a lane's arithmetic is most of its instructions).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
template <int VEC>
__device__ __forceinline__ void add_to(float (&y)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 1) y[0] += b[0];
    else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) unpack2(add2(pack2(y[e], y[e + 1]), pack2(b[e], b[e + 1])), y[e], y[e + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ uint64_t squares(const float (&y)[VEC], uint64_t sum) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
        const uint64_t v = pack2(y[e], VEC == 1 ? 0.f : y[(e + 1) % VEC]);
        sum = fma2(v, v, sum);
    }
    return sum;
}
template <int VEC>
__device__ __forceinline__ void weigh(float (&y)[VEC], float r, const float (&w)[VEC]) {
    if constexpr (VEC == 1) y[0] = y[0] * r * w[0];
    else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
            unpack2(mul2(mul2(pack2(y[e], y[e + 1]), pack2(r, r)), pack2(w[e], w[e + 1])), y[e], y[e + 1]);
    }
}
// (a, b) -> (a c - b s, b c + a s); b s takes its sign in the last step, which is not packed
template <int VEC>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC], bool adjacent) {
    if constexpr (VEC == 1) {
        turn_pairs<VEC>(a, b, c, s, adjacent);
    } else if (adjacent) {
        turn_pairs<VEC>(a, b, c, s, true);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const uint64_t c2 = pack2(c[e], c[e + 1]), s2 = pack2(s[e], s[e + 1]);
            const uint64_t a2 = pack2(a[e], a[e + 1]), b2 = pack2(b[e], b[e + 1]);
            float t0, t1;
            unpack2(mul2(b2, s2), t0, t1);
            unpack2(fma2(a2, s2, mul2(b2, c2)), b[e], b[e + 1]);
            a[e] = fmaf(a[e], c[e], -t0);
            a[e + 1] = fmaf(a[e + 1], c[e + 1], -t1);
        }
    }
}

// VEC fp32 values to elements i .. of an array of type dt (kF32, kF16, kBF16), rounded to nearest even.
template <int VEC>
__device__ __forceinline__ void st_vals(void* base, long long i, const float (&x)[VEC], int dt) {
    if (dt == kF32) {
        float* q = static_cast<float*>(base) + i;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int e = 0; e < VEC; e += 4) *reinterpret_cast<float4*>(q + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else {
            Chunk<float, VEC> c;
#pragma unroll
            for (int e = 0; e < VEC; ++e) c.e[e] = x[e];
            c.store(q);
        }
    } else if (dt == kF16) {
        Chunk<__half, VEC> c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) c.e[e] = __float2half_rn(x[e]);
        c.store(static_cast<__half*>(base) + i);
    } else {
        Chunk<__nv_bfloat16, VEC> c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) c.e[e] = __float2bfloat16_rn(x[e]);
        c.store(static_cast<__nv_bfloat16*>(base) + i);
    }
}

__device__ __noinline__ uint32_t code_by_quotient(float x, float scale) {
    return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(x, scale))))) & 0xffu;
}

// VEC codes rint(x / scale) of a row with the given scale (inv: its reciprocal) to bytes i ..  x inv differs from the
// quotient by at most 127 * 2^-22, so it rounds to the same code unless it lies that near to a half; then, one value of
// thousands, and for values that are no numbers, the quotients themselves are formed.  |x / scale| < 127.5, so the code is
// the low byte of x inv + 1.5 * 2^23.
template <int VEC>
__device__ __forceinline__ void st_codes(unsigned char* base, long long i, const float (&x)[VEC], float scale, float inv) {
    constexpr float kShift = 12582912.f;
    float m[VEC], off = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        m[e] = fmaf(x[e], inv, kShift);
        const float d = fabsf(fmaf(x[e], inv, kShift - m[e]));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(off) : "f"(d));
    }
    uint32_t w[(VEC + 3) / 4] = {};
    if (off < 0.4999f) {
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                w[e / 4] = __byte_perm(__byte_perm(__float_as_uint(m[e]), __float_as_uint(m[e + 1]), 0x0040),
                                       __byte_perm(__float_as_uint(m[e + 2]), __float_as_uint(m[e + 3]), 0x0040), 0x5410);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[0] |= (__float_as_uint(m[e]) & 0xffu) << (8 * e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e / 4] |= code_by_quotient(x[e], scale) << (8 * (e % 4));
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(base + i) = make_uint2(w[0], w[1]);
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(base + i) = w[0];
    else if constexpr (VEC == 2) *reinterpret_cast<unsigned short*>(base + i) = static_cast<unsigned short>(w[0]);
    else base[i] = static_cast<unsigned char>(w[0]);
}

// LPH: lanes of a head (D / 16); VEC: elements per access.
template <typename T, int LPH, int VEC>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int D = 16 * LPH;
    constexpr int NU = 8 / VEC;       // units of a lane: two runs of VEC elements, the pairs of one or neighbours
    constexpr int ITEMS = LPH * NU;   // units of a head
    __shared__ __align__(16) float cs[2][kNormTile][64], sn[2][kNormTile][64];
    __shared__ long long crow[2][kNormTile];  // cache row of head 0 of a token, -1: none
    __shared__ uint64_t step[64];
    __shared__ int axis[64];
    const int lane = threadIdx.x & 31, hl = lane & (LPH - 1);
    const int half = p.R >> 1;
    const int turning = half / VEC;   // units of a head that turn
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        step[i] = p.step[i];
        axis[i] = p.axis[i];
    }
    // this lane's head (the last block's idle lanes follow the last head, without storing)
    const int at = blockIdx.y * p.heads_per_block + static_cast<int>(threadIdx.x) / LPH;
    const bool active = at < p.heads && static_cast<int>(threadIdx.x) / LPH < p.heads_per_block;
    const int head = min(at, p.heads - 1);
    const bool isq = head < p.Hq, isk = !isq && head < p.Hq + p.Hkv, turns = isq || isk;
    const int kvh = head - p.Hq - (isk ? 0 : p.Hkv);
    const bool neighbours = p.adjacent || !turns;
    const T* src = isq ? static_cast<const T*>(p.q) + static_cast<long long>(head) * D
                       : static_cast<const T*>(isk ? p.k : p.v) + static_cast<long long>(kvh) * D;
    const long long stride = isq ? p.q_stride : p.kv_stride;
    const void* weight = isq ? p.qw : isk ? p.kw : nullptr;
    const bool to_cache = p.slots && !isq;
    int at_e[2 * NU];  // elements of the head where this lane's runs begin
#pragma unroll
    for (int j = 0; j < NU; ++j) unit_at<VEC>(j * LPH + hl, turning, half, neighbours, at_e[2 * j], at_e[2 * j + 1]);
    float bias[2 * NU][VEC], wt[2 * NU][VEC];
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
#pragma unroll
    for (int j = 0; j < 2 * NU; ++j) {
        Chunk<T, VEC> c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) bias[j][e] = wt[j][e] = 0.f;
        if (p.bias) {
            c.load(static_cast<const T*>(p.bias) + static_cast<long long>(head) * D + at_e[j]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) bias[j][e] = to_f<T>(c.e[e]);
        }
        if (weight) {
            c.load(static_cast<const T*>(weight) + at_e[j]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) wt[j][e] = to_f<T>(c.e[e]) + p.offset;
        }
    }
    const int inv_half = half ? (65535 + half) / half : 0;  // i / half = (i * inv_half) >> 16 for i < 64 kNormTile
    int buf = 0;
    for (long long t0 = static_cast<long long>(blockIdx.x) * p.tile; t0 < p.n; t0 += static_cast<long long>(gridDim.x) * p.tile) {
        const int nt = static_cast<int>(min(static_cast<long long>(p.tile), p.n - t0));
        Chunk<T, VEC> x[2 * NU];
        auto load = [&](int tok) {
            const T* row = src + (t0 + tok) * stride;
#pragma unroll
            for (int j = 0; j < 2 * NU; ++j) x[j].load(row + at_e[j]);
        };
        load(0);
        for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
            const int tok = (i * inv_half) >> 16, pair = i - tok * half;
            const int pos = __ldcg(p.pos + static_cast<long long>(axis[pair]) * p.n + t0 + tok);
            float s, c;
            turn_sincos(pos, step[pair], &s, &c);
            cs[buf][tok][table_at<VEC>(pair, ITEMS)] = c;
            sn[buf][tok][table_at<VEC>(pair, ITEMS)] = s;
        }
        if (p.slots && threadIdx.x < nt) {
            const int s = __ldcg(p.slots + t0 + threadIdx.x);
            long long r = -1;
            if (s >= 0 && s < p.n_slots) r = static_cast<long long>(s / p.unit) * p.Hkv * p.unit + s % p.unit;
            else if (s >= 0 && blockIdx.y == 0) atomicOr(p.err, kErrBadPage);
            crow[buf][threadIdx.x] = r;
        }
        __syncthreads();  // (the other buffer is written only after every thread has passed here again)
#pragma unroll 1
        for (int tok = 0; tok < nt; ++tok) {
            float y[2 * NU][VEC];
#pragma unroll
            for (int j = 0; j < 2 * NU; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[j][e] = to_f<T>(x[j].e[e]);
#pragma unroll
            for (int j = 0; j < 2 * NU; ++j) add_to<VEC>(y[j], bias[j]);
            if (tok + 1 < nt) load(tok + 1);
            if (weight) {  // (a head's lanes come here together, and so do all lanes of the mask)
                uint64_t two = 0;
#pragma unroll
                for (int j = 0; j < 2 * NU; ++j) two = squares<VEC>(y[j], two);
                float ss, other;
                unpack2(two, ss, other);
                ss += other;
                const unsigned lanes = ((1u << LPH) - 1u) << (lane & ~(LPH - 1));
#pragma unroll
                for (int m = LPH / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(lanes, ss, m);
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int j = 0; j < 2 * NU; ++j) weigh<VEC>(y[j], r, wt[j]);
            }
            if (turns) {
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    const int unit = j * LPH + hl;
                    if (unit >= turning) continue;
                    float c[VEC], s[VEC];
                    if constexpr (VEC < 4) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            c[e] = cs[buf][tok][unit * VEC + e];
                            s[e] = sn[buf][tok][unit * VEC + e];
                        }
                    } else {
#pragma unroll
                        for (int q4 = 0; q4 < VEC / 4; ++q4) {
                            *reinterpret_cast<float4*>(c + 4 * q4) =
                                *reinterpret_cast<const float4*>(&cs[buf][tok][(q4 * ITEMS + unit) * 4]);
                            *reinterpret_cast<float4*>(s + 4 * q4) =
                                *reinterpret_cast<const float4*>(&sn[buf][tok][(q4 * ITEMS + unit) * 4]);
                        }
                    }
                    turn<VEC>(y[2 * j], y[2 * j + 1], c, s, p.adjacent);
                }
            }
            // where the row goes
            if (!to_cache) {
                if (!active) continue;
                const long long t = t0 + tok;
                T* dst;
                if (isq) dst = static_cast<T*>(p.qo) + (t * p.Hq + head) * D;
                else dst = static_cast<T*>(isk ? p.ko : p.vo) + (t * p.Hkv + kvh) * D;
#pragma unroll
                for (int j = 0; j < 2 * NU; ++j) {
                    Chunk<T, VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o.e[e] = from_f<T>(y[j][e]);
                    o.store(dst + at_e[j]);
                }
            } else {
                const long long r0 = crow[buf][tok];
                const long long row = r0 + static_cast<long long>(kvh) * p.unit;
                unsigned char* cache = isk ? p.k_cache : p.v_cache;
                float amax = 0.f;
                if (p.cache_dt == kCacheI8) {
#pragma unroll
                    for (int j = 0; j < 2 * NU; ++j)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(y[j][e]));
                    // (a head's lanes come here together, so only they take part)
                    const unsigned lanes = ((1u << LPH) - 1u) << (lane & ~(LPH - 1));
#pragma unroll
                    for (int m = LPH / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, m));
                }
                if (!active || r0 < 0) continue;
                const float scale = amax == 0.f ? 1.f : __fdiv_rn(amax, 127.f);
                const float inv = __frcp_rn(scale);
                if (p.cache_dt == kCacheI8 && hl == 0) (isk ? p.k_scales : p.v_scales)[row] = scale;
#pragma unroll
                for (int j = 0; j < 2 * NU; ++j) {
                    if (p.cache_dt == kCacheI8) st_codes<VEC>(cache, row * D + at_e[j], y[j], scale, inv);
                    else st_vals<VEC>(cache, row * D + at_e[j], y[j], p.cache_dt);
                }
            }
        }
        buf ^= 1;
    }
}

template <typename T, int LPH>
const void* pick(int vec) {
    if constexpr (sizeof(T) == 2)
        if (vec == 8) return reinterpret_cast<const void*>(&norm_rope_kernel<T, LPH, 8>);
    return vec == 4   ? reinterpret_cast<const void*>(&norm_rope_kernel<T, LPH, 4>)
           : vec == 2 ? reinterpret_cast<const void*>(&norm_rope_kernel<T, LPH, 2>)
                      : reinterpret_cast<const void*>(&norm_rope_kernel<T, LPH, 1>);
}
template <typename T>
const void* pick(int D, int vec) {
    return D == 64 ? pick<T, 4>(vec) : pick<T, 8>(vec);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int vec, int sms, cudaStream_t stream) {
    const void* fn = p.dt == kF32 ? pick<float>(p.D, vec) : p.dt == kF16 ? pick<__half>(p.D, vec) : pick<__nv_bfloat16>(p.D, vec);
    // Heads of a block: as many as its threads take, whole warps of them and evenly, so that few lanes idle (at most
    // twice the blocks for that); one warp's where there are few tokens.
    const int lph = p.D / 16, per_warp = 32 / lph;
    const int most = p.n * p.heads < static_cast<long long>(sms) * kNormThreads / lph ? per_warp : kNormThreads / lph;
    int gy = (p.heads + most - 1) / most;
    auto heads_of = [&](int g) { return ((p.heads + g - 1) / g + per_warp - 1) / per_warp * per_warp; };
    for (int g = gy + 1, until = 2 * gy; g <= until; ++g)
        if (g * heads_of(g) < gy * heads_of(gy)) gy = g;
    p.heads_per_block = heads_of(gy);
    gy = (p.heads + p.heads_per_block - 1) / p.heads_per_block;
    // Tokens of a tile: fewer where that would leave an SM fewer than two blocks.  Three times as many blocks as are resident at
    // once (two of 256 threads an SM) walk the tiles, each as many: bias and weights are loaded three times, but a late block
    // holds up less.  As many as are resident / three times as many, us, with the L2 flushed: 16381 tokens of 64 + 2 * 8 heads into bf16 pages
    // 150 / 154 and dense 146 / 150, 4001 of them 52 / 54, 4001 tokens of 32 + 2 * 32 heads into an INT8 cache 66 / 62.
    p.tile = kNormTile;
    while (p.tile > 1 && (p.n + p.tile - 1) / p.tile * gy < 2LL * sms) p.tile >>= 1;
    const long long tiles = (p.n + p.tile - 1) / p.tile;
    const long long at_once = std::max(1LL, 6LL * kNormThreads / (p.heads_per_block * lph) * sms / gy);
    const long long each = (tiles + at_once - 1) / at_once, cap = (tiles + each - 1) / each;
    const dim3 grid(static_cast<unsigned>(tiles < cap ? tiles : cap), static_cast<unsigned>(gy));
    void* args[] = {&p};
    return launch_pdl(fn, grid, p.heads_per_block * lph, 0, args, stream);
}

}  // namespace ftd
