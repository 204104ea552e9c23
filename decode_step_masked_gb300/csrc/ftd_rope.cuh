// ftd_rope.cuh -- what the kernels that turn heads by positions share (ftd_rope.cu,
// ftd_norm_rope.cu): element access, angles, pairs, and the cut of a call into blocks.
#pragma once

#include <type_traits>

#include "ftd_ops.cuh"

namespace ftd {

template <typename T>
__device__ __forceinline__ float to_f(T x) {
    if constexpr (std::is_same_v<T, float>) return x;
    else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
    else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x) {
    if constexpr (std::is_same_v<T, float>) return x;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

// VEC consecutive elements, as one access of 2 to 16 bytes.
template <typename T, int VEC>
struct Chunk {
    static constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    using W = std::conditional_t<BYTES == 16, uint4,
                                 std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, uint32_t, T>>>;
    alignas(BYTES) T e[VEC];
    __device__ __forceinline__ void load(const T* p) { *reinterpret_cast<W*>(e) = *reinterpret_cast<const W*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<W*>(p) = *reinterpret_cast<const W*>(e); }
};

// Place of pair p's value in a token's table: the quads of an item's pairs lie a whole
// row of items apart, so the threads of a quarter-warp read consecutive 16-byte words.
template <int VEC>
__device__ __forceinline__ int table_at(int pair, int items) {
    if constexpr (VEC < 4) return pair;
    return (((pair % VEC) >> 2) * items + pair / VEC) * 4 + (pair & 3);
}

// Sine and cosine of the angle of position pos, for a pair whose step is in units of 2^-64 turns.
__device__ __forceinline__ void turn_sincos(int pos, uint64_t step, float* s, float* c) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(pos)) * step;
    // half turns in [-1, 1): the wrapped angle over pi
    const float x = __ll2float_rn(static_cast<long long>(turn)) * 1.0842021724855044e-19f;  // 2^-63
    sincospif(x, s, c);
}

// First elements of a unit's two chunks: the two members of its pairs, or neighbours (adjacent
// pairs, value heads, and the elements behind the rotary part).
template <int VEC>
__device__ __forceinline__ void unit_at(int unit, int turning, int half, bool neighbours, int& ea, int& eb) {
    if (neighbours || unit >= turning) {
        ea = 2 * unit * VEC;
        eb = ea + VEC;
    } else {
        ea = unit * VEC;
        eb = half + unit * VEC;
    }
}

// Turns a unit's VEC pairs.
template <int VEC>
__device__ __forceinline__ void turn_pairs(float (&xa)[VEC], float (&xb)[VEC], const float (&c)[VEC], const float (&s)[VEC],
                                           bool adjacent) {
    if (adjacent) {
        // pair e: elements 2e and 2e + 1 of the unit's 2 VEC
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float& y0 = 2 * e < VEC ? xa[(2 * e) % VEC] : xb[(2 * e) % VEC];
            float& y1 = 2 * e + 1 < VEC ? xa[(2 * e + 1) % VEC] : xb[(2 * e + 1) % VEC];
            const float u0 = y0, u1 = y1;
            y0 = u0 * c[e] - u1 * s[e];
            y1 = u1 * c[e] + u0 * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float u0 = xa[e], u1 = xb[e];
            xa[e] = u0 * c[e] - u1 * s[e];
            xb[e] = u1 * c[e] + u0 * s[e];
        }
    }
}

// Tokens of a tile and heads of a block, for per_token items a token and tiles of at most max_tile
// tokens and max_items items: large calls get tiles up to that and fewer tokens where that would give an SM
// fewer than four blocks; calls with fewer tiles than SMs spread their heads over enough blocks to
// reach every SM (at least 8 heads each).
inline void plan_rope(RopeParams& p, int per_token, int max_tile, int max_items, int sms) {
    p.tile = max_tile;
    while (p.tile > 1 && (p.tile * per_token > max_items || p.n < 4LL * p.tile * sms)) p.tile >>= 1;
    const long long tiles = (p.n + p.tile - 1) / p.tile;
    const long long split = tiles >= sms ? 1 : sms / tiles;
    p.heads_per_block = static_cast<int>((p.heads + split - 1) / split);
    if (p.heads_per_block < 8) p.heads_per_block = p.heads < 8 ? p.heads : 8;
    if (p.heads_per_block > 4096) p.heads_per_block = 4096;
    const int gy = (p.heads + p.heads_per_block - 1) / p.heads_per_block;
    // ceil(2^32 / H): hh / H as the high half of a product, exact for hh < tile * H <= 16 * 2^12
    for (int last = 0; last < 2; ++last) {
        const uint32_t h = static_cast<uint32_t>(last ? p.heads - (gy - 1) * p.heads_per_block : p.heads_per_block);
        p.div_h[last] = h == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + h - 1) / h);
    }
}

}  // namespace ftd
