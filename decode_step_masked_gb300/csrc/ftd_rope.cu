// ftd_rope.cu -- rotary positions with one to four axes for the query and key heads
// of a step's or a prompt's tokens, with the fused QKV bias (ftd_rope_qkv).
//
// Pair i of a head, elements (i, i + R/2) or (2i, 2i + 1), turns by the angle
// w = pos[axis(i)][token] * f_i:
//   a' = a cos w - b sin w,   b' = b cos w + a sin w.
// Far positions lose their angle in fp32 (position 10^6 times a step of 1 radian
// leaves 2^-4 radians), so the angle is kept as a fraction of a turn in 64-bit
// integers: step_i = f_i / 2 pi mod 1 in units of 2^-64, and pos * step_i mod 2^64
// is the wrapped angle exactly, for any int32 position of either sign, with one
// integer multiplication; only the wrapped fraction is rounded to fp32 for sincospi.
//
// Bound: each head is read and written once.  A block takes a tile of tokens, forms
// each token's cosines and sines once in shared memory and applies them to all its heads, 16 bytes
// (less where runs of pairs or addresses want it) of both members of eight (four in fp32)
// pairs per thread and item, two items in flight.  Small calls spread one token's heads over several
// blocks instead.
// Measured: 16381 tokens of 64 + 2 x 8 bf16 heads of 128 from a fused projection
// 111 us, 6.0 TB/s (tiles of 1280 / 2560 / 5120 / 10240 items 123 / 115 / 111 / 121 us; one / two / four
// items in flight 117 / 116 / 125 us; blocks that keep one group of heads and walk the tokens, with the
// bias in registers, 119 us at best); eight tokens of 32 + 32 heads 1.7 us a call in a graph.
// Narrower accesses, where R / 2 or an address is no multiple of 16 bytes, cost as much more as they
// are more: that prompt with R 120 / 52 / 22 (accesses of 8 / 4 / 2 bytes) 142 / 205 / 346 us, with
// rows one element past a boundary 348.
#include <cuda_runtime.h>

#include "ftd_internal.cuh"
#include "ftd_ops.cuh"

namespace ftd {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTile = 16;         // most tokens of a tile
constexpr int kRopeTileItems = 5120;  // most items of a large call's tile

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

template <typename T, int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int U = 2;
    __shared__ __align__(16) float cs[2][kRopeTile][64], sn[2][kRopeTile][64];
    const int D = p.D, half = p.R >> 1;
    const int items = D / (2 * VEC);          // items per head (a power of two)
    const int ishift = 31 - __clz(items);
    const int turning = half / VEC;           // items of a head that turn
    const int tile = p.tile;
    // this block's heads: [h0, h0 + H) of Hq query, Hkv key and (when present) Hkv value heads
    const int h0 = blockIdx.y * p.heads_per_block;
    const int H = min(p.heads_per_block, p.heads - h0);
    // the pairs' steps and axes: read from the parameters once (a warp's divergent reads of
    // constant memory go one address at a time)
    __shared__ uint64_t step[64];
    __shared__ int axis[64];
    for (int i = threadIdx.x; i < half; i += kRopeThreads) {
        step[i] = p.step[i];
        axis[i] = p.axis[i];
    }
    const uint32_t div = p.div_h[blockIdx.y == gridDim.y - 1];
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    int buf = 0;
    for (long long t0 = static_cast<long long>(blockIdx.x) * tile; t0 < p.n; t0 += static_cast<long long>(gridDim.x) * tile) {
        const int nt = static_cast<int>(min(static_cast<long long>(tile), p.n - t0));
        for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
            const int tok = i / half, pair = i - tok * half;
            const int pos = __ldcg(p.pos + static_cast<long long>(axis[pair]) * p.n + t0 + tok);
            const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(pos)) * step[pair];
            // half turns in [-1, 1): the wrapped angle over pi
            const float x = __ll2float_rn(static_cast<long long>(turn)) * 1.0842021724855044e-19f;  // 2^-63
            float s, c;
            sincospif(x, &s, &c);
            cs[buf][tok][table_at<VEC>(pair, items)] = c;
            sn[buf][tok][table_at<VEC>(pair, items)] = s;
        }
        __syncthreads();  // (the other buffer is written only after every thread has passed here again)
        const int total = nt * H * items;
        for (int base = threadIdx.x; base < total; base += U * kRopeThreads) {
            Chunk<T, VEC> a[U], b[U], ba[U], bb[U];
            T* oa[U];
            T* ob[U];
            int tk[U], it[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int idx = base + u * kRopeThreads;
                tk[u] = -1;
                if (idx >= total) continue;
                const int hh = idx >> ishift, i = idx & (items - 1);
                const int tok = div ? static_cast<int>(__umulhi(static_cast<uint32_t>(hh), div)) : hh;  // hh / H
                const int head = h0 + hh - tok * H;
                const long long t = t0 + tok;
                const T* src;
                T* dst;
                bool turns = true;
                if (head < p.Hq) {
                    src = static_cast<const T*>(p.q) + t * p.q_stride + static_cast<long long>(head) * D;
                    dst = static_cast<T*>(p.qo) + (t * p.Hq + head) * D;
                } else if (head < p.Hq + p.Hkv) {
                    src = static_cast<const T*>(p.k) + t * p.kv_stride + static_cast<long long>(head - p.Hq) * D;
                    dst = static_cast<T*>(p.ko) + (t * p.Hkv + head - p.Hq) * D;
                } else {
                    src = static_cast<const T*>(p.v) + t * p.kv_stride + static_cast<long long>(head - p.Hq - p.Hkv) * D;
                    dst = static_cast<T*>(p.vo) + (t * p.Hkv + head - p.Hq - p.Hkv) * D;
                    turns = false;
                }
                turns = turns && i < turning;
                int ea, eb;  // first elements of the item's two chunks
                if (p.adjacent || !turns) {
                    // neighbours; (halves) the elements behind the rotary part, or a value head's
                    ea = 2 * i * VEC;
                    eb = ea + VEC;
                } else {
                    ea = i * VEC;
                    eb = half + i * VEC;
                }
                tk[u] = tok;
                it[u] = turns ? i : -1;
                a[u].load(src + ea);
                b[u].load(src + eb);
                oa[u] = dst + ea;
                ob[u] = dst + eb;
                if (p.bias) {
                    const T* bs = static_cast<const T*>(p.bias) + static_cast<long long>(head) * D;
                    ba[u].load(bs + ea);
                    bb[u].load(bs + eb);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (tk[u] < 0) continue;
                float xa[VEC], xb[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    xa[e] = to_f<T>(a[u].e[e]);
                    xb[e] = to_f<T>(b[u].e[e]);
                    if (p.bias) {
                        xa[e] += to_f<T>(ba[u].e[e]);
                        xb[e] += to_f<T>(bb[u].e[e]);
                    }
                }
                if (it[u] >= 0) {
                    float c[VEC], s[VEC];
                    if constexpr (VEC < 4) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            c[e] = cs[buf][tk[u]][it[u] * VEC + e];
                            s[e] = sn[buf][tk[u]][it[u] * VEC + e];
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < VEC / 4; ++h) {
                            *reinterpret_cast<float4*>(c + 4 * h) =
                                *reinterpret_cast<const float4*>(&cs[buf][tk[u]][(h * items + it[u]) * 4]);
                            *reinterpret_cast<float4*>(s + 4 * h) =
                                *reinterpret_cast<const float4*>(&sn[buf][tk[u]][(h * items + it[u]) * 4]);
                        }
                    }
                    if (p.adjacent) {
                        // pair e: elements 2e and 2e + 1 of the item's 2 VEC
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
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    a[u].e[e] = from_f<T>(xa[e]);
                    b[u].e[e] = from_f<T>(xb[e]);
                }
                a[u].store(oa[u]);
                b[u].store(ob[u]);
            }
        }
        buf ^= 1;
    }
}

template <typename T>
const void* pick(int vec) {
    if constexpr (sizeof(T) == 2)
        if (vec == 8) return reinterpret_cast<const void*>(&rope_kernel<T, 8>);
    return vec == 4   ? reinterpret_cast<const void*>(&rope_kernel<T, 4>)
           : vec == 2 ? reinterpret_cast<const void*>(&rope_kernel<T, 2>)
                      : reinterpret_cast<const void*>(&rope_kernel<T, 1>);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int vec, int sms, cudaStream_t stream) {
    const void* fn = p.dt == kF32 ? pick<float>(vec) : p.dt == kF16 ? pick<__half>(vec) : pick<__nv_bfloat16>(vec);
    // Large calls: tiles of up to kRopeTileItems items, up to eight blocks an SM; fewer tokens where
    // that would give an SM fewer than four blocks (64 + 2 x 8 bf16 heads, 1200 / 2400 / 4000 tokens 11.2 /
    // 22.1 / 37.6 -> 9.9 / 19.2 / 33.3 us; 40 + 2 x 40 fp32 heads, 200 / 600 / 1001 tokens 8.4 / 13.1 / 19.9 -> 7.5 / 10.1 / 20.3).
    // Calls with fewer tiles than SMs: their heads over enough blocks to reach every SM (at least
    // 8 heads each).
    const int per_token = p.heads * (p.D / (2 * vec));
    p.tile = kRopeTile;
    while (p.tile > 1 && (p.tile * per_token > kRopeTileItems || p.n < 4LL * p.tile * sms)) p.tile >>= 1;
    const long long tiles = (p.n + p.tile - 1) / p.tile;
    long long split = tiles >= sms ? 1 : sms / tiles;
    p.heads_per_block = static_cast<int>((p.heads + split - 1) / split);
    if (p.heads_per_block < 8) p.heads_per_block = p.heads < 8 ? p.heads : 8;
    if (p.heads_per_block > 4096) p.heads_per_block = 4096;
    const int gy = (p.heads + p.heads_per_block - 1) / p.heads_per_block;
    // ceil(2^32 / H): hh / H as the high half of a product, exact for hh < tile * H <= 16 * 2^12
    for (int last = 0; last < 2; ++last) {
        const uint32_t h = static_cast<uint32_t>(last ? p.heads - (gy - 1) * p.heads_per_block : p.heads_per_block);
        p.div_h[last] = h == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + h - 1) / h);
    }
    const long long cap = static_cast<long long>(sms) * 8;
    const dim3 grid(static_cast<unsigned>(tiles < cap ? tiles : cap), static_cast<unsigned>(gy));
    void* args[] = {&p};
    return launch_pdl(fn, grid, kRopeThreads, 0, args, stream);
}

}  // namespace ftd
