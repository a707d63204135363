// cache_attn.cuh -- device helpers of the two cache_attention kernels: 4-bit
// rows to bf16, and the exact path for rows that share a tile with a key they
// must not see.
#pragma once

#include "cache_internal.cuh"

namespace qkr {

__device__ __forceinline__ uint32_t sub136(uint32_t x)
{
    const __nv_bfloat162 k = __floats2bfloat162_rn(136.f, 136.f);
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162 *>(&x);
    v = __hsub2(v, k);
    return *reinterpret_cast<uint32_t *>(&v);
}

// Nibbles i and i + 4 of w as the bf16 pair (128 + n_i, 128 + n_{i+4}).
__device__ __forceinline__ uint32_t nibbles(uint32_t w, int i)
{
    // one three-input instruction: with both constants written as immediates the
    // compiler makes two of it
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;"
        : "=r"(r) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
    return r;
}

// The same as (16 + n_i, 16 + n_{i+4}), where sums run on the numbers with their offset.
__device__ __forceinline__ uint32_t nibbles16(uint32_t w, int i)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;"
        : "=r"(r) : "r"(i ? w >> (4 * i - 3) : w << 3), "r"(0x00780078u), "r"(0x41804180u));
    return r;
}

__device__ __forceinline__ bool nonfinite2(uint32_t w)  // either bf16 of the word
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ float bf16_at(uint32_t w, int hi)
{
    return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
}

__device__ __forceinline__ const uint8_t *row_ptr(const CachePlane &pl, int page, int row, int head)
{
    return pl.base + page * pl.ps + row * pl.rs + head * pl.hs;
}

// Element d of a cached row, as fp32 (the exact path below).
template <bool Q4>
__device__ float cached(const CachePlane &pl, const CachePlane &sc, int page, int row, int head,
                        int d, int D, bool is_v)
{
    const uint8_t *src = row_ptr(pl, page, row, head);
    if constexpr (Q4) {
        const int w = d >> 5, r = d & 31;
        const int byte = is_v ? (r >> 2) * (D / 16) + 2 * w + ((r & 3) >> 1)
                              : (r >> 3) * (D / 8) + 4 * w + ((r & 7) >> 1);
        const int code = (src[byte] >> (4 * (d & 1))) & 15;
        const uint16_t s = reinterpret_cast<const uint16_t *>(row_ptr(sc, page, row, head))[w];
        return (float)(code - 8) * __uint_as_float((uint32_t)s << 16);
    } else {
        const uint16_t x = reinterpret_cast<const uint16_t *>(src)[d];
        return __uint_as_float((uint32_t)x << 16);
    }
}

// One row over the tiles [i0, i1) of a block, key by key, by one warp: the
// lane sums o for its DP/32 dims.  A key the row does not see is skipped, so
// nothing it holds can reach the row; the blocks whose values hold an infinity
// or a NaN in a key that only some of their rows see take this path, because in
// a matrix product 0 * NaN is NaN.  Slow and rare: some microseconds a key.  `beat`
// (or null) is counted up once a tile, for whoever waits meanwhile.
template <int DP, bool Q4>
__device__ __noinline__ void attn_row_exact(const AttnParams &p, const AttnBlock &k, int kvh,
                                            int r, int i0, int i1, float *m_out, float *l_out,
                                            float (&o)[DP / 32], int *beat)
{
    constexpr int E = DP / 32;
    const int lane = threadIdx.x & 31;
    int64_t t;
    int h;
    attn_row_of(p, k, kvh, r, &t, &h);
    const int pos = k.L - k.n + (k.row0 + r) / p.G;
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        q[e] = d < p.c.D ? __bfloat162float(p.q[t * p.q_ts + h * p.q_hs + d]) : 0.f;
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int i = i0; i < i1; ++i) {
        const int j0 = k.tile_at(i) * p.tile;
        if (beat && lane == 0)
            atomicAdd(beat, 1);
        for (int j = j0; j < j0 + p.tile; ++j) {
            if (!attn_sees(p, pos, j))
                continue;
            const int page = attn_page(p, k.b, j, lane == 0);
            const int row = j % p.c.page_size;
            float s = 0.f, v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = lane * E + e;
                const bool ok = page >= 0 && d < p.c.D;
                s += ok ? q[e] * cached<Q4>(p.c.k, p.c.ks, page, row, kvh, d, p.c.D, false) : 0.f;
                v[e] = ok ? cached<Q4>(p.c.v, p.c.vs, page, row, kvh, d, p.c.D, true) : 0.f;
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= p.scale_log2;
            const float mn = fmaxf(m, s);
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float f = exp2_fast(m - ref), w = exp2_fast(s - ref);
            l = l * f + w;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = o[e] * f + w * v[e];
            m = mn;
        }
    }
    *m_out = m;
    *l_out = l;
}


}  // namespace qkr
