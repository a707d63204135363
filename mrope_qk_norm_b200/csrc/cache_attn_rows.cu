// cache_attn_rows.cu -- cache_attention for sequences with few rows (a decode
// step: one new token, the query heads of a KV head), bf16 or 4-bit cache, and
// the kernel that joins the parts of a split axis.
//
// Every key and value is read once per block and used for a handful of rows,
// so the bound is HBM.  The products run on mma.sync with the roles turned
// round: keys (or dims) are the 16 rows of the A operand and the block's rows
// the 8 columns of B, so no half of a tile is padding for a group of 8 heads:
//   S^T [16 keys x 8 rows]  = K [16 x D] . Q^T [D x 8]
//   O^T [16 dims x 8 rows] += V^T [16 x 16 keys] . P^T [16 x 8]
// The dims of a head may be summed in any order, so a lane takes 16 consecutive
// bytes of a key's row for its K operand (the matching order of Q is set up
// once), and for V^T 16 consecutive bytes of each of its four keys, paired key
// by key with byte permutes.  Keys and values thus go from global memory
// straight into the operand registers: no shared memory, no barrier, and every
// warp walks its own keys with its own running maximum.  The next tile's K is
// requested when this one's has been used and likewise V, so a warp always has
// about one tile of 16 keys in flight (8 KB at D = 128; 12 warps an SM keep
// the 40-50 KB in flight that HBM's latency asks for).
//
// The running maximum is a reference, not the maximum: it moves only when a
// score exceeds it by 2^8, so the usual step has no cross-lane reduction and
// no rescaling; weights stay below 2^8, and l and O (fp32) share the reference,
// which the division removes exactly.  The weights are rounded to bf16 for the
// matrix instruction (at most 2^-9 of each, as the output itself is); l sums
// them unrounded.
//
// 4 bits: a nibble n becomes the bf16 number 128 + n by one AND-OR on two
// nibbles at a time.  For K the products run on 128 + n against an accumulator
// that starts at -136 * (sum of q), per group of 32 dims, and the group's scale
// multiplies the sum in fp32.  For V, 136 is subtracted (exact) and the scale
// goes onto the weight, group by group, before its one rounding.

#include <atomic>

#include "cache_attn.cuh"

namespace qkr {
namespace {

constexpr int kWarps = 4;
constexpr float kSlack = 8.f;  // log2 units the reference may lag behind the maximum

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// What a lane holds of a tile of 16 keys.  g = lane / 4, c = lane % 4.
//   K: keys g and g + 8, dims 32w + 8c .. + 7
//   V: keys 2c, 2c + 1, 2c + 8, 2c + 9; bf16: dims 64h + 8g .. + 7,
//      4 bits: dims 32w + 4g .. + 3
//   scales: keys g and g + 8 of both (the weights are scaled where they are made)
template <int DP, bool Q4>
struct KTile {
    uint32_t w[2][Q4 ? DP / 32 : DP / 8];
    uint32_t s[2][Q4 ? DP / 64 : 1];
};
template <int DP, bool Q4>
struct VTile {
    uint32_t w[4][Q4 ? DP / 64 : DP / 16];
    uint32_t s[2][Q4 ? DP / 64 : 1];
};

template <int N>
__device__ __forceinline__ void ld_words(uint32_t *w, const uint8_t *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
        static_assert(N == 1, "1, 2 or a multiple of 4 words");
        w[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
    }
}

// Loads of the tile at key j0 (a multiple of 16, so within one page).  Keys
// no row of the block sees read as zeros: what lies there may be anything.
template <int DP, bool Q4>
__device__ __forceinline__ void load_k(KTile<DP, Q4> &t, const AttnParams &p, const AttnBlock &k,
                                       int kvh, int j0, int page)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int r0 = j0 % p.c.page_size;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool ok = page >= 0 && attn_block_sees(k, j0 + g + 8 * i);
        const uint8_t *src = row_ptr(p.c.k, page, r0 + g + 8 * i, kvh);
        if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < DP / 32; ++w)
                t.w[i][w] = 0x88888888u;
#pragma unroll
            for (int w = 0; w < DP / 64; ++w)
                t.s[i][w] = 0u;
            if (ok) {
                ld_words<DP / 32>(t.w[i], src + c * (DP / 8));
                ld_words<DP / 64>(t.s[i], row_ptr(p.c.ks, page, r0 + g + 8 * i, kvh));
            }
        } else {
#pragma unroll
            for (int w = 0; w < DP / 32; ++w) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    t.w[i][4 * w + x] = 0u;
                if (ok && 32 * w + 8 * c < p.c.D)
                    ld_words<4>(&t.w[i][4 * w], src + 2 * (32 * w + 8 * c));
            }
        }
    }
}

template <int DP, bool Q4>
__device__ __forceinline__ void load_v(VTile<DP, Q4> &t, const AttnParams &p, const AttnBlock &k,
                                       int kvh, int j0, int page)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int r0 = j0 % p.c.page_size;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = 2 * c + (i & 1) + 8 * (i >> 1);
        const bool ok = page >= 0 && attn_block_sees(k, j0 + x);
        const uint8_t *src = row_ptr(p.c.v, page, r0 + x, kvh);
        if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < DP / 64; ++w)
                t.w[i][w] = 0x88888888u;
            if (ok)
                ld_words<DP / 64>(t.w[i], src + g * (DP / 16));
        } else {
#pragma unroll
            for (int h = 0; h < DP / 64; ++h) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    t.w[i][4 * h + y] = 0u;
                if (ok && 64 * h + 8 * g < p.c.D)
                    ld_words<4>(&t.w[i][4 * h], src + 2 * (64 * h + 8 * g));
            }
        }
    }
    if constexpr (Q4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int w = 0; w < DP / 64; ++w)
                t.s[i][w] = 0u;
            if (page >= 0 && attn_block_sees(k, j0 + g + 8 * i))
                ld_words<DP / 64>(t.s[i], row_ptr(p.c.vs, page, r0 + g + 8 * i, kvh));
        }
    }
}

template <int DP, int NT, bool Q4>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2)
attn_rows_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int KS = DP / 16;       // k steps of S^T, m tiles of O^T
    constexpr int GR = DP / 32;       // 4-bit groups of a row
    constexpr int ROWS = 8 * NT;
    constexpr int E = DP / 32;
    constexpr int PITCH = DP + 4;
    __shared__ float sm_o[kWarps][ROWS][PITCH];
    __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
    __shared__ int sm_poison;

    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t x = blockIdx.x;
    const int kvh = (int)(x % p.c.Hkv);
    const int part = (int)(x / p.c.Hkv / p.n_blocks);
    const AttnBlock k = attn_block(p, x / p.c.Hkv % p.n_blocks);
    if (k.b < 0)
        return;
    const int nparts = max(1, (k.ntiles + p.split_tiles - 1) / p.split_tiles);
    if (part >= nparts)
        return;
    const int i0 = part * p.split_tiles, i1 = min(k.ntiles, i0 + p.split_tiles);
    if (threadIdx.x == 0)
        sm_poison = 0;
    __syncthreads();

    // ---- this block's rows: Q as the B operand, positions of a lane's columns
    uint32_t qf[NT][KS][2];
    float qs[NT][2][Q4 ? GR : 1];     // -136 * sum of q over a group, columns 2c and 2c + 1
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        int64_t t;
        int h;
        attn_row_of(p, k, kvh, min(r, k.nrows - 1), &t, &h);
        const __nv_bfloat16 *src = p.q + t * p.q_ts + h * p.q_hs;
#pragma unroll
        for (int w = 0; w < GR; ++w) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < k.nrows && 32 * w + 8 * c < p.c.D)
                v = ld_stream(src + 32 * w + 8 * c);
            if constexpr (Q4) {
                // nibble i of a word pairs with nibble i + 4: dims i and i + 4 of the eight
                const uint32_t a[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                       __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += bf16_at(a[i], 0) + bf16_at(a[i], 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qs[n][0][w] = -136.f * __shfl_sync(0xffffffffu, sum, 8 * c);
                qs[n][1][w] = -136.f * __shfl_sync(0xffffffffu, sum, 8 * c + 4);
                qf[n][2 * w][0] = a[0];
                qf[n][2 * w][1] = a[1];
                qf[n][2 * w + 1][0] = a[2];
                qf[n][2 * w + 1][1] = a[3];
            } else {
                qf[n][2 * w][0] = v.x;
                qf[n][2 * w][1] = v.y;
                qf[n][2 * w + 1][0] = v.z;
                qf[n][2 * w + 1][1] = v.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 8 * n + 2 * c + e;
            pos[n][e] = col < k.nrows ? k.L - k.n + (k.row0 + col) / p.G : -1;
        }
    }

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
            o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    bool poison = false;

    // ---- this warp's tiles: i0 + warp, then every kWarps-th
    KTile<DP, Q4> kt;
    VTile<DP, Q4> vt;
    int i = i0 + warp;
    int page_next = -1;
    if (i < i1) {
        const int j0 = k.tile_at(i) * 16;
        const int page = attn_page(p, k.b, j0, lane == 0);
        load_k<DP, Q4>(kt, p, k, kvh, j0, page);
        load_v<DP, Q4>(vt, p, k, kvh, j0, page);
        if (i + kWarps < i1)
            page_next = attn_page(p, k.b, k.tile_at(i + kWarps) * 16, lane == 0);
    }
    for (; i < i1; i += kWarps) {
        const int j0 = k.tile_at(i) * 16;
        const bool more = i + kWarps < i1;
        const int j0n = more ? k.tile_at(i + kWarps) * 16 : 0;
        const int page = page_next;
        if (i + 2 * kWarps < i1)
            page_next = attn_page(p, k.b, k.tile_at(i + 2 * kWarps) * 16, lane == 0);

        // S^T: lane has keys g, g + 8 (second index 0/1, 2/3) of columns 2c, 2c + 1
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            if constexpr (Q4) {
#pragma unroll
                for (int w = 0; w < GR; ++w) {
                    float a[4] = {qs[n][0][w], qs[n][1][w], qs[n][0][w], qs[n][1][w]};
                    mma16816(a, nibbles(kt.w[0][w], 0), nibbles(kt.w[1][w], 0),
                             nibbles(kt.w[0][w], 1), nibbles(kt.w[1][w], 1), qf[n][2 * w][0],
                             qf[n][2 * w][1]);
                    mma16816(a, nibbles(kt.w[0][w], 2), nibbles(kt.w[1][w], 2),
                             nibbles(kt.w[0][w], 3), nibbles(kt.w[1][w], 3), qf[n][2 * w + 1][0],
                             qf[n][2 * w + 1][1]);
                    const float s0 = bf16_at(kt.s[0][w / 2], w & 1);
                    const float s1 = bf16_at(kt.s[1][w / 2], w & 1);
                    s[n][0] = fmaf(a[0], s0, s[n][0]);
                    s[n][1] = fmaf(a[1], s0, s[n][1]);
                    s[n][2] = fmaf(a[2], s1, s[n][2]);
                    s[n][3] = fmaf(a[3], s1, s[n][3]);
                }
            } else {
#pragma unroll
                for (int x2 = 0; x2 < KS; ++x2)
                    mma16816(s[n], kt.w[0][2 * x2], kt.w[1][2 * x2], kt.w[0][2 * x2 + 1],
                             kt.w[1][2 * x2 + 1], qf[n][x2][0], qf[n][x2][1]);
            }
        }
        if (more)
            load_k<DP, Q4>(kt, p, k, kvh, j0n, page);

        const bool full = attn_all_see(p, k, j0, 16);
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][e] *= p.scale_log2;
                if (!full && !attn_sees(p, pos[n][e & 1], j0 + g + 8 * (e >> 1)))
                    s[n][e] = -INFINITY;
                raise |= s[n][e] > m[n][e & 1] + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[n][e], s[n][e + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    mx = fmaxf(mx, m[n][e]);
                    const float f = m[n][e] == -INFINITY ? 0.f : exp2_fast(m[n][e] - mx);
                    m[n][e] = mx;
                    l[n][e] *= f;
#pragma unroll
                    for (int y = 0; y < KS; ++y) {
                        o[n][y][e] *= f;
                        o[n][y][e + 2] *= f;
                    }
                }
            }
        }
        if (!full && k.p_first != k.p_last) {
            // a key only some rows see must not reach the others through 0 * NaN
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if constexpr (!Q4) {
#pragma unroll
                    for (int w = 0; w < DP / 16; ++w)
                        poison |= nonfinite2(vt.w[y][w]);
                }
            }
            if constexpr (Q4) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int w = 0; w < DP / 64; ++w)
                        poison |= nonfinite2(vt.s[y][w]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
                s[n][e] = exp2_fast(s[n][e] - ref);
                l[n][e & 1] += s[n][e];
            }
        }

        // O^T: two rows of dims and one pair of keys per register
        if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < GR; ++w) {
                uint32_t b[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float s0 = bf16_at(vt.s[0][w / 2], w & 1);
                    const float s1 = bf16_at(vt.s[1][w / 2], w & 1);
                    b[n][0] = transpose8(pack2(s[n][0] * s0, s[n][1] * s0));
                    b[n][1] = transpose8(pack2(s[n][2] * s1, s[n][3] * s1));
                }
                const int sel = w & 1 ? 0x7632 : 0x5410;
                const uint32_t lo = __byte_perm(vt.w[0][w / 2], vt.w[1][w / 2], sel);
                const uint32_t hi = __byte_perm(vt.w[2][w / 2], vt.w[3][w / 2], sel);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t a0 = sub136(nibbles(lo, 2 * y));
                    const uint32_t a1 = sub136(nibbles(lo, 2 * y + 1));
                    const uint32_t a2 = sub136(nibbles(hi, 2 * y));
                    const uint32_t a3 = sub136(nibbles(hi, 2 * y + 1));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(o[n][2 * w + y], a0, a1, a2, a3, b[n][0], b[n][1]);
                }
            }
        } else {
            uint32_t b[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                b[n][0] = transpose8(pack2(s[n][0], s[n][1]));
                b[n][1] = transpose8(pack2(s[n][2], s[n][3]));
            }
#pragma unroll
            for (int w = 0; w < DP / 16; ++w) {
                const uint32_t a0 = __byte_perm(vt.w[0][w], vt.w[1][w], 0x5410);
                const uint32_t a1 = __byte_perm(vt.w[0][w], vt.w[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(vt.w[2][w], vt.w[3][w], 0x5410);
                const uint32_t a3 = __byte_perm(vt.w[2][w], vt.w[3][w], 0x7632);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(o[n][w], a0, a1, a2, a3, b[n][0], b[n][1]);
            }
        }
        if (more)
            load_v<DP, Q4>(vt, p, k, kvh, j0n, page);
    }

    // ---- join the warps: columns 2c, 2c + 1 of the lane are rows of the block
    if (poison)
        sm_poison = 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = l[n][e];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int r = 8 * n + 2 * c + e;
            if (g == 0) {
                sm_m[warp][r] = m[n][e];
                sm_l[warp][r] = t;
            }
            float *dst = &sm_o[warp][r][0];
#pragma unroll
            for (int y = 0; y < KS; ++y) {
                // registers e, e + 2 of m tile y: two neighbouring dims
                const int d = Q4 ? 32 * (y / 2) + 4 * g + 2 * (y & 1)
                                 : 64 * (y / 4) + 8 * g + 2 * (y & 3);
                *reinterpret_cast<float2 *>(dst + d) = make_float2(o[n][y][e], o[n][y][e + 2]);
            }
        }
    }
    __syncthreads();
    for (int r = warp; r < k.nrows; r += kWarps) {
        float M = -INFINITY, L = 0.f, acc[E];
        if (sm_poison) {
            attn_row_exact<DP, Q4>(p, k, kvh, r, i0, i1, &M, &L, acc);
        } else {
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                M = fmaxf(M, sm_m[w][r]);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = M == -INFINITY ? 0.f : exp2_fast(sm_m[w][r] - M);
                L += f * sm_l[w][r];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] += f * sm_o[w][r][lane * E + e];
            }
        }
        attn_emit<E>(p, k, kvh, r, part, nparts == 1, M, L, acc);
    }
}

// Joins the parts of a row: one CTA per block row and KV head; the warps take
// every fourth part.
template <int DP>
__global__ void __launch_bounds__(32 * kWarps) attn_join_kernel(const __grid_constant__ AttnParams p,
                                                                int rows_used)
{
    constexpr int E = DP / 32;
    __shared__ float sm_o[kWarps][DP];
    __shared__ float sm_l[kWarps], sm_m[kWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t x = blockIdx.x;
    const int r = (int)(x % rows_used);
    const int kvh = (int)(x / rows_used % p.c.Hkv);
    const AttnBlock k = attn_block(p, x / rows_used / p.c.Hkv);
    if (k.b < 0 || r >= k.nrows)
        return;
    const int nparts = max(1, (k.ntiles + p.split_tiles - 1) / p.split_tiles);
    if (nparts == 1)
        return;  // written already
    int64_t t;
    int h;
    attn_row_of(p, k, kvh, r, &t, &h);
    const int64_t row = t * p.Hq + h, step = p.T * p.Hq;
    float m = -INFINITY;
    for (int s = warp * 32 + lane; s < nparts; s += 32 * kWarps)
        m = fmaxf(m, p.ws_ml[row + s * step].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0)
        sm_m[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    const int d = lane * E;
#pragma unroll 4
    for (int s = warp; s < nparts; s += kWarps) {
        const float2 ml = p.ws_ml[row + s * step];
        const float f = m == -INFINITY ? 0.f : exp2_fast(ml.x - m);
        l += f * ml.y;
        if (d < p.c.D) {
            const float *w = p.ws_o + (row + s * step) * p.c.D + d;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(w + e);
                acc[e] += f * v.x;
                acc[e + 1] += f * v.y;
            }
        }
    }
    if (lane == 0)
        sm_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        sm_o[warp][d + e] = acc[e];
    __syncthreads();
    if (warp)
        return;
    l = ((sm_l[0] + sm_l[1]) + sm_l[2]) + sm_l[3];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = ((sm_o[0][d + e] + sm_o[1][d + e]) + sm_o[2][d + e]) + sm_o[3][d + e];
    attn_emit<E>(p, k, kvh, r, 0, true, m, l, acc);
}

template <int DP, int NT>
cudaError_t rows_launch(const AttnParams &p, int q4, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.n_blocks * p.c.Hkv * p.nsplit));
    auto fn = q4 ? attn_rows_kernel<DP, NT, true> : attn_rows_kernel<DP, NT, false>;
    return launch(fn, grid, dim3(32 * kWarps), 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnParams &p, int q4, cudaStream_t stream, LaunchRecord *rec)
{
    cudaError_t e;
    if (p.rows == 8)
        e = p.c.D <= 64 ? rows_launch<64, 1>(p, q4, stream) : rows_launch<128, 1>(p, q4, stream);
    else
        e = p.c.D <= 64 ? rows_launch<64, 2>(p, q4, stream) : rows_launch<128, 2>(p, q4, stream);
    if (e == cudaSuccess && rec) {
        rec->kernel = QKR_KERNEL_ATTN_ROWS;
        rec->block = 32 * kWarps;
        rec->grid = p.n_blocks * p.c.Hkv * p.nsplit;
        rec->stages = p.nsplit;
        rec->heads_per_item = p.rows;
        rec->launches += 1;
    }
    return e;
}

cudaError_t launch_attn_join(const AttnParams &p, cudaStream_t stream)
{
    const int64_t most = (int64_t)p.max_q * p.G;
    const int used = (int)(most < p.rows ? most : p.rows);
    const dim3 grid((unsigned)(p.n_blocks * p.c.Hkv * used));
    return p.c.D <= 64 ? launch(attn_join_kernel<64>, grid, dim3(32 * kWarps), 0, stream, 1, p, used)
                       : launch(attn_join_kernel<128>, grid, dim3(32 * kWarps), 0, stream, 1, p,
                                used);
}

}  // namespace qkr
