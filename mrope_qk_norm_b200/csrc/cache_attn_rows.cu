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
// about one step of keys in flight: 16 (8 KB) in bf16, 32 (4.5 KB) in 4 bits at D
// = 128; 12 to 16 warps an SM keep the 40-50 KB in flight that HBM's latency asks
// for.
//
// Who takes which keys.  Much work: as many CTAs as stay resident, each with the
// same number of tiles of the row (sequence, KV head, tile), found on the device
// from the lengths, so a batch of one long and many short sequences is as even as
// any; a block cut between CTAs leaves its pieces in the workspace and a second
// kernel joins them.  Little work (the launch latency shows): a thread-block
// cluster a block, whose CTAs share its tiles and join them through distributed
// shared memory in the same launch.
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
// multiplies the sum in fp32.  For V the scale goes onto the weight, group by
// group, before its one rounding, and a second product takes -136 times the
// same rounded weights off again, tile by tile, so the offset never builds up
// in the sum: two matrix instructions in place of eight subtractions.

#include <cooperative_groups.h>

#include <climits>

#include "cache_attn.cuh"

namespace cg = cooperative_groups;

namespace qkr {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kMinus136 = 0xc308c308u;  // bf16 pair
constexpr float kSlack = 8.f;  // log2 units the reference may lag behind the maximum

// Tiles a warp takes together.
constexpr int rows_unroll(int dp, bool q4) { return q4 || dp == 64 ? 2 : 1; }

// CTAs of the even-shares kernel an SM holds (by registers).
constexpr int rows_ctas(int dp, int nt, bool q4)
{
    return nt == 2 ? 2 : (dp == 64 && q4 ? 4 : 3);
}

// d = a b + c on 16 x 8 x 16.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    mma16816(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
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

// A tile: its first key and its page (-1: reads as zeros), the row in it.
struct Tile {
    int j0, page, row;
};

// A lane's place in the rows of a KV head.
struct LanePtr {
    const uint8_t *k, *v, *ks, *vs;
};

__device__ __forceinline__ const uint8_t *tile_ptr(const uint8_t *lane, const CachePlane &pl,
                                                   const Tile &at)
{
    // page and row strides are below 2^32
    return lane + (uint64_t)(uint32_t)at.page * (uint32_t)pl.ps +
           (uint64_t)(uint32_t)at.row * (uint32_t)pl.rs;
}

// Loads of a tile (16 keys from a multiple of 16, so within one page).  Keys
// no row of the block sees read as zeros: what lies there may be anything.
template <int DP, bool Q4>
__device__ __forceinline__ void load_k(KTile<DP, Q4> &t, const AttnParams &p, const AttnBlock &k,
                                       const LanePtr &lp, const Tile &at, bool all)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint8_t *src = tile_ptr(lp.k, p.c.k, at);
    const uint8_t *ss = Q4 ? tile_ptr(lp.ks, p.c.ks, at) : nullptr;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool ok = all || (at.page >= 0 && attn_block_sees(k, at.j0 + g + 8 * i));
        if constexpr (Q4) {
            if (!all) {
#pragma unroll
                for (int w = 0; w < DP / 32; ++w)
                    t.w[i][w] = 0x88888888u;
#pragma unroll
                for (int w = 0; w < DP / 64; ++w)
                    t.s[i][w] = 0u;
            }
            if (ok) {
                ld_words<DP / 32>(t.w[i], src + 8 * i * p.c.k.rs);
                ld_words<DP / 64>(t.s[i], ss + 8 * i * p.c.ks.rs);
            }
        } else {
#pragma unroll
            for (int w = 0; w < DP / 32; ++w) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    t.w[i][4 * w + x] = 0u;
                if (ok && 32 * w + 8 * c < p.c.D)
                    ld_words<4>(&t.w[i][4 * w], src + 8 * i * p.c.k.rs + 64 * w);
            }
        }
    }
}

template <int DP, bool Q4>
__device__ __forceinline__ void load_v(VTile<DP, Q4> &t, const AttnParams &p, const AttnBlock &k,
                                       const LanePtr &lp, const Tile &at, bool all)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint8_t *src = tile_ptr(lp.v, p.c.v, at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = (i & 1) + 8 * (i >> 1);       // key 2c + x
        const bool ok = all || (at.page >= 0 && attn_block_sees(k, at.j0 + 2 * c + x));
        if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < DP / 64; ++w)
                if (!all)
                    t.w[i][w] = 0x88888888u;
            if (ok)
                ld_words<DP / 64>(t.w[i], src + x * p.c.v.rs);
        } else {
#pragma unroll
            for (int h = 0; h < DP / 64; ++h) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    t.w[i][4 * h + y] = 0u;
                if (ok && 64 * h + 8 * g < p.c.D)
                    ld_words<4>(&t.w[i][4 * h], src + x * p.c.v.rs + 128 * h);
            }
        }
    }
    if constexpr (Q4) {
        const uint8_t *ss = tile_ptr(lp.vs, p.c.vs, at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int w = 0; w < DP / 64; ++w)
                if (!all)
                    t.s[i][w] = 0u;
            if (all || (at.page >= 0 && attn_block_sees(k, at.j0 + g + 8 * i)))
                ld_words<DP / 64>(t.s[i], ss + 8 * i * p.c.vs.rs);
        }
    }
}

template <int DP, int NT>
struct RowsShared {
    float o[kWarps][8 * NT][DP + 4];
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    int poison;
    int scan[kWarps];
};

// The tiles [i0, i1) of a block and KV head by one CTA; each warp's maxima,
// sums and outputs go to sh.  Ends with a barrier.
template <int DP, int NT, bool Q4>
__device__ __forceinline__ void attn_piece(const AttnParams &p, const AttnBlock &k, int kvh, int i0,
                                           int i1, RowsShared<DP, NT> &sh)
{
    constexpr int KS = DP / 16;       // k steps of S^T, m tiles of O^T
    constexpr int GR = DP / 32;       // 4-bit groups of a row
    constexpr int U = rows_unroll(DP, Q4);   // tiles a warp takes together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;

    // ---- the warp's first tiles are asked for before anything else
    LanePtr lp;
    lp.k = p.c.k.base + kvh * p.c.k.hs + g * p.c.k.rs + c * (Q4 ? DP / 8 : 16);
    lp.v = p.c.v.base + kvh * p.c.v.hs + 2 * c * p.c.v.rs + g * (Q4 ? DP / 16 : 16);
    lp.ks = lp.vs = nullptr;
    if constexpr (Q4) {
        lp.ks = p.c.ks.base + kvh * p.c.ks.hs + g * p.c.ks.rs;
        lp.vs = p.c.vs.base + kvh * p.c.vs.hs + g * p.c.vs.rs;
    }
    const int32_t *table = p.table + (int64_t)k.b * p.table_stride;
    auto locate = [&](int i, Tile *t) {
        if (i >= i1) {
            t->j0 = INT_MAX / 2;   // no row sees it
            t->page = -1;
            t->row = 0;
            return;
        }
        const int at = k.tile_at(i);
        // division by the tiles of a page: exact for tiles below 2^26
        const int pg = (int)((uint64_t)at * p.page_recip >> 38);
        t->j0 = at * 16;
        t->row = t->j0 - pg * p.c.page_size;
        t->page = table[pg];
    };
    // a page id outside the cache
    auto admit = [&](Tile *t) {
        if ((unsigned)t->page >= (unsigned)p.c.n_pages) {
            if (t->j0 < INT_MAX / 2 && lane == 0)
                atomicOr(p.status, kStatusBounds);
            t->page = -1;
        }
    };
    // Tiles [in0, in1) of the piece: every row sees all their keys.
    const int in0 = k.c_sink +
                    (p.window ? max(0, (max(0, k.p_last - p.window + 1) + 15) / 16 - k.c0) : 0);
    const int in1 = min(i1, k.c_sink + (k.p_first + 1) / 16 - k.c0);
    // two copies of the loads: with and without a question per key
    auto get_k = [&](KTile<DP, Q4> &t, const Tile &at, bool plain) {
        if (plain)
            load_k<DP, Q4>(t, p, k, lp, at, true);
        else
            load_k<DP, Q4>(t, p, k, lp, at, false);
    };
    auto get_v = [&](VTile<DP, Q4> &t, const Tile &at, bool plain) {
        if (plain)
            load_v<DP, Q4>(t, p, k, lp, at, true);
        else
            load_v<DP, Q4>(t, p, k, lp, at, false);
    };
    KTile<DP, Q4> kt[U];
    VTile<DP, Q4> vt[U];
    Tile cur[U], next[U];
    int i = i0 + warp * U;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        locate(i + u, &cur[u]);
        locate(i + kWarps * U + u, &next[u]);
    }

    // ---- this block's rows: Q as the B operand, positions of a lane's columns
    uint32_t qf[NT][KS][2];
    float qs[NT][2][Q4 ? GR : 1];     // -136 * sum of q over a group, columns 2c and 2c + 1
    int pos[NT][2];
    uint4 qv[NT][GR];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        int64_t t;
        int h;
        attn_row_of(p, k, kvh, min(r, k.nrows - 1), &t, &h);
        const __nv_bfloat16 *src = p.q + t * p.q_ts + h * p.q_hs + 8 * c;
#pragma unroll
        for (int w = 0; w < GR; ++w) {
            qv[n][w] = make_uint4(0, 0, 0, 0);
            if (r < k.nrows && 32 * w + 8 * c < p.c.D)
                qv[n][w] = ld_stream(src + 32 * w);
        }
    }
    bool full = i >= in0 && i + U <= in1, plain = full;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        admit(&cur[u]);
        plain &= cur[u].page >= 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        get_k(kt[u], cur[u], plain);
        get_v(vt[u], cur[u], plain);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int w = 0; w < GR; ++w) {
            const uint4 v = qv[n][w];
            if constexpr (Q4) {
                // nibble i of a word pairs with nibble i + 4: dims i and i + 4 of the eight
                const uint32_t a[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                       __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sum += bf16_at(a[x], 0) + bf16_at(a[x], 1);
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
        for (int y = 0; y < KS; ++y)
            o[n][y][0] = o[n][y][1] = o[n][y][2] = o[n][y][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    bool poison = false;

    for (; i < i1; i += kWarps * U) {
        // S^T: lane has keys g, g + 8 (elements 0 and 1, 2 and 3) of columns 2c, 2c + 1
        float s[U][NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
            if constexpr (Q4) {
#pragma unroll
                for (int w = 0; w < GR; ++w) {
                    uint32_t a[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        a[2 * x] = nibbles(kt[u].w[0][w], x);
                        a[2 * x + 1] = nibbles(kt[u].w[1][w], x);
                    }
                    const float s0 = bf16_at(kt[u].s[0][w / 2], w & 1);
                    const float s1 = bf16_at(kt[u].s[1][w / 2], w & 1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4];
                        mma16816(d, a[0], a[1], a[2], a[3], qf[n][2 * w][0], qf[n][2 * w][1],
                                 qs[n][0][w], qs[n][1][w], qs[n][0][w], qs[n][1][w]);
                        mma16816(d, a[4], a[5], a[6], a[7], qf[n][2 * w + 1][0],
                                 qf[n][2 * w + 1][1]);
                        s[u][n][0] = fmaf(d[0], s0, s[u][n][0]);
                        s[u][n][1] = fmaf(d[1], s0, s[u][n][1]);
                        s[u][n][2] = fmaf(d[2], s1, s[u][n][2]);
                        s[u][n][3] = fmaf(d[3], s1, s[u][n][3]);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < KS; ++x)
                        mma16816(s[u][n], kt[u].w[0][2 * x], kt[u].w[1][2 * x],
                                 kt[u].w[0][2 * x + 1], kt[u].w[1][2 * x + 1], qf[n][x][0],
                                 qf[n][x][1]);
            }
        }
        const int in = i + kWarps * U;
        const bool more = in < i1, was_full = full;
        int was[U];
        plain = full = in >= in0 && in + U <= in1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            was[u] = cur[u].j0;
            cur[u] = next[u];
            admit(&cur[u]);
            plain &= cur[u].page >= 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (more)
                get_k(kt[u], cur[u], plain);
            locate(in + kWarps * U + u, &next[u]);
        }

        bool raise = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[u][n][e] *= p.scale_log2;
        if (!was_full) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!attn_sees(p, pos[n][e & 1], was[u] + g + 8 * (e >> 1)))
                            s[u][n][e] = -INFINITY;
                // a key only some rows see must not reach the others through 0 * NaN
                if (k.p_first != k.p_last)
#pragma unroll
                    for (int y = 0; y < (Q4 ? 2 : 4); ++y)
#pragma unroll
                        for (int w = 0; w < DP / (Q4 ? 64 : 16); ++w)
                            poison |= nonfinite2(Q4 ? vt[u].s[y][w] : vt[u].w[y][w]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = s[0][n][e];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    mx = fmaxf(mx, fmaxf(s[u][n][e], s[u][n][e + 2]));
                raise |= mx > m[n][e] + kSlack;
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = m[n][e];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        mx = fmaxf(mx, fmaxf(s[u][n][e], s[u][n][e + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
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
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][n][e] = exp2_fast(s[u][n][e] - ref);
                    l[n][e & 1] += s[u][n][e];
                }
            }
        }

        // O^T: two rows of dims and one pair of keys per register
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (Q4) {
#pragma unroll
                for (int w = 0; w < GR; ++w) {
                    uint32_t b[NT][2];
                    const float s0 = bf16_at(vt[u].s[0][w / 2], w & 1);
                    const float s1 = bf16_at(vt[u].s[1][w / 2], w & 1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b[n][0] = transpose8(pack2(s[u][n][0] * s0, s[u][n][1] * s0));
                        b[n][1] = transpose8(pack2(s[u][n][2] * s1, s[u][n][3] * s1));
                    }
                    const int sel = w & 1 ? 0x7632 : 0x5410;
                    const uint32_t lo = __byte_perm(vt[u].w[0][w / 2], vt[u].w[1][w / 2], sel);
                    const uint32_t hi = __byte_perm(vt[u].w[2][w / 2], vt[u].w[3][w / 2], sel);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a0 = nibbles(lo, 2 * y), a1 = nibbles(lo, 2 * y + 1);
                        const uint32_t a2 = nibbles(hi, 2 * y), a3 = nibbles(hi, 2 * y + 1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(o[n][2 * w + y], a0, a1, a2, a3, b[n][0], b[n][1]);
                            mma16816(o[n][2 * w + y], kMinus136, kMinus136, kMinus136, kMinus136,
                                     b[n][0], b[n][1]);
                        }
                    }
                }
            } else {
                uint32_t b[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    b[n][0] = transpose8(pack2(s[u][n][0], s[u][n][1]));
                    b[n][1] = transpose8(pack2(s[u][n][2], s[u][n][3]));
                }
#pragma unroll
                for (int w = 0; w < DP / 16; ++w) {
                    const uint32_t a0 = __byte_perm(vt[u].w[0][w], vt[u].w[1][w], 0x5410);
                    const uint32_t a1 = __byte_perm(vt[u].w[0][w], vt[u].w[1][w], 0x7632);
                    const uint32_t a2 = __byte_perm(vt[u].w[2][w], vt[u].w[3][w], 0x5410);
                    const uint32_t a3 = __byte_perm(vt[u].w[2][w], vt[u].w[3][w], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(o[n][w], a0, a1, a2, a3, b[n][0], b[n][1]);
                }
            }
            if (more)
                get_v(vt[u], cur[u], plain);
        }
    }

    // ---- columns 2c, 2c + 1 of the lane are rows of the block
    if (poison)
        sh.poison = 1;
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
                sh.m[warp][r] = m[n][e];
                sh.l[warp][r] = t;
            }
            float *dst = &sh.o[warp][r][0];
#pragma unroll
            for (int y = 0; y < KS; ++y) {
                // elements e, e + 2 of m tile y: two neighbouring dims
                const int d = Q4 ? 32 * (y / 2) + 4 * g + 2 * (y & 1)
                                 : 64 * (y / 4) + 8 * g + 2 * (y & 3);
                *reinterpret_cast<float2 *>(dst + d) = make_float2(o[n][y][e], o[n][y][e + 2]);
            }
        }
    }
    __syncthreads();
}

// Row r of the piece: the warps' parts joined, in fixed order.
template <int DP, int NT, bool Q4>
__device__ __forceinline__ void attn_piece_row(const AttnParams &p, const AttnBlock &k, int kvh,
                                               int i0, int i1, const RowsShared<DP, NT> &sh, int r,
                                               float *m, float *l, float (&acc)[DP / 32])
{
    constexpr int E = DP / 32;
    const int lane = threadIdx.x & 31;
    *m = -INFINITY;
    *l = 0.f;
    if (sh.poison) {
        attn_row_exact<DP, Q4>(p, k, kvh, r, i0, i1, m, l, acc);
        return;
    }
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        M = fmaxf(M, sh.m[w][r]);
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = M == -INFINITY ? 0.f : exp2_fast(sh.m[w][r] - M);
        L += f * sh.l[w][r];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] += f * sh.o[w][r][lane * E + e];
    }
    *m = M;
    *l = L;
}

// Little work: a cluster shares the tiles of a block and joins them.
template <int DP, int NT, bool Q4>
__global__ void __launch_bounds__(32 * kWarps)
attn_cluster_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int E = DP / 32;
    __shared__ __align__(16) RowsShared<DP, NT> sh;
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int size = p.cluster, rank = (int)(blockIdx.x % size);
    const int item = (int)(blockIdx.x / size);
    const int kvh = item % p.c.Hkv;
    const AttnBlock k = attn_block(p, item / p.c.Hkv);
    if (k.b < 0)
        return;     // the whole cluster
    if (threadIdx.x == 0)
        sh.poison = 0;
    __syncthreads();
    const int share = (k.ntiles + size - 1) / size;
    const int i0 = min(k.ntiles, rank * share), i1 = min(k.ntiles, i0 + share);
    attn_piece<DP, NT, Q4>(p, k, kvh, i0, i1, sh);
    for (int r = warp; r < k.nrows; r += kWarps) {
        float m, l, acc[E];
        attn_piece_row<DP, NT, Q4>(p, k, kvh, i0, i1, sh, r, &m, &l, acc);
        if (size == 1) {
            attn_emit<E>(p, k, kvh, r, 0, true, m, l, acc);
            continue;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < E; ++e)
            sh.o[0][r][lane * E + e] = acc[e];
        if (lane == 0) {
            sh.m[0][r] = m;
            sh.l[0][r] = l;
        }
    }
    if (size == 1)
        return;
    cluster.sync();
    // rows go round the cluster's warps; parts are added in rank order
    for (int r = rank * kWarps + warp; r < k.nrows; r += size * kWarps) {
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
        for (int c = 0; c < size; ++c)
            m = fmaxf(m, *cluster.map_shared_rank(&sh.m[0][r], c));
        for (int c = 0; c < size; ++c) {
            const float f =
                m == -INFINITY ? 0.f : exp2_fast(*cluster.map_shared_rank(&sh.m[0][r], c) - m);
            l += f * *cluster.map_shared_rank(&sh.l[0][r], c);
            const float *o = cluster.map_shared_rank(&sh.o[0][r][lane * E], c);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] += f * o[e];
        }
        attn_emit<E>(p, k, kvh, r, 0, true, m, l, acc);
    }
    cluster.sync();     // nobody leaves while its memory is read
}

// What a piece costs beside its tiles (the first loads' latency, the warps'
// join), in tiles: counted at the front of every block's share.
constexpr int kPieceCost = 8;

// Much work: every CTA takes the same number of tiles, kPieceCost more a block.
template <int DP, int NT, bool Q4>
__global__ void __launch_bounds__(32 * kWarps, rows_ctas(DP, NT, Q4))
attn_rows_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int E = DP / 32;
    __shared__ __align__(16) RowsShared<DP, NT> sh;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t Hkv = p.c.Hkv;
    // tiles of sequence b (a block that sees nothing still has its rows to write)
    auto tiles_of = [&](int b) -> int {
        if (b >= p.B)
            return 0;
        int64_t t0;
        bool bad;
        const int n = attn_seq(p, b, &t0, &bad);
        return attn_blocks_of(p, n)
                   ? kPieceCost + max(1, attn_block_at(p, b, 0, n, t0, bad).ntiles)
                   : 0;
    };
    // inclusive sum over the CTA's threads, and the total
    auto scan = [&](int v, int *total) -> int {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += up;
        }
        __syncthreads();
        if (lane == 31)
            sh.scan[warp] = v;
        __syncthreads();
        int add = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            add += w < warp ? sh.scan[w] : 0;
            all += sh.scan[w];
        }
        *total = all;
        return v + add;
    };
    int64_t all_tiles = 0;
    int mine = 0, upto = 0;        // of the chunk of sequences looked at last
    for (int b0 = 0; b0 < p.B; b0 += 32 * kWarps) {
        int total;
        mine = tiles_of(b0 + threadIdx.x);
        upto = scan(mine, &total);
        all_tiles += total;
    }
    const int64_t work = all_tiles * Hkv;
    int64_t quota = (work + p.ctas - 1) / p.ctas;
    if (quota < p.split_tiles)
        quota = p.split_tiles;
    int64_t at = blockIdx.x * quota;
    const int64_t end = min(work, at + quota);
    if (threadIdx.x == 0 && blockIdx.x < p.ctas)
        p.ws_span[blockIdx.x].b = -1;
    if (at >= end)
        return;

    // the sequence `at` falls in
    int64_t before = 0;
    int b = -1;
    for (int b0 = 0; b < 0; b0 += 32 * kWarps) {
        int total;
        if (p.B > 32 * kWarps) {
            mine = tiles_of(b0 + threadIdx.x);
            upto = scan(mine, &total);
        } else {
            total = (int)all_tiles;
        }
        if (at < (before + total) * Hkv) {
            const int64_t hi = (before + upto) * Hkv, lo = hi - (int64_t)mine * Hkv;
            __syncthreads();
            if (lo <= at && at < hi) {
                sh.scan[0] = b0 + threadIdx.x;
                sh.scan[1] = upto - mine;
            }
            __syncthreads();
            b = sh.scan[0];
            before += sh.scan[1];
        } else {
            before += total;
        }
    }

    bool first = true;
    while (at < end) {
        // the next sequence with rows of this launch
        int64_t t0;
        bool bad;
        int n = attn_seq(p, b, &t0, &bad);
        while (!attn_blocks_of(p, n))
            n = attn_seq(p, ++b, &t0, &bad);
        const AttnBlock k = attn_block_at(p, b, 0, n, t0, bad);
        const int tiles = max(1, k.ntiles), cost = kPieceCost + tiles;
        const int64_t off = at - before * Hkv;
        int kvh = (int)(off / cost), from = (int)(off % cost);
        for (; kvh < Hkv && at < end; ++kvh, from = 0) {
            const int to = (int)min((int64_t)cost, from + end - at);
            const int i0 = max(0, from - kPieceCost), i1 = max(0, to - kPieceCost);
            const int64_t last = at - from + cost - 1;   // the block's last unit
            at += to - from;
            if (i0 == i1)
                continue;        // the share ends before the block's first tile
            __syncthreads();     // sh is free
            if (threadIdx.x == 0)
                sh.poison = 0;
            __syncthreads();
            attn_piece<DP, NT, Q4>(p, k, kvh, i0, min(i1, k.ntiles), sh);
            const bool only = i0 == 0 && i1 == tiles;
            const int slot = 2 * (int)blockIdx.x + (first ? 0 : 1);
            for (int r = warp; r < k.nrows; r += kWarps) {
                float m, l, acc[E];
                attn_piece_row<DP, NT, Q4>(p, k, kvh, i0, min(i1, k.ntiles), sh, r, &m, &l, acc);
                if (only) {
                    attn_emit<E>(p, k, kvh, r, 0, true, m, l, acc);
                } else {
                    const int64_t row = (int64_t)slot * p.rows + r;
                    if (lane * E < p.c.D) {
                        float *w = p.ws_o + row * p.c.D + lane * E;
#pragma unroll
                        for (int e = 0; e < E; e += 2)
                            *reinterpret_cast<float2 *>(w + e) = make_float2(acc[e], acc[e + 1]);
                    }
                    if (lane == 0)
                        p.ws_ml[row] = make_float2(m, l);
                }
            }
            if (i0 == 0 && i1 < tiles && threadIdx.x == 0) {
                // begins here, goes on in the CTAs after this one
                AttnSpan s;
                s.b = b;
                s.kvh = kvh;
                s.parts = (int)(last / quota) - (int)blockIdx.x + 1;
                s.slot = slot;
                s.n = n;
                s.L = k.L;
                s.t0 = t0;
                p.ws_span[blockIdx.x] = s;
            }
            first = false;
        }
        if (at < end) {
            before += cost;
            ++b;
        }
    }
}

// Joins the pieces of the block that CTA x / rows began, row x % rows.
template <int DP>
__global__ void __launch_bounds__(32 * kWarps)
attn_rows_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int E = DP / 32;
    __shared__ float sm_o[kWarps][DP];
    __shared__ float sm_l[kWarps], sm_m[kWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = (int)(blockIdx.x / p.rows), r = (int)(blockIdx.x % p.rows);
    const AttnSpan s = p.ws_span[cta];
    if (s.b < 0 || r >= s.n * p.G)
        return;
    // part i lies in slot 2(cta + i), the first one in its own
    auto row_at = [&](int i) -> int64_t {
        return (int64_t)(i ? 2 * (cta + i) : s.slot) * p.rows + r;
    };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < s.parts; i += 32 * kWarps)
        m = fmaxf(m, p.ws_ml[row_at(i)].x);
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
    for (int i = warp; i < s.parts; i += kWarps) {
        const int64_t row = row_at(i);
        const float2 ml = p.ws_ml[row];
        const float f = m == -INFINITY ? 0.f : exp2_fast(ml.x - m);
        l += f * ml.y;
        if (d < p.c.D) {
            const float *w = p.ws_o + row * p.c.D + d;
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
    AttnBlock k;
    k.t0 = s.t0;
    k.n = s.n;
    k.L = s.L;
    k.row0 = 0;
    attn_emit<E>(p, k, s.kvh, r, 0, true, m, l, acc);
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

template <int DP, int NT, bool Q4>
cudaError_t rows_launch(const AttnParams &p, cudaStream_t stream, LaunchRecord *rec)
{
    const dim3 block(32 * kWarps);
    if (p.ctas == 0) {
        rec->grid = p.n_blocks * p.c.Hkv * p.cluster;
        rec->cluster = p.cluster;
        return launch(attn_cluster_kernel<DP, NT, Q4>, dim3((unsigned)rec->grid), block, 0, stream,
                      p.cluster, p);
    }
    rec->grid = p.ctas;
    cudaError_t e = launch(attn_rows_kernel<DP, NT, Q4>, dim3((unsigned)p.ctas), block, 0, stream, 1,
                           p);
    if (e == cudaSuccess) {
        e = launch(attn_rows_join_kernel<DP>, dim3((unsigned)(p.ctas * p.rows)), block, 0, stream, 1,
                   p);
        rec->launches += 1;
    }
    return e;
}

}  // namespace

int attn_rows_resident(int64_t D, int rows, int q4)
{
    return rows_ctas(D <= 64 ? 64 : 128, rows == 8 ? 1 : 2, q4 != 0);
}

cudaError_t launch_attn_rows(const AttnParams &p, int q4, cudaStream_t stream, LaunchRecord *rec)
{
    cudaError_t e;
    if (p.rows == 8)
        e = p.c.D <= 64 ? (q4 ? rows_launch<64, 1, true>(p, stream, rec)
                              : rows_launch<64, 1, false>(p, stream, rec))
                        : (q4 ? rows_launch<128, 1, true>(p, stream, rec)
                              : rows_launch<128, 1, false>(p, stream, rec));
    else
        e = p.c.D <= 64 ? (q4 ? rows_launch<64, 2, true>(p, stream, rec)
                              : rows_launch<64, 2, false>(p, stream, rec))
                        : (q4 ? rows_launch<128, 2, true>(p, stream, rec)
                              : rows_launch<128, 2, false>(p, stream, rec));
    if (e == cudaSuccess) {
        rec->kernel = QKR_KERNEL_ATTN_ROWS;
        rec->block = 32 * kWarps;
        rec->stages = p.ctas ? p.ctas : p.cluster;
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
