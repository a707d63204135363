// cache_attn_tiles.cu -- cache_attention for sequences with many rows (prompts
// and parts of prompts), on the fifth-generation tensor cores.
//
// A block is 256 rows of one sequence and KV head (row = new token x query
// head of the group, so any group size fills the tiles) as two tiles of 128.
// Per 128 keys and tile i:  S_i = Q_i K^T  and  O_i += P_i V, both tcgen05.mma
// with 128 accumulator rows; O_i stays in tensor memory for the whole axis and
// P_i (bf16) takes the place of S_i there, so neither passes through shared
// memory.  Tensor memory: S0 | S1 | O0 | O1.
//
// The softmax warps take registers from the others (setmaxnreg): 216 + 216 + 72
// of the 3 x 168 launched (4 bits: 184 + 184 + 72 + 72 of 4 x 128), so a row's 128
// scores stay in registers.
//
//   warps 0-3, 4-7  softmax of tile 0 and tile 1, one row a thread
//   warp 8          issues the matrix instructions, in the order
//                   P0 V(j), Q0 K(j+1), P1 V(j), Q1 K(j+1): while one tile's
//                   softmax runs, the tensor cores work for the other
//   bf16: warp 9    K and V tiles by TMA, a ring of 32 KB (16 KB) stages
//         10, 11    clear the values no row of the block sees (below)
//   4 bits: 12-15   K and V tiles from nibbles to bf16 in shared memory, one
//                   key a thread
//
// Per tile and 128 keys at D = 128 the two products take 1024 clocks of the
// tensor cores and the 16384 exponentials 1024 clocks of the SM's exponential
// units, so these two bound the kernel together; loads are 64 KB per 2048
// clocks and mostly hit L2.
//
// The running maximum is a reference that moves only when a score exceeds it by
// 2^8: the usual tile leaves O alone, and a weight stays below 2^8.  When the
// softmax of tile i sees S_i(j), its product P_i V(j-1) has finished (the
// instructions complete in order), so rescaling O_i needs no further wait.
//
// A tile that some row does not see in full is masked by selects on S.  Its
// values need more: 0 * NaN is NaN in a product.  Pages that no row sees are
// read as zeros (an out-of-range page coordinate), keys in other pages that no
// row sees are cleared in shared memory, and where a key that only some rows
// see holds an infinity or a NaN the block is computed again key by key
// (attn_row_exact).
//
// Every wait is bounded: one that runs out raises bit 16 of the status word,
// all roles stop issuing, copies and matrix instructions in flight are waited
// for (bounded), tensor memory is freed and the block ends.

#include "cache_attn.cuh"
#include "cache_tma.cuh"

namespace qkr {
namespace {

constexpr int kTile = 128;               // keys of a tile, rows of a tile
constexpr float kSlack = 8.f;
constexpr uint32_t kWaitLimit = 1u << 21;

template <int DP>
struct Layout {
    static constexpr int kHalves = DP / 64;
    static constexpr int kStageBytes = kHalves * kTile * 128;
    static constexpr int kQBytes = 2 * kStageBytes;
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kBytes = kQBytes + kStages * kStageBytes + 1024 /* alignment */;
};

struct Shared {
    uint64_t raw[8], empty[8];            // ring: full, free
    uint64_t land[4];                     // a V tile to be cleared first has landed, in turn
    uint64_t q_full, s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int abort, poison;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint64_t *b, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)),
                 "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// False when the wait ran out or another role's has.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, int *abort)
{
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (bar_try(b, parity))
            return true;
        if ((i & 15u) == 15u && *reinterpret_cast<volatile int *>(abort))
            return false;
    }
    *reinterpret_cast<volatile int *>(abort) = 1;
    return false;
}

__device__ __forceinline__ void fence_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *b)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(b)) : "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle (bits 61-63 = 2), the
// fixed bit 46, addresses in 16-byte units.  K-major rows of 128 bytes: groups
// of 8 rows 1024 bytes apart.  MN-major: groups of 8 keys 1024 bytes apart,
// blocks of 64 dims a half tile apart.
__device__ __forceinline__ uint64_t desc_base(uint32_t lead_bytes)
{
    return (uint64_t)2 << 61 | (uint64_t)1 << 46 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)(lead_bytes >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t addr)
{
    return base | (uint64_t)((addr >> 4) & 0x3fffu);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

#define QKR_R8(a, o) "=r"(a[o]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), "=r"(a[o + 4]), \
                     "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])
#define QKR_I8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), \
                     "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])
#define QKR_LIST32                                                                               \
    "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, " \
    "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}"

// 32 columns of the warp's 32 lanes, one lane a thread.
__device__ __forceinline__ void tm_load32(uint32_t *r, uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " QKR_LIST32 ", [%32];"
                 : QKR_R8(r, 0), QKR_R8(r, 8), QKR_R8(r, 16), QKR_R8(r, 24)
                 : "r"(addr));
}
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " QKR_LIST32 ";" ::QKR_I8(r, 0),
                 QKR_I8(r, 8), QKR_I8(r, 16), QKR_I8(r, 24), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tm_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int REGS>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

// Order of the eight elements of a 16-byte chunk of a 4-bit row in shared
// memory: 0 4 1 5 2 6 3 7, as the nibbles pair up.  Q's chunks follow it for
// the first product, O's columns are read back through it.
__device__ __forceinline__ uint4 pair_order(const uint4 &v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

template <int DP, bool Q4>
__global__ void __launch_bounds__(Q4 ? 512 : 384, 1)
attn_tiles_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps map)
{
    using Lay = Layout<DP>;
    constexpr int NST = Lay::kStages;
    constexpr int E = DP / 32;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    uint8_t *base = reinterpret_cast<uint8_t *>(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
    uint8_t *ring = base + Lay::kQBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_wait();
    pdl_trigger();
    const int64_t x = blockIdx.x;
    const int kvh = (int)(x % p.c.Hkv);
    const int part = (int)(x / p.c.Hkv / p.n_blocks);
    const AttnBlock k = attn_block(p, x / p.c.Hkv % p.n_blocks);
    if (k.b < 0)
        return;
    const int nparts = max(1, (k.ntiles + p.split_tiles - 1) / p.split_tiles);
    if (part >= nparts)
        return;
    const int i0 = part * p.split_tiles;
    const int nt = min(k.ntiles - i0, p.split_tiles);   // tiles of this part
    const int halves = k.nrows > kTile ? 2 : 1;         // row tiles in use

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            bar_init(&sh.raw[i], Q4 ? 128 : 1);
            bar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 4; ++i)
            bar_init(&sh.land[i], 1);
        bar_init(&sh.q_full, 256);
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.s_full[i], 1);
            bar_init(&sh.p_full[i], 128);
            bar_init(&sh.o_full[i], 1);
        }
        bar_init(&sh.drain, 1);
        sh.abort = 0;
        sh.poison = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t tm_s[2] = {tmem, tmem + 128}, tm_o[2] = {tmem + 256, tmem + 256 + DP};

    if (warp < 8) {
        regs_up<Q4 ? 184 : 216>();
        // ================================================ softmax, one row a thread
        const int h = warp >> 2;                       // row tile
        const int r = h * kTile + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // lane offset of the warp: 32 << 16
        const bool live = r < k.nrows;
        const int pos = live ? k.L - k.n + (k.row0 + r) / p.G : -1;
        // Q row into its K-major tile; a negative scale goes into Q's signs
        {
            int64_t t;
            int qh;
            attn_row_of(p, k, kvh, live ? r : 0, &t, &qh);
            const __nv_bfloat16 *src = p.q + t * p.q_ts + qh * p.q_hs;
            const int row = r & (kTile - 1);
            uint8_t *dst = base + h * Lay::kStageBytes + row * 128;
            const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int ch = 0; ch < DP / 8; ++ch) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live && 8 * ch < p.c.D)
                    v = ld_stream(src + 8 * ch);
                v.x ^= flip;
                v.y ^= flip;
                v.z ^= flip;
                v.w ^= flip;
                if constexpr (Q4)
                    v = pair_order(v);
                *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (kTile * 128) +
                                           (((ch & 7) ^ (row & 7)) << 4)) = v;
            }
            fence_async();
            bar_arrive(&sh.q_full);
        }
        const float scale = fabsf(p.scale_log2);
        const int lo_r = p.window ? pos - p.window + 1 : 0;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        if (h < halves) {
            for (int j = 0; j < nt && ok; ++j) {
                const int j0 = k.tile_at(i0 + j) * kTile;
                ok = bar_wait(&sh.s_full[h], j & 1, &sh.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                uint32_t s[kTile];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tm_load32(s + 32 * c, tm_s[h] + lanes + 32 * c);
                tm_wait_load();
                if (!attn_all_see(p, k, j0, kTile)) {
                    const int hi_c = pos - j0, lo_c = lo_r - j0, sink_c = p.n_sink - j0;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!(c <= hi_c && (c >= lo_c || c < sink_c)))
                            s[c] = 0xff800000u;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTile; ++c)
                    mx4[c & 3] = fmaxf(mx4[c & 3], __uint_as_float(s[c]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale;
                if (__any_sync(0xffffffffu, mx > m + kSlack)) {
                    const float mn = fmaxf(m, mx);
                    const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                    m = mn;
                    l *= f;
                    if (j) {
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t o[32];
                            tm_load32(o, tm_o[h] + lanes + 32 * c);
                            tm_wait_load();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tm_store32(tm_o[h] + lanes + 32 * c, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < kTile; c += 2) {
                    const float a = exp2_fast(fmaf(__uint_as_float(s[c]), scale, -ref));
                    const float b = exp2_fast(fmaf(__uint_as_float(s[c + 1]), scale, -ref));
                    sum[(c >> 1) & 3] += a + b;
                    s[c >> 1] = pack2(a, b);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tm_store32(tm_s[h] + lanes, s);
                tm_store32(tm_s[h] + lanes + 32, s + 32);
                tm_wait_store();
                tc_fence_before();
                bar_arrive(&sh.p_full[h]);
            }
            if (nt > 0 && ok)
                ok = __all_sync(0xffffffffu, bar_wait(&sh.o_full[h], 0, &sh.abort));
            tc_fence_after();
            const bool only = nparts == 1;
            const bool poison = *reinterpret_cast<volatile int *>(&sh.poison) != 0;
            if (poison) {
                for (int rr = r - lane; rr < min(r - lane + 32, k.nrows); ++rr) {
                    float pm, pl, po[E];
                    attn_row_exact<DP, Q4>(p, k, kvh, rr, i0, i0 + nt, &pm, &pl, po);
                    attn_emit<E>(p, k, kvh, rr, part, only, pm, pl, po);
                }
            } else {
                int64_t t;
                int qh;
                attn_row_of(p, k, kvh, live ? r : 0, &t, &qh);
                const bool empty = pos < 0;
                const float inv = 1.f / l;
                const int64_t wrow = ((int64_t)part * p.T + t) * p.Hq + qh;
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    if (nt > 0) {
                        tm_load32(o, tm_o[h] + lanes + 32 * c);
                        tm_wait_load();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = 0u;
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int d = 32 * c + 8 * g;
                        if (!live || d >= p.c.D)
                            continue;
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int at = Q4 ? (e < 4 ? 2 * e : 2 * e - 7) : e;
                            f[e] = __uint_as_float(o[8 * g + at]);
                            if (only)
                                f[e] = empty ? 0.f : f[e] * inv;
                        }
                        if (only) {
                            *reinterpret_cast<uint4 *>(p.out + t * p.o_ts + (int64_t)qh * p.c.D +
                                                       d) = pack8(f);
                        } else {
                            float4 *w = reinterpret_cast<float4 *>(p.ws_o + wrow * p.c.D + d);
                            w[0] = make_float4(f[0], f[1], f[2], f[3]);
                            w[1] = make_float4(f[4], f[5], f[6], f[7]);
                        }
                    }
                }
                if (live) {
                    if (!only)
                        p.ws_ml[wrow] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[t * p.Hq + qh] =
                            empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
                }
            }
        }
    } else {
    regs_down<72>();
    if (warp == 8) {
        // ================================================ matrix instructions, one lane
        if (lane == 0) {
            constexpr uint32_t kId = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(kTile / 16) << 24;
            constexpr uint32_t kIdS = kId | (uint32_t)(kTile / 8) << 17;
            constexpr uint32_t kIdO = kId | 1u << 16 | (uint32_t)(DP / 8) << 17;
            const uint64_t dk = desc_base(16), dv = desc_base(kTile * 128);
            const uint32_t q_at = smem_u32(base), ring_at = smem_u32(ring);
            bool ok = bar_wait(&sh.q_full, 0, &sh.abort);
            for (int j = -1; j < nt && ok; ++j) {
                // items of the ring: K(0) V(0) K(1) V(1) ...
                const int iv = 2 * j + 1, ik = 2 * j + 2;
                const int sv = iv % NST, sk = ik % NST;
                if (j >= 0) {
                    ok = bar_wait(&sh.raw[sv], (iv / NST) & 1, &sh.abort);
                    if (!ok)
                        break;
                }
                const bool next = j + 1 < nt;
                bool have_k = false;
                for (int h = 0; h < halves && ok; ++h) {
                    if (j >= 0) {
                        ok = bar_wait(&sh.p_full[h], j & 1, &sh.abort);
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int s = 0; s < kTile / 16; ++s)
                            mma_ts(tm_o[h], tm_s[h] + 8 * s,
                                   desc_at(dv, ring_at + sv * Lay::kStageBytes + s * 2048), kIdO,
                                   j > 0 || s > 0);
                        if (!next)
                            tc_commit(&sh.o_full[h]);
                    }
                    if (next) {
                        if (!have_k) {
                            ok = bar_wait(&sh.raw[sk], (ik / NST) & 1, &sh.abort);
                            if (!ok)
                                break;
                            tc_fence_after();
                            have_k = true;
                        }
#pragma unroll
                        for (int s = 0; s < DP / 16; ++s) {
                            const uint32_t off = (s >> 2) * (kTile * 128) + (s & 3) * 32;
                            mma_ss(tm_s[h], desc_at(dk, q_at + h * Lay::kStageBytes + off),
                                   desc_at(dk, ring_at + sk * Lay::kStageBytes + off), kIdS, s > 0);
                        }
                        tc_commit(&sh.s_full[h]);
                    }
                }
                if (!ok)
                    break;
                if (j >= 0)
                    tc_commit(&sh.empty[sv]);
                if (next)
                    tc_commit(&sh.empty[sk]);
            }
            tc_commit(&sh.drain);
            // everything issued has finished, whatever became of the rest
            for (uint32_t i = 0; i < kWaitLimit && !bar_try(&sh.drain, 0); ++i) {
            }
        }
        __syncwarp();
    } else if (!Q4 && warp == 9) {
        // ================================================ TMA
        // A lane owns one copy of a tile: `box` keys, 64 dims.  It looks its page
        // up once for K and V and asks for the next tile's before it waits.
        const int copies = kTile / map.k.box * Lay::kHalves;
        const int hf = lane % Lay::kHalves, c = lane / Lay::kHalves * map.k.box;
        const bool mine = lane < copies;
        auto look = [&](int j, int *page, int *row) {
            // a copy no row sees any key of reads zeros: a page past the last
            const int a = k.tile_at(i0 + j) * kTile + c, z = a + map.k.box;
            *page = -1;
            if (mine && j < nt && ((a < k.hi && z > k.lo) || a < k.sink))
                *page = attn_page(p, k.b, a, hf == 0);
            if (*page < 0)
                *page = p.c.n_pages;
            *row = a % p.c.page_size;
        };
        int page, row, page_next, row_next;
        look(0, &page, &row);
        bool ok = true;
        int it = 0, edges = 0;
        for (; it < 2 * nt; ++it) {
            const int st = it % NST;
            const bool is_v = it & 1;
            if (!is_v)
                look((it >> 1) + 1, &page_next, &row_next);
            if (it >= NST)
                ok = bar_wait(&sh.empty[st], (it / NST - 1) & 1, &sh.abort);
            if (!__all_sync(0xffffffffu, ok))
                break;
            // the values of a tile that not every row sees go past a clearing warp
            uint64_t *bar = &sh.raw[st];
            if (is_v && !attn_all_see(p, k, k.tile_at(i0 + (it >> 1)) * kTile, kTile))
                bar = &sh.land[edges++ & 3];
            if (lane == 0)
                bar_expect(bar, Lay::kStageBytes);
            __syncwarp();
            if (mine) {
                plane_load(is_v ? map.v : map.k,
                           smem_u32(ring + st * Lay::kStageBytes + hf * kTile * 128) + c * 128,
                           smem_u32(bar), 64 * hf, row, kvh, page);
            }
            if (is_v) {
                page = page_next;
                row = row_next;
            }
        }
        // no copy is left in flight
        if (lane == 0) {
            for (int i = it > NST ? it - NST : 0; i < it; ++i)
                for (uint32_t n = 0; n < kWaitLimit && !bar_try(&sh.raw[i % NST], (i / NST) & 1); ++n) {
                }
            for (int i = edges > 4 ? edges - 4 : 0; i < edges; ++i)
                for (uint32_t n = 0; n < kWaitLimit && !bar_try(&sh.land[i & 3], (i >> 2) & 1); ++n) {
                }
        }
        __syncwarp();
    } else if (!Q4 && (warp == 10 || warp == 11)) {
        // ================================================ values no row, or not every row, sees
        // the two warps take such tiles in turn
        const bool mixed = k.p_first != k.p_last;
        int edges = 0;
        for (int j = 0; j < nt; ++j) {
            const int j0 = k.tile_at(i0 + j) * kTile;
            if (attn_all_see(p, k, j0, kTile))
                continue;
            const int e = edges++;
            if ((e & 1) != warp - 10)
                continue;
            const int st = (2 * j + 1) % NST;
            if (!__all_sync(0xffffffffu, bar_wait(&sh.land[e & 3], (e >> 2) & 1, &sh.abort)))
                break;
            uint8_t *tile = ring + st * Lay::kStageBytes;
            bool bad = false;
            // 4 rows of 128 bytes at a time, 8 lanes each
#pragma unroll 4
            for (int rr = lane >> 3; rr < kTile; rr += 4) {
                const bool seen = attn_block_sees(k, j0 + rr);
#pragma unroll
                for (int hf = 0; hf < Lay::kHalves; ++hf) {
                    uint4 *at = reinterpret_cast<uint4 *>(tile + hf * kTile * 128 + rr * 128 +
                                                          (lane & 7) * 16);
                    if (!seen) {
                        *at = make_uint4(0, 0, 0, 0);
                    } else if (mixed) {
                        const uint4 v = *at;
                        bad |= nonfinite2(v.x) | nonfinite2(v.y) | nonfinite2(v.z) | nonfinite2(v.w);
                    }
                }
            }
            if (bad)
                *reinterpret_cast<volatile int *>(&sh.poison) = 1;
            fence_async();
            __syncwarp();
            if (lane == 0)
                bar_arrive(&sh.raw[st]);
        }
    } else if (Q4 && warp >= 12) {
        // ================================================ 4 bits to bf16, one key a thread
        const int row = threadIdx.x - 384;
        constexpr int GR = DP / 32;
        uint32_t code[4 * GR], sc[GR / 2];
        auto fetch = [&](int it) {
            const int j = k.tile_at(i0 + (it >> 1)) * kTile + row;
            const bool is_v = it & 1;
#pragma unroll
            for (int i = 0; i < 4 * GR; ++i)
                code[i] = 0x88888888u;
#pragma unroll
            for (int i = 0; i < GR / 2; ++i)
                sc[i] = 0u;
            if (attn_block_sees(k, j)) {
                const int page = attn_page(p, k.b, j, true);
                if (page >= 0) {
                    const int pr = j % p.c.page_size;
                    const uint8_t *src = row_ptr(is_v ? p.c.v : p.c.k, page, pr, kvh);
                    const uint8_t *ss = row_ptr(is_v ? p.c.vs : p.c.ks, page, pr, kvh);
#pragma unroll
                    for (int i = 0; i < GR; ++i) {
                        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
                        code[4 * i] = v.x;
                        code[4 * i + 1] = v.y;
                        code[4 * i + 2] = v.z;
                        code[4 * i + 3] = v.w;
                    }
                    if constexpr (GR == 4) {
                        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(ss));
                        sc[0] = v.x;
                        sc[1] = v.y;
                    } else {
                        sc[0] = __ldcs(reinterpret_cast<const uint32_t *>(ss));
                    }
                }
            }
        };
        const bool mixed = k.p_first != k.p_last;
        bool ok = true;
        if (nt > 0)
            fetch(0);
        for (int it = 0; it < 2 * nt && ok; ++it) {
            const int st = it % NST;
            const bool is_v = it & 1;
            if (it >= NST) {
                ok = __all_sync(0xffffffffu, bar_wait(&sh.empty[st], (it / NST - 1) & 1, &sh.abort));
                if (!ok)
                    break;
            }
            if (is_v && mixed && !attn_all_see(p, k, k.tile_at(i0 + (it >> 1)) * kTile, kTile)) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i < GR / 2; ++i)
                    bad |= nonfinite2(sc[i]);
                if (bad)
                    *reinterpret_cast<volatile int *>(&sh.poison) = 1;
            }
            uint8_t *dst = ring + st * Lay::kStageBytes + row * 128;
#pragma unroll
            for (int w = 0; w < GR; ++w) {
                const uint32_t s1 = w & 1 ? sc[w / 2] >> 16 : sc[w / 2] & 0xffffu;
                const uint32_t s2 = s1 | s1 << 16;
                const __nv_bfloat162 sv = *reinterpret_cast<const __nv_bfloat162 *>(&s2);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // the eight elements 32w + 8c ..: a word of K, two half words of V
                    uint32_t n;
                    if (is_v)
                        n = __byte_perm(code[GR * c + w / 2], code[GR * c + GR / 2 + w / 2],
                                        w & 1 ? 0x7632 : 0x5410);
                    else
                        n = code[GR * c + w];
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b = sub136(nibbles(n, i));
                        const __nv_bfloat162 f =
                            __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&b), sv);
                        o[i] = *reinterpret_cast<const uint32_t *>(&f);
                    }
                    const int ch = 4 * w + c;
                    *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (kTile * 128) +
                                               (((ch & 7) ^ (row & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            fence_async();
            bar_arrive(&sh.raw[st]);
            if (it + 1 < 2 * nt)
                fetch(it + 1);
        }
    }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
    if (threadIdx.x == 0 && sh.abort)
        atomicOr(p.status, kStatusWait);
}

template <int DP, bool Q4>
cudaError_t tiles_launch(const AttnParams &p, const CacheMaps &map, cudaStream_t stream)
{
    auto fn = attn_tiles_kernel<DP, Q4>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(fn), Layout<DP>::kBytes);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)(p.n_blocks * p.c.Hkv * p.nsplit));
    return launch(fn, grid, dim3(Q4 ? 512 : 384), Layout<DP>::kBytes, stream, 1, p, map);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnParams &p, int q4, cudaStream_t stream, LaunchRecord *rec)
{
    CacheMaps map = {};
    cudaError_t e = cudaSuccess;
    if (!q4)
        e = cache_maps(p.c, false, kTile, &map);
    if (e == cudaSuccess) {
        if (p.c.D <= 64)
            e = q4 ? tiles_launch<64, true>(p, map, stream) : tiles_launch<64, false>(p, map, stream);
        else
            e = q4 ? tiles_launch<128, true>(p, map, stream)
                   : tiles_launch<128, false>(p, map, stream);
    }
    if (e == cudaSuccess && rec) {
        rec->kernel = QKR_KERNEL_ATTN_TILES;
        rec->block = q4 ? 512 : 384;
        rec->grid = p.n_blocks * p.c.Hkv * p.nsplit;
        rec->stages = p.nsplit;
        rec->heads_per_item = p.rows;
        rec->launches += 1;
    }
    return e;
}

}  // namespace qkr
