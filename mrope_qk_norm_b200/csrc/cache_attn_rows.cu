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
// once), and for V^T the same 16 bytes of each of its four keys, paired key by
// key with byte permutes.
//
// One warp feeds, four compute.  The feeding warp looks the pages up and copies
// rows by TMA into a ring in shared memory, up to 96 KB ahead; the ring runs on
// from block to block, so a short sequence costs no pause.  A stage holds a step
// of every computing warp: 16 keys in bf16, 32 in 4 bits (18 KB).  A tile is what
// one copy takes: 64 keys, or 32 or 16 where the page is not a multiple of that.
// Which of 16 keys is which row of the operand is free as well; the order
// below makes the operand loads of eight lanes meet eight different banks in
// the layout the copies leave.  Where a scale row is not one of a dense run,
// its 8 (4) bytes come by cp.async.  Before this the warps loaded their own
// operands into registers (two sequences of 130,000 tokens in 4 bits, 8 KV heads of
// 128: 141 us, three warps a scheduler each waiting for its own loads; now 95), and
// with a feeding warp that copied 16 bytes a lane that warp was the bound (100,000
// tokens in bf16: 344 us against 146; now 134, 94% of the copy rate).  In 4 bits
// no unit is full (issue slots 54%, integer pipe 52%, DRAM 40%, tensor pipe 26%): a warp's
// 400 instructions a 16 keys are one chain from nibbles to the second product, and three
// computing warps a scheduler (128 registers, with spills) leave 45% of the cycles
// without one that can issue.
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
// 4 bits: a nibble n becomes the bf16 number 16 + n by a shift and one AND-OR on two
// nibbles at a time.  For K the products run on 16 + n against an accumulator
// that starts at -24 * (sum of q), per group of 32 dims, and the group's scale
// multiplies the sum in fp32.  For V the scale goes onto the weight, group by
// group, before its one rounding, and a second product takes -24 times the
// same rounded weights off again, tile by tile, so the offset never builds up
// in the sum: two matrix instructions in place of eight subtractions.  What the offset
// costs is fp32 rounding at 31 steps of a scale instead of 8.  (128 + n saves one shift in
// four, 0.5% of two sequences of 130,000 tokens, and rounds at 143 steps.)

#include <cooperative_groups.h>

#include <climits>

#include "cache_attn.cuh"
#include "cache_tma.cuh"

namespace cg = cooperative_groups;

namespace qkr {
namespace {

constexpr int kWarps = 4;              // computing warps; one more feeds them
constexpr int kThreads = 32 * (kWarps + 1);
// A wait asks so often at most, 8.6 s (an asking that fails takes some 4 us).  Roles that
// run ahead sleep in between (their polls would take issue slots from the others).
constexpr uint32_t kWaitLimit = 1u << 21;
constexpr uint32_t kMinus24 = 0xc1c0c1c0u;  // bf16 pair
constexpr float kSlack = 8.f;  // log2 units the reference may lag behind the maximum

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

template <int DP, bool Q4, int NT>
struct Rows {
    static constexpr int U = Q4 ? 2 : 1;                    // tiles a warp takes together
    static constexpr int kKeys = kWarps * U * 16;           // keys of a stage
    static constexpr int kHalves = DP / 64;
    static constexpr int kRowPart = Q4 ? DP / 2 : 128;      // bytes of a row in one copy
    static constexpr int kScale = Q4 ? DP / 16 : 0;         // bytes of its scales
    static constexpr int kPart = kKeys * (Q4 ? DP / 2 : DP * 2);   // K or V of a stage
    static constexpr int kStageBytes = 2 * (kPart + kKeys * kScale);
    static constexpr int kStages = Q4 ? (DP == 64 ? 4 : 3) : (DP == 64 ? 4 : (NT == 1 ? 3 : 2));
    // CTAs an SM holds (by shared memory and registers).  (bf16, D = 64, two tiles of rows:
    // 32 sequences of 16384, 16 heads over one: 44 us with 2 of 4 stages, 46 with 3 of 3.)
    static constexpr int kCtas = DP == 128 ? (Q4 && NT == 1 ? 3 : 2)
                                           : (NT == 1 ? (Q4 ? 4 : 3) : (Q4 ? 3 : 2));
};

// After the ring, which the copies want on a 1024-byte boundary.
template <int DP, int NT>
struct alignas(16) RowsShared {
    float o[kWarps][8 * NT][DP + 4];
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    int poison, abort;
    int beat;                  // counted up where rows are computed key by key
    int64_t scan[kWarps + 1];
    uint64_t full[4], empty[4];
};

// Which of 16 keys is row `r` of the operand, and where 16-byte chunk `ch`
// of key t of the stage lies from the start of its K or V part.
template <int DP, bool Q4>
__device__ __forceinline__ int key_of(int r)
{
    // eight 4-bit fields, key of row i in field i; rows 8..15 likewise
    constexpr uint32_t order = !Q4 ? 0x36147250u         // 0 5 2 7 4 1 6 3
                                   : (DP == 128 ? 0x65742130u
                                                : 0x67453210u); // 0 1 2 3 5 4 7 6
    return (r & 8) + (int)(order >> (4 * (r & 7)) & 7u);
}
// (Adding a multiple of 8 to t adds that many rows: the turning has period 8.)
template <int DP, bool Q4, int KEYS>
__device__ __forceinline__ int chunk_at(int t, int ch)
{
    if constexpr (!Q4)                      // 64 dims of all keys, then the next 64
        return (ch >> 3) * (KEYS * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4);
    else if constexpr (DP == 128)
        return t * 64 + ((ch ^ (t >> 1 & 3)) << 4);
    else
        return t * 32 + (ch << 4);
}

__device__ __forceinline__ uint32_t sm_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
                 "r"(take ? N : 0) : "memory");
}
__device__ __forceinline__ void full_when_copied(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm_u32(bar)) : "memory");
}
__device__ __forceinline__ void bar_init(uint64_t *bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sm_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sm_u32(bar)),
                 "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sm_u32(bar)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(sm_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded; after a wait that ran out no other waits (the result is reported as
// not valid, nothing is accessed that would not be otherwise).  Where `beat` is
// given the count starts again whenever that moves: the computing warps free no stage
// while they go through a piece key by key (16 rows: 2 us a key, so that the limit alone
// would allow some 4 million keys).
__device__ __noinline__ void bar_wait_long(uint64_t *bar, uint32_t parity, int *abort, int sleep,
                                           const int *beat)
{
    int last = beat ? *reinterpret_cast<const volatile int *>(beat) : 0;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (bar_try(bar, parity))
            return;
        if (*reinterpret_cast<volatile int *>(abort))
            return;
        if (sleep)
            __nanosleep(sleep);
        if (beat && *reinterpret_cast<const volatile int *>(beat) != last) {
            last = *reinterpret_cast<const volatile int *>(beat);
            i = 0;
        }
    }
    *reinterpret_cast<volatile int *>(abort) = 1;
}
__device__ __forceinline__ void bar_wait(uint64_t *bar, uint32_t parity, int *abort, int sleep = 0,
                                         const int *beat = nullptr)
{
    if (!__all_sync(0xffffffffu, bar_try(bar, parity)))
        bar_wait_long(bar, parity, abort, sleep, beat);
}

// A warp's place in the ring.
template <int STAGES>
struct RingAt {
    int st = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++st == STAGES) {
            st = 0;
            phase ^= 1u;
        }
    }
};

// The computing warps among themselves.
__device__ __forceinline__ void compute_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t *w, const uint8_t *p)
{
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Untiled copy of a run of scale rows; by a whole warp, as plane_load.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// The feeding warp: tiles [i0, i1) of a block and KV head into the ring from
// `at` on.  A lane owns one copy of a stage: a tile of
// K or V, 64 dims (bf16) or the codes or the scales (4 bits).
template <int DP, bool Q4, int NT>
__device__ __forceinline__ void attn_feed(const AttnParams &p, const CacheMaps &maps,
                                          const AttnBlock &k, int kvh, int i0, int i1,
                                          RowsShared<DP, NT> &sh, uint8_t *ring,
                                          RingAt<Rows<DP, Q4, NT>::kStages> *at)
{
    using R = Rows<DP, Q4, NT>;
    constexpr int KINDS = Q4 ? 4 : 2 * R::kHalves;
    const int lane = threadIdx.x & 31;
    const int box = p.tile, step = R::kKeys >> p.tile_shift;
    const int kind = lane % KINDS, first = lane / KINDS * box;
    const bool mine = first < R::kKeys;
    const bool is_v = Q4 ? kind & 1 : kind >= R::kHalves;
    const bool scales = Q4 && kind >= 2;
    const uint32_t to = 2 * R::kPart + ((is_v ? R::kKeys : 0) + first) * R::kScale;   // scales
    const uint32_t bytes = scales ? box * R::kScale : box * R::kRowPart;
    const int32_t *table = p.table + (int64_t)k.b * p.table_stride;
    // this lane's tile of the stage at tile i: false past the piece's end, else its
    // page as the table has it and the row there
    auto look = [&](int i, int *page, int *row) -> bool {
        *page = -1;
        *row = 0;
        i += first >> p.tile_shift;
        if (!mine || i >= i1)
            return false;
        const int at = k.tile_at(i);
        // division by the tiles of a page: exact for tiles below 2^26
        const int pg = (int)((uint64_t)at * p.page_recip >> 38);
        *row = (at << p.tile_shift) - pg * p.c.page_size;
        *page = table[pg];
        return true;
    };
    int page, row;
    bool wanted = look(i0, &page, &row);
    for (int i = i0; i < i1; i += step, at->next()) {
        const int st = at->st;
        const uint32_t bar = sm_u32(&sh.full[st]);
        int page_next, row_next;
        const bool wanted_next = look(i + step, &page_next, &row_next);
        if (wanted && (unsigned)page >= (unsigned)p.c.n_pages) {
            atomicOr(p.status, kStatusBounds);
            page = -1;      // reads as zeros
        }
        // (the stages' first use finds the phase before the first complete)
        bar_wait(&sh.empty[st], at->phase ^ 1u, &sh.abort, 100, &sh.beat);
        __syncwarp();
        const bool by_bulk = !scales || p.dense_scales;
        const bool issue = by_bulk && wanted && (page >= 0 || !scales);
        if (wanted && scales && p.dense_scales && page < 0) {
            for (int x = 0; x < (int)bytes; x += 16)
                *reinterpret_cast<uint4 *>(ring + st * R::kStageBytes + to + x) = make_uint4(0, 0, 0, 0);
            // the stage's next fill may copy over these zeros: not before they are there
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        uint32_t total = issue ? bytes : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, o);
        __syncwarp();       // the zeros above come before the arrival
        if (lane == 0)
            bar_expect(&sh.full[st], total);
        __syncwarp();
        // copy x of the stage: lane x's
        const int used = (R::kKeys >> p.tile_shift) * KINDS;
        const unsigned go = __ballot_sync(0xffffffffu, issue);
        const uint32_t stage = sm_u32(ring) + st * R::kStageBytes;
        int c1, c2, c3;
        plane_coords(is_v ? maps.v : maps.k, row, kvh, page < 0 ? p.c.n_pages : page, &c1, &c2, &c3);
        const CachePlane &sp = is_v ? p.c.vs : p.c.ks;
        const uint64_t from = reinterpret_cast<uint64_t>(sp.base) + kvh * sp.hs +
                              (uint64_t)(uint32_t)max(page, 0) * (uint32_t)sp.ps +
                              (uint64_t)(uint32_t)row * (uint32_t)sp.rs;
        for (int f = 0; f < used; f += KINDS) {
#pragma unroll
            for (int kd = 0; kd < KINDS; ++kd) {
                const int x = f + kd;
                const bool v = Q4 ? kd & 1 : kd >= R::kHalves;
                const int hf = Q4 ? 0 : kd % R::kHalves;
                if (Q4 && kd >= 2) {
                    const uint64_t a = __shfl_sync(0xffffffffu, from, x);
                    if (go >> x & 1u)
                        bulk_load(stage + 2 * R::kPart +
                                      ((v ? R::kKeys : 0) + f / KINDS * box) * R::kScale,
                                  reinterpret_cast<const void *>(a), box * R::kScale, bar);
                } else {
                    const int a1 = __shfl_sync(0xffffffffu, c1, x), a2 = __shfl_sync(0xffffffffu, c2, x),
                              a3 = __shfl_sync(0xffffffffu, c3, x);
                    if (go >> x & 1u)
                        plane_copy(v ? maps.v : maps.k,
                                   stage + (v ? R::kPart : 0) + hf * (R::kKeys * 128) +
                                       f / KINDS * box * R::kRowPart,
                                   bar, 64 * hf, a1, a2, a3);
                }
            }
        }
        if constexpr (Q4) {
            if (!p.dense_scales) {
                // one row a lane and step, K and V in turn
                for (int x = lane; x < 2 * R::kKeys; x += 32) {
                    const int t = x % R::kKeys, own = (t >> p.tile_shift) * KINDS + 2 + x / R::kKeys;
                    const int pg = __shfl_sync(0xffffffffu, page, own);
                    const int rw = __shfl_sync(0xffffffffu, row, own) + (t & (box - 1));
                    const CachePlane &pl = x < R::kKeys ? p.c.ks : p.c.vs;
                    const uint8_t *src = pl.base + kvh * pl.hs +
                                         (pg < 0 ? 0 : (uint64_t)pg * (uint32_t)pl.ps +
                                                           (uint64_t)(uint32_t)rw * (uint32_t)pl.rs);
                    copy_small<R::kScale>(sm_u32(ring) + st * R::kStageBytes + 2 * R::kPart +
                                              x * R::kScale, src, pg >= 0);
                }
                full_when_copied(&sh.full[st]);
            }
        }
        page = page_next;
        row = row_next;
        wanted = wanted_next;
    }
}

// No copy is left in flight (only a wait that ran out could leave one): the
// stages filled last, behind `at`, become full.
template <int STAGES, int DP, int NT>
__device__ __forceinline__ void feed_end(RowsShared<DP, NT> &sh, RingAt<STAGES> at)
{
    // of each stage the fill before `at`; a stage never filled counts as complete
    for (int i = 0; i < STAGES; ++i, at.next())
        for (uint32_t n = 0; n < kWaitLimit && !bar_try(&sh.full[at.st], at.phase ^ 1u); ++n) {
        }
}

// The tiles [i0, i1) of a block and KV head by the computing warps, out of the
// ring; each warp's maxima, sums and outputs go to sh.  Ends with their barrier.
template <int DP, int NT, bool Q4>
__device__ __forceinline__ void attn_piece(const AttnParams &p, const AttnBlock &k, int kvh, int i0,
                                           int i1, RowsShared<DP, NT> &sh, const uint8_t *ring,
                                           RingAt<Rows<DP, Q4, NT>::kStages> *at)
{
    using R = Rows<DP, Q4, NT>;
    constexpr int KS = DP / 16;       // k steps of S^T, m tiles of O^T
    constexpr int GR = DP / 32;       // 4-bit groups of a row
    constexpr int U = R::U;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;

    // ---- this block's rows: Q as the B operand, positions of a lane's columns
    uint32_t qf[NT][KS][2];
    float qs[NT][2][Q4 ? GR : 1];     // -24 * sum of q over a group, columns 2c and 2c + 1
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
                qs[n][0][w] = -24.f * __shfl_sync(0xffffffffu, sum, 8 * c);
                qs[n][1][w] = -24.f * __shfl_sync(0xffffffffu, sum, 8 * c + 4);
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
    // Tiles [in0, in1) of the piece: every row sees all their keys.
    const int sh_t = p.tile_shift;
    const int in0 =
        k.c_sink +
        (p.window ? max(0, ((max(0, k.p_last - p.window + 1) + p.tile - 1) >> sh_t) - k.c0) : 0);
    const int in1 = min(i1, k.c_sink + ((k.p_first + 1) >> sh_t) - k.c0);
    const int t0 = warp * U * 16;           // the warp's first key of a stage
    const int step = R::kKeys >> sh_t;      // tiles of a stage
    constexpr int KEYS = R::kKeys;
    const int gk = key_of<DP, Q4>(g);       // the lane's keys: gk, gk + 8 of K and S ...
    const int vk[2] = {key_of<DP, Q4>(2 * c), key_of<DP, Q4>(2 * c + 1)};   // ... these, + 8 of V
    // where the lane's operands lie in its warp's part of a stage
    const int k_off = t0 * R::kRowPart + chunk_at<DP, Q4, KEYS>(gk, Q4 ? c * (DP / 8) >> 4 : c) +
                      (Q4 ? c * (DP / 8) & 15 : 0);
    const int k_off4 = t0 * R::kRowPart + chunk_at<DP, Q4, KEYS>(gk, 4 + c);   // bf16: dims 32 on
    int v_off[2];
#pragma unroll
    for (int y = 0; y < 2; ++y)
        v_off[y] = R::kPart + t0 * R::kRowPart +
                   chunk_at<DP, Q4, KEYS>(vk[y], Q4 ? g * (DP / 16) >> 4 : g) +
                   (Q4 ? g * (DP / 16) & 15 : 0);
    const int s_off = 2 * R::kPart + (t0 + gk) * R::kScale;
    auto key_at = [&](int i, int t) {       // the token that is key t of the stage at tile i
        i += t >> sh_t;
        return i < i1 ? (k.tile_at(i) << sh_t) + (t & (p.tile - 1)) : INT_MAX / 2;
    };

    for (int i = i0; i < i1; i += step, at->next()) {
        const int st = at->st;
        bar_wait(&sh.full[st], at->phase, &sh.abort);
        if (i + (t0 >> sh_t) < i1) {
        const uint8_t *stage = ring + st * R::kStageBytes;
        const bool full = i + (t0 >> sh_t) >= in0 && i + ((t0 + 16 * U - 1) >> sh_t) < in1;

        // S^T: lane has keys g, g + 8 (elements 0 and 1, 2 and 3) of columns 2c, 2c + 1
        float s[U][NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
            if constexpr (Q4) {
                uint32_t kw[2][GR], ks[2][GR / 2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    lds_words<GR>(kw[y], stage + k_off + (16 * u + 8 * y) * R::kRowPart);
                    lds_words<GR / 2>(ks[y], stage + s_off + (16 * u + 8 * y) * R::kScale);
                }
#pragma unroll
                for (int w = 0; w < GR; ++w) {
                    uint32_t a[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        a[2 * x] = nibbles16(kw[0][w], x);
                        a[2 * x + 1] = nibbles16(kw[1][w], x);
                    }
                    const float s0 = bf16_at(ks[0][w / 2], w & 1);
                    const float s1 = bf16_at(ks[1][w / 2], w & 1);
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
                for (int w = 0; w < GR; ++w) {
                    const uint8_t *kp = stage + (w & 1 ? k_off4 : k_off) + (w >> 1) * (KEYS * 128) +
                                        16 * u * R::kRowPart;
                    const uint4 a = *reinterpret_cast<const uint4 *>(kp);
                    const uint4 b = *reinterpret_cast<const uint4 *>(kp + 8 * R::kRowPart);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(s[u][n], a.x, b.x, a.y, b.y, qf[n][2 * w][0], qf[n][2 * w][1]);
                        mma16816(s[u][n], a.z, b.z, a.w, b.w, qf[n][2 * w + 1][0],
                                 qf[n][2 * w + 1][1]);
                    }
                }
            }
        }

#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[u][n][e] *= p.scale_log2;
        if (!full) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j0 = key_at(i, t0 + 16 * u);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!attn_sees(p, pos[n][e & 1], j0 + gk + 8 * (e >> 1)))
                            s[u][n][e] = -INFINITY;
            }
        }
        bool raise = false;
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
            // the second of two tiles may lie beyond the piece: nothing was copied there
            if (u && i + ((t0 + 16 * u) >> sh_t) >= i1)
                break;
            const int j0 = full ? 0 : key_at(i, t0 + 16 * u);
            if constexpr (Q4) {
                uint32_t vw[4][GR / 2], vs[2][GR / 2];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    lds_words<GR / 2>(vw[y], stage + v_off[y & 1] +
                                                 (16 * u + 8 * (y >> 1)) * R::kRowPart);
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    lds_words<GR / 2>(vs[y], stage + s_off + (KEYS + 16 * u + 8 * y) * R::kScale);
                if (!full) {
                    // 0 * NaN: a key no row sees becomes zero; one that only some
                    // rows see must not reach the others
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int w = 0; w < GR / 2; ++w) {
                            if (!attn_block_sees(k, j0 + gk + 8 * y))
                                vs[y][w] = 0u;
                            poison |= k.p_first != k.p_last && nonfinite2(vs[y][w]);
                        }
                }
#pragma unroll
                for (int w = 0; w < GR; ++w) {
                    uint32_t b[NT][2];
                    const float s0 = bf16_at(vs[0][w / 2], w & 1);
                    const float s1 = bf16_at(vs[1][w / 2], w & 1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b[n][0] = transpose8(pack2(s[u][n][0] * s0, s[u][n][1] * s0));
                        b[n][1] = transpose8(pack2(s[u][n][2] * s1, s[u][n][3] * s1));
                    }
                    const int sel = w & 1 ? 0x7632 : 0x5410;
                    const uint32_t lo = __byte_perm(vw[0][w / 2], vw[1][w / 2], sel);
                    const uint32_t hi = __byte_perm(vw[2][w / 2], vw[3][w / 2], sel);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a0 = nibbles16(lo, 2 * y), a1 = nibbles16(lo, 2 * y + 1);
                        const uint32_t a2 = nibbles16(hi, 2 * y), a3 = nibbles16(hi, 2 * y + 1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(o[n][2 * w + y], a0, a1, a2, a3, b[n][0], b[n][1]);
                            mma16816(o[n][2 * w + y], kMinus24, kMinus24, kMinus24, kMinus24,
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
                for (int h = 0; h < DP / 64; ++h) {
                    uint4 v[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        v[y] = *reinterpret_cast<const uint4 *>(
                            stage + v_off[y & 1] + (16 * u + 8 * (y >> 1)) * R::kRowPart +
                            h * (KEYS * 128));
                    if (!full) {
                        // 0 * NaN: a key no row sees becomes zero; one that only
                        // some rows see must not reach the others
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (!attn_block_sees(k, j0 + vk[y & 1] + 8 * (y >> 1)))
                                v[y] = make_uint4(0, 0, 0, 0);
                            poison |= k.p_first != k.p_last &&
                                      (nonfinite2(v[y].x) | nonfinite2(v[y].y) |
                                       nonfinite2(v[y].z) | nonfinite2(v[y].w));
                        }
                    }
                    const uint32_t q0[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                    const uint32_t q1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
                    const uint32_t q2[4] = {v[2].x, v[2].y, v[2].z, v[2].w};
                    const uint32_t q3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = __byte_perm(q0[w], q1[w], 0x5410);
                        const uint32_t a1 = __byte_perm(q0[w], q1[w], 0x7632);
                        const uint32_t a2 = __byte_perm(q2[w], q3[w], 0x5410);
                        const uint32_t a3 = __byte_perm(q2[w], q3[w], 0x7632);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816(o[n][4 * h + w], a0, a1, a2, a3, b[n][0], b[n][1]);
                    }
                }
            }
        }
        }
        __syncwarp();
        if (lane == 0)
            bar_arrive(&sh.empty[st]);
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
    compute_sync();
}

template <int DP, int NT>
__device__ __forceinline__ void rows_setup(RowsShared<DP, NT> &sh, int fills)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            bar_init(&sh.full[i], fills);
            bar_init(&sh.empty[i], kWarps);
        }
        sh.poison = 0;
        sh.abort = 0;
        sh.beat = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}

// Row r of the piece: the warps' parts joined, in fixed order.
template <int DP, int NT, bool Q4>
__device__ __forceinline__ void attn_piece_row(const AttnParams &p, const AttnBlock &k, int kvh,
                                               int i0, int i1, RowsShared<DP, NT> &sh, int r,
                                               float *m, float *l, float (&acc)[DP / 32])
{
    constexpr int E = DP / 32;
    const int lane = threadIdx.x & 31;
    *m = -INFINITY;
    *l = 0.f;
    if (sh.poison) {
        attn_row_exact<DP, Q4>(p, k, kvh, r, i0, i1, m, l, acc, &sh.beat);
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
__global__ void __launch_bounds__(kThreads)
attn_cluster_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps maps)
{
    constexpr int E = DP / 32;
    using R = Rows<DP, Q4, NT>;
    extern __shared__ __align__(1024) uint8_t ring[];
    auto &sh = *reinterpret_cast<RowsShared<DP, NT> *>(ring + R::kStages * R::kStageBytes);
    if (sm_u32(ring) & 1023u) {     // the copies' swizzle counts on it
        if (threadIdx.x == 0)
            atomicOr(p.status, kStatusWait);
        return;
    }
    rows_setup<DP, NT>(sh, Q4 && !p.dense_scales ? 33 : 1);
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int size = p.cluster, rank = (int)(blockIdx.x % (uint32_t)size);
    const uint32_t item = blockIdx.x / (uint32_t)size;
    const int kvh = (int)(item % (uint32_t)p.c.Hkv);
    const AttnBlock k = attn_block(p, item / (uint32_t)p.c.Hkv);
    if (k.b < 0)
        return;     // the whole cluster
    const int share = (k.ntiles + size - 1) / size;
    const int i0 = min(k.ntiles, rank * share), i1 = min(k.ntiles, i0 + share);
    RingAt<R::kStages> it;
    if (warp == kWarps) {
        attn_feed<DP, Q4, NT>(p, maps, k, kvh, i0, i1, sh, ring, &it);
        feed_end(sh, it);
    } else
        attn_piece<DP, NT, Q4>(p, k, kvh, i0, i1, sh, ring, &it);
    for (int r = warp; warp < kWarps && r < k.nrows; r += kWarps) {
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
    if (warp == 0 && lane == 0 && sh.abort)
        atomicOr(p.status, kStatusWait);
    if (size == 1)
        return;
    cluster.sync();
    // rows go round the cluster's warps; parts are added in rank order
    for (int r = rank * kWarps + warp; warp < kWarps && r < k.nrows; r += size * kWarps) {
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

// Much work: every CTA takes the same number of tiles, a block counting for
// p.piece_cost more at its front (the first loads' latency, the warps' join).
template <int DP, int NT, bool Q4>
__global__ void __launch_bounds__(kThreads, Rows<DP, Q4, NT>::kCtas)
attn_rows_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps maps)
{
    constexpr int E = DP / 32;
    using R = Rows<DP, Q4, NT>;
    extern __shared__ __align__(1024) uint8_t ring[];
    auto &sh = *reinterpret_cast<RowsShared<DP, NT> *>(ring + R::kStages * R::kStageBytes);
    if (sm_u32(ring) & 1023u) {     // the copies' swizzle counts on it
        if (threadIdx.x == 0)
            atomicOr(p.status, kStatusWait);
        return;
    }
    rows_setup<DP, NT>(sh, Q4 && !p.dense_scales ? 33 : 1);
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
        if (blockIdx.x == 0)
            attn_report(p, b, bad);
        return attn_blocks_of(p, n)
                   ? p.piece_cost + max(1, attn_block_at(p, b, 0, n, t0, bad).ntiles)
                   : 0;
    };
    // inclusive sum over the CTA's threads, and the total.  A sequence has at most 2^25
    // tiles (2^29 keys of 16) and its piece_cost: 32 of them fit 32 bits, 160 do not.
    auto scan = [&](int v, int64_t *total) -> int64_t {
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
        int64_t add = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps + 1; ++w) {
            add += w < warp ? sh.scan[w] : 0;
            all += sh.scan[w];
        }
        *total = all;
        return v + add;
    };
    int64_t all_tiles = 0, upto = 0;
    int mine = 0;                  // of the chunk of sequences looked at last
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        int64_t total;
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
    for (int b0 = 0; b < 0; b0 += kThreads) {
        int64_t total;
        if (p.B > kThreads) {
            mine = tiles_of(b0 + threadIdx.x);
            upto = scan(mine, &total);
        } else {
            total = all_tiles;
        }
        if (at < (before + total) * Hkv) {
            const int64_t hi = (before + upto) * Hkv, lo = hi - (int64_t)mine * Hkv;
            __syncthreads();
            if (lo <= at && at < hi) {
                sh.scan[0] = b0 + threadIdx.x;
                sh.scan[1] = upto - mine;
            }
            __syncthreads();
            b = (int)sh.scan[0];
            before += sh.scan[1];
        } else {
            before += total;
        }
    }

    // The feeding warp and the computing ones walk the same pieces, each at its
    // own pace.
    const bool feeds = warp == kWarps;
    RingAt<R::kStages> it;
    bool first = true;
    // cu and lens of the next sequence are asked for while this one is worked on
    int cu0 = p.cu[b], cu1 = p.cu[b + 1], len = p.lens[b];
    while (at < end) {
        // the next sequence with rows of this launch
        int64_t t0;
        bool bad;
        int n = attn_clamp(p, cu0, cu1, &t0, &bad);
        while (!attn_blocks_of(p, n)) {
            ++b;
            cu0 = cu1;
            cu1 = p.cu[b + 1];
            len = p.lens[b];
            n = attn_clamp(p, cu0, cu1, &t0, &bad);
        }
        const AttnBlock k = attn_block_of(p, b, 0, n, len, t0, bad);
        cu0 = cu1;
        if (b + 1 < p.B) {
            cu1 = p.cu[b + 2];
            len = p.lens[b + 1];
        }
        const int tiles = max(1, k.ntiles), cost = p.piece_cost + tiles;
        const int64_t off = at - before * Hkv;
        int kvh = (int)(off / cost), from = (int)(off % cost);
        for (; kvh < Hkv && at < end; ++kvh, from = 0) {
            const int to = (int)min((int64_t)cost, from + end - at);
            const int i0 = max(0, from - p.piece_cost), i1 = max(0, to - p.piece_cost);
            const int64_t last = at - from + cost - 1;   // the block's last unit
            at += to - from;
            if (i0 == i1)
                continue;        // the share ends before the block's first tile
            if (feeds) {
                attn_feed<DP, Q4, NT>(p, maps, k, kvh, i0, min(i1, k.ntiles), sh, ring, &it);
                continue;
            }
            compute_sync();      // the last piece has been written out
            if (threadIdx.x == 0)
                sh.poison = 0;
            compute_sync();
            attn_piece<DP, NT, Q4>(p, k, kvh, i0, min(i1, k.ntiles), sh, ring, &it);
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
    if (feeds)
        feed_end(sh, it);
    else if (threadIdx.x == 0 && sh.abort)
        atomicOr(p.status, kStatusWait);
}

// Joins the pieces of the block that CTA x / used began, row x % used (`used`: the
// most rows a block of this launch has).
template <int DP>
__global__ void __launch_bounds__(32 * kWarps)
attn_rows_join_kernel(const __grid_constant__ AttnParams p, int used)
{
    constexpr int E = DP / 32;
    __shared__ float sm_o[kWarps][DP];
    __shared__ float sm_l[kWarps], sm_m[kWarps];
    pdl_wait();
    // no early launch of the next kernel: were it another even-shares one, its CTAs
    // would find the SMs unevenly full and some come a wave late (64 sequences,
    // window 1000, back to back: 39 us against 32)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = (int)(blockIdx.x / (uint32_t)used), r = (int)(blockIdx.x % (uint32_t)used);
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

// Joins the parts of the tiles kernel: a CTA takes 64 rows of a block, a warp a
// row at a time (a row has few parts, each D consecutive numbers).
constexpr int kJoinRows = 64, kJoinWarps = 8;
template <int DP>
__global__ void __launch_bounds__(32 * kJoinWarps)
attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int E = DP / 32;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = lane * E;
    const uint32_t chunks = (p.rows + kJoinRows - 1) / kJoinRows, x = blockIdx.x;
    const int r0 = (int)(x % chunks) * kJoinRows;
    const int kvh = (int)(x / chunks % (uint32_t)p.c.Hkv);
    const AttnBlock k = attn_block(p, x / chunks / (uint32_t)p.c.Hkv);
    if (k.b < 0 || r0 >= k.nrows)
        return;
    const int nparts = max(1, (k.ntiles + p.split_tiles - 1) / p.split_tiles);
    if (nparts == 1)
        return;  // written already
    const int64_t step = p.T * p.Hq;
    for (int r = r0 + warp; r < min(k.nrows, r0 + kJoinRows); r += kJoinWarps) {
        int64_t t;
        int h;
        attn_row_of(p, k, kvh, r, &t, &h);
        const int64_t row = t * p.Hq + h;
        float m = -INFINITY;
        for (int s = lane; s < nparts; s += 32)
            m = fmaxf(m, p.ws_ml[row + s * step].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
#pragma unroll 4
        for (int s = 0; s < nparts; ++s) {
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
        attn_emit<E>(p, k, kvh, r, 0, true, m, l, acc);
    }
}

template <int DP, int NT, bool Q4>
cudaError_t rows_launch(const AttnParams &p, cudaStream_t stream, LaunchRecord *rec)
{
    using R = Rows<DP, Q4, NT>;
    constexpr int smem = R::kStages * R::kStageBytes + (int)sizeof(RowsShared<DP, NT>);
    // even shares are made for CTAs that all run at once (an SM has 228 KB; 1 KB a CTA
    // is the system's)
    static_assert(R::kCtas * (smem + 1024) <= 228 * 1024);
    CacheMaps maps;
    auto fn = p.ctas ? attn_rows_kernel<DP, NT, Q4> : attn_cluster_kernel<DP, NT, Q4>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(fn), smem);
    if (e == cudaSuccess)
        e = cache_maps(p.c, Q4, p.tile, &maps);
    if (e != cudaSuccess)
        return e;
    rec->grid = p.ctas ? p.ctas : p.n_blocks * p.c.Hkv * p.cluster;
    rec->cluster = p.ctas ? 1 : p.cluster;
    e = launch(fn, dim3((unsigned)rec->grid), dim3(kThreads), smem, stream, rec->cluster, p,
               maps);
    if (e == cudaSuccess && p.ctas) {
        const int64_t most = (int64_t)p.max_q * p.G;
        const int used = (int)(most < p.rows ? most : p.rows);
        e = launch(attn_rows_join_kernel<DP>, dim3((unsigned)(p.ctas * used)), dim3(32 * kWarps), 0,
                   stream, 1, p, used);
        rec->launches += 1;
    }
    return e;
}

}  // namespace

int attn_rows_resident(int64_t D, int rows, int q4)
{
    if (D <= 64)
        return rows == 8 ? (q4 ? Rows<64, true, 1>::kCtas : Rows<64, false, 1>::kCtas)
                         : (q4 ? Rows<64, true, 2>::kCtas : Rows<64, false, 2>::kCtas);
    return rows == 8 ? (q4 ? Rows<128, true, 1>::kCtas : Rows<128, false, 1>::kCtas)
                     : (q4 ? Rows<128, true, 2>::kCtas : Rows<128, false, 2>::kCtas);
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
        rec->block = kThreads;
        rec->stages = p.ctas ? p.ctas : p.cluster;
        rec->heads_per_item = p.rows;
        rec->launches += 1;
    }
    return e;
}

cudaError_t launch_attn_join(const AttnParams &p, cudaStream_t stream)
{
    const int64_t chunks = (p.rows + kJoinRows - 1) / kJoinRows;
    const dim3 grid((unsigned)(p.n_blocks * p.c.Hkv * chunks)), block(32 * kJoinWarps);
    return p.c.D <= 64 ? launch(attn_join_kernel<64>, grid, block, 0, stream, 1, p)
                       : launch(attn_join_kernel<128>, grid, block, 0, stream, 1, p);
}

}  // namespace qkr
