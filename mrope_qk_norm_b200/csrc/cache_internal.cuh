// cache_internal.cuh -- what the kernels of the paged cache share: launch
// parameters, the split of the queries into blocks and of a block's keys into
// tiles, and the page look-up.
#pragma once

#include "qkr_internal.cuh"

namespace qkr {

struct CachePlane {
    uint8_t *base;
    int64_t ps, rs, hs;  // bytes between pages, rows of a page, heads
};

struct CacheView {
    CachePlane k, v, ks, vs;
    int page_size;
    int n_pages;
    int Hkv, D;
};

// A block whose keys several CTAs of the rows kernel share.
struct AttnSpan {
    int b, kvh;     // b < 0: none begins here
    int parts;      // CTAs that share it
    int slot;       // the first one's slot; the others' are their first
    int n, L;
    int64_t t0;
};

// One cache_attention call.  The queries of a sequence that share a KV head
// are numbered as rows r = i*G + g (new token i, g-th query head of the KV
// head), and a block is `rows` consecutive ones: its keys are loaded once for
// all of them.
struct AttnParams {
    CacheView c;
    const __nv_bfloat16 *q;
    int64_t q_ts, q_hs;
    __nv_bfloat16 *out;
    int64_t o_ts;
    float *lse;
    const int32_t *table, *lens, *cu;
    int64_t table_stride;
    int64_t T;
    int B, Hq, G;
    int max_q, max_len;
    int window, n_sink;      // window 0: none
    float scale_log2;        // scale * log2(e): the softmax works in powers of two
    int rows;                // rows of a block
    int rows_lo, rows_hi;    // this launch serves sequences with rows_lo < n*G <= rows_hi
    int blocks_max;          // blocks a sequence can have (max_q*G over rows)
    int direct;              // 1: block index = b*blocks_max + block; 0: blocks counted from cu
    int64_t n_blocks;        // block indices of the grid
    int tile;                // keys of a tile: 16, 32 or 64 (rows kernel), 128
    int tile_shift;          // its logarithm
    int piece_cost;          // rows kernel: what a block counts for beside its tiles
    int split_tiles;         // tiles of a part of a block's keys
    int nsplit;              // parts at most
    uint64_t page_recip;     // rows kernel: ceil(2^38 / tiles of a page)
    int ctas;                // rows kernel: CTAs that share all keys evenly; 0: a cluster a block
    int cluster;             // CTAs of such a cluster
    // Partial outputs (not divided by l), their maxima (log2 units) and sums.
    // Tiles kernel: [nsplit][T*Hq][D] and [nsplit][T*Hq].  Rows kernel: a CTA's
    // first and last piece, [2*ctas][rows][D] and [2*ctas][rows], and what the
    // CTA's last piece begins, [ctas].
    float *ws_o;
    float2 *ws_ml;
    struct AttnSpan *ws_span;
    int dense_scales;        // 4 bits: the scale rows of a page and head are one run, on 16 bytes
    unsigned *status;
};

constexpr unsigned kStatusRow = 4u, kStatusBounds = 8u, kStatusWait = 16u;

// A block of rows of one sequence and the keys it sees.
struct AttnBlock {
    int b;                   // sequence; -1: this block index is not used
    int64_t t0;              // its first token
    int n, L;                // new tokens, cached tokens
    int row0, nrows;         // first row of the block, rows in it
    int p_first, p_last;     // positions of its first and last row's token
    int lo, hi, sink;        // keys [0, sink) and [lo, hi) are seen by some row
    int c_sink, c0, ntiles;  // as tiles: c_sink from 0, then from tile c0 on
    __device__ __forceinline__ int tile_at(int i) const { return i < c_sink ? i : c0 + i - c_sink; }
};

// New tokens and start of the sequence between cu entries a and e, clamped into
// [0, T] and max_q.
__device__ __forceinline__ int attn_clamp(const AttnParams &p, int64_t a, int64_t e, int64_t *t0,
                                          bool *bad)
{
    const int64_t s = a < 0 ? 0 : (a > p.T ? p.T : a);
    int64_t n = (e > p.T ? p.T : e) - s;
    n = n < 0 ? 0 : (n > p.max_q ? p.max_q : n);
    *bad = a < 0 || e > p.T || e < a || e - a > p.max_q;
    *t0 = s;
    return (int)n;
}
__device__ __forceinline__ int attn_seq(const AttnParams &p, int b, int64_t *t0, bool *bad)
{
    return attn_clamp(p, p.cu[b], p.cu[b + 1], t0, bad);
}

// Raises the status bit if sequence b's offsets or length are outside their bounds.
// (attn_block_of does it for a sequence with blocks; clamping may leave none.)
__device__ __forceinline__ void attn_report(const AttnParams &p, int b, bool bad)
{
    const int L = p.lens[b];
    if (bad || L < 0 || L > p.max_len)
        atomicOr(p.status, kStatusBounds);
}

__device__ __forceinline__ int attn_blocks_of(const AttnParams &p, int n)
{
    const int64_t r = (int64_t)n * p.G;
    return r > p.rows_lo && r <= p.rows_hi ? (int)((r + p.rows - 1) / p.rows) : 0;
}

// Block `blk` of sequence b (n new tokens from t0 on, lens entry L) and what it sees.
__device__ __forceinline__ AttnBlock attn_block_of(const AttnParams &p, int b, int blk, int n, int L,
                                                   int64_t t0, bool bad)
{
    AttnBlock k;
    if (L < 0 || L > p.max_len) {
        bad = true;
        L = L < 0 ? 0 : p.max_len;
    }
    if (bad && (threadIdx.x & 31) == 0)
        atomicOr(p.status, kStatusBounds);
    k.b = b;
    k.t0 = t0;
    k.n = n;
    k.L = L;
    k.row0 = blk * p.rows;
    k.nrows = min(p.rows, n * p.G - k.row0);
    k.p_first = L - n + k.row0 / p.G;
    k.p_last = L - n + (k.row0 + k.nrows - 1) / p.G;
    k.hi = max(0, k.p_last + 1);
    k.lo = p.window ? max(0, k.p_first - p.window + 1) : 0;
    k.lo = min(k.lo, k.hi);
    k.sink = min(p.n_sink, k.lo);
    k.c_sink = (k.sink + p.tile - 1) / p.tile;
    k.c0 = max(k.lo / p.tile, k.c_sink);
    const int c1 = (k.hi + p.tile - 1) / p.tile;
    k.ntiles = k.c_sink + max(0, c1 - k.c0);
    return k;
}

__device__ __forceinline__ AttnBlock attn_block_at(const AttnParams &p, int b, int blk, int n,
                                                   int64_t t0, bool bad)
{
    return attn_block_of(p, b, blk, n, p.lens[b], t0, bad);
}

// The block of block index `idx`, computed by a whole warp.  Where the blocks
// are not laid out per sequence, each lane counts those of one sequence and
// the warp adds them up, 32 sequences at a time.  (Of sequences without blocks only
// those laid out per sequence are reported here.)
__device__ __forceinline__ AttnBlock attn_block(const AttnParams &p, uint32_t idx)
{
    AttnBlock none = {};
    none.b = -1;
    int b = -1, blk = 0, nblk = 0, n_of = 0;
    int64_t t0_of = 0;
    bool bad = false;
    if (p.direct) {
        b = (int)(idx / (uint32_t)p.blocks_max);
        blk = (int)(idx % (uint32_t)p.blocks_max);
        n_of = attn_seq(p, b, &t0_of, &bad);
        nblk = attn_blocks_of(p, n_of);
        if (blk >= nblk) {
            if (blk == 0 && (threadIdx.x & 31) == 0)
                attn_report(p, b, bad);
            return none;
        }
    } else {
        const int lane = threadIdx.x & 31;
        int64_t before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int mine = 0, n = 0;
            int64_t t0 = 0;
            bool mbad = false;
            if (b0 + lane < p.B) {
                n = attn_seq(p, b0 + lane, &t0, &mbad);
                mine = attn_blocks_of(p, n);
            }
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += up;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + sum > idx);
            if (past) {
                const int src = __ffs(past) - 1;
                b = b0 + src;
                nblk = __shfl_sync(0xffffffffu, mine, src);
                blk = (int)(idx - before - (__shfl_sync(0xffffffffu, sum, src) - nblk));
                n_of = __shfl_sync(0xffffffffu, n, src);
                t0_of = __shfl_sync(0xffffffffu, t0, src);
                bad = __shfl_sync(0xffffffffu, (int)mbad, src) != 0;
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (b < 0)
            return none;
    }
    // the last blocks of a sequence see most keys: they go first
    return attn_block_at(p, b, nblk - 1 - blk, n_of, t0_of, bad);
}

// Does the token at position pos see key j?
__device__ __forceinline__ bool attn_sees(const AttnParams &p, int pos, int j)
{
    return j <= pos && (p.window == 0 || pos - j < p.window || j < p.n_sink);
}

// Does any row of the block see key j?
__device__ __forceinline__ bool attn_block_sees(const AttnBlock &k, int j)
{
    return j < k.hi && (j >= k.lo || j < k.sink);
}

// Do all rows of the block see all keys of [j, j + len)?
__device__ __forceinline__ bool attn_all_see(const AttnParams &p, const AttnBlock &k, int j, int len)
{
    return j + len - 1 <= k.p_first &&
           (p.window == 0 || k.p_last - j < p.window || j + len <= p.n_sink);
}

// Page of token j of sequence b, -1 (and the status bit) where the table names none.
__device__ __forceinline__ int attn_page(const AttnParams &p, int b, int j, bool report)
{
    const int pg = p.table[(int64_t)b * p.table_stride + j / p.c.page_size];
    if ((unsigned)pg < (unsigned)p.c.n_pages)
        return pg;
    if (report)
        atomicOr(p.status, kStatusBounds);
    return -1;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where row r of the block starts in q / out / lse.
__device__ __forceinline__ void attn_row_of(const AttnParams &p, const AttnBlock &k, int kvh, int r,
                                            int64_t *t, int *h)
{
    const int row = k.row0 + r;
    *t = k.t0 + row / p.G;
    *h = kvh * p.G + row % p.G;
}

// Row r's result, by one warp: lane holds the elements [lane*E, lane*E + E) of
// the sum o over its part of the keys, m (log2 units) and l.  The only part of
// a block is divided and written out; one of several goes to the workspace.
template <int E>
__device__ __forceinline__ void attn_emit(const AttnParams &p, const AttnBlock &k, int kvh, int r,
                                          int part, bool only, float m, float l,
                                          const float (&o)[E])
{
    const int lane = threadIdx.x & 31;
    int64_t t;
    int h;
    attn_row_of(p, k, kvh, r, &t, &h);
    const int d = lane * E;
    if (!only) {
        const int64_t row = ((int64_t)part * p.T + t) * p.Hq + h;
        if (d < p.c.D) {
            float *w = p.ws_o + row * p.c.D + d;
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *reinterpret_cast<float2 *>(w + i) = make_float2(o[i], o[i + 1]);
        }
        if (lane == 0)
            p.ws_ml[row] = make_float2(m, l);
        return;
    }
    const bool empty = k.L - k.n + (k.row0 + r) / p.G < 0;  // sees nothing
    const float inv = empty ? 0.f : 1.f / l;
    if (d < p.c.D) {
        uint32_t *w = reinterpret_cast<uint32_t *>(p.out + t * p.o_ts + (int64_t)h * p.c.D + d);
#pragma unroll
        for (int i = 0; i < E; i += 2)
            w[i / 2] = empty ? 0u : pack2(o[i] * inv, o[i + 1] * inv);
    }
    if (p.lse && lane == 0)
        p.lse[t * p.Hq + h] =
            empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// CTAs of the even-shares rows kernel an SM holds.
int attn_rows_resident(int64_t D, int rows, int q4);

// Lets a kernel have `bytes` of dynamic shared memory on the current device;
// asked of the driver once for each kernel and device.
cudaError_t allow_smem(const void *fn, int bytes);

// Launchers.
cudaError_t launch_attn_rows(const AttnParams &p, int q4, cudaStream_t stream, LaunchRecord *rec);
cudaError_t launch_attn_tiles(const AttnParams &p, int q4, cudaStream_t stream, LaunchRecord *rec);
cudaError_t launch_attn_join(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_set_rows_q4(const CacheView &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                               const int64_t *rows, int64_t T, int64_t k_ts, int64_t v_ts,
                               unsigned *status, cudaStream_t stream, LaunchRecord *rec);
cudaError_t launch_get_rows_q4(const CacheView &c, __nv_bfloat16 *k, __nv_bfloat16 *v,
                               const int64_t *rows, int64_t T, int64_t k_ts, int64_t v_ts,
                               unsigned *status, cudaStream_t stream, LaunchRecord *rec);

// qkr_api.cu: records the outcome of a call for qkr_last_error / qkr_last_launch.
qkr_status api_fail(qkr_status st, const char *fmt, ...);
qkr_status api_done(const LaunchRecord &rec);

}  // namespace qkr
